"""Linear layers over a bank's matrices with products in 4 bits (MXFP4).

The three products of a layer, y = dropout(x) W^T, dx = dropout'(dy W) and
dW = dy^T dropout(x), read the parameters that an optimizer step wrote and
make the gradient that the next one reads. Each operand is quantised with its
blocks along that product's contraction: weights and activations to nearest,
the output's gradient stochastically (so that small gradients keep their
mean). The layer keeps the quantised weights between steps and the quantised
activations between the forward and the backward pass, and nothing else: masks
and random numbers are formed again from (seed, offset, site).

Every buffer is allocated once, in the constructor; the calls only enqueue
work on the current stream, so a whole training step (forward, backward, Muon
step, `refresh`) can be captured in one CUDA graph.

Random numbers depend on seed and offset + site. Call `advance(rng, layers)`
after every backward pass (of each micro-batch, where several are accumulated),
which moves the offset past all the layers' sites. A smaller step, such as one,
would give a layer the masks and roundings that its neighbour had the step
before. Processes that train on different data need seeds of their own.
"""
from __future__ import annotations

from typing import Sequence, Tuple

import muon_newton_schulz_05_b200 as mb


class Mxfp4Linear:
    """Matrices [count, rows, cols] (rows: outputs, cols: inputs) applied to
    `tokens` rows of input each. Matrices that share their input are one matrix:
    use the bank's view (1, count * rows, cols), of which dx is then one product.

    p: dropout on the input. site: the layer's place in the step, from 0 on
    (layers of a step need different ones)."""

    def __init__(self, shape, tokens: int, p: float = 0.0, site: int = 0, device="cuda"):
        count, rows, cols = (int(v) for v in shape)
        if tokens < 1:
            raise ValueError("tokens must be positive")
        if not 0 <= int(site) < 1 << 62:
            raise ValueError("site must be from 0 to 2^62 - 1")
        self.shape, self.tokens, self.p, self.site = (count, rows, cols), int(tokens), float(p), int(site)
        new = lambda *s: mb.alloc_mxfp4(s, device)  # noqa: E731
        self.w, self.w_t = new(count, rows, cols), new(count, cols, rows)
        self.x, self.x_t = new(count, tokens, cols), new(count, cols, tokens)
        self.dy, self.dy_t = new(count, tokens, rows), new(count, rows, tokens)
        # one workspace per product: they may run on different streams. The first
        # one serves `infer` with fewer tokens too, whose product may be split
        # along cols where the whole batch's is not.
        sizes = [((count, min(256 * t, tokens), cols), self.w.shape)
                 for t in range(1, min(-(-tokens // 256), 74) + 1)]
        self.ws_y = mb.alloc_matmul_workspace(*max(sizes, key=lambda s: mb.matmul_workspace_size(*s)), device)
        self.ws_dx = mb.alloc_matmul_workspace(self.dy.shape, self.w_t.shape, device)
        self.ws_dw = mb.alloc_matmul_workspace(self.dy_t.shape, self.x_t.shape, device)
        self._has_w = self._has_x = False   # `refresh` and `forward` have been called

    def _check(self, t, shape: Tuple[int, int, int], name: str) -> None:
        s = tuple(t.shape)
        if s != shape and (shape[0] != 1 or s != shape[1:]):
            raise ValueError(f"{name} must be {list(shape)}, not {list(s)}")

    def refresh(self, param, ema=None, w_final: float = 0.35) -> None:
        """Quantises the parameters (bf16 or fp32 [count, rows, cols]) for the
        passes that follow; call it after every step that changes them. With
        ema (fp32) the layer gets the readout blend w_final param + (1 - w_final)
        ema instead, which is not stored."""
        self._check(param, self.shape, "param")
        if ema is None:
            mb.mxfp4_quantize(param, self.w, self.w_t)
        else:
            self._check(ema, self.shape, "ema")
            mb.mxfp4_readout(param, ema, self.w, self.w_t, w_final=w_final)
        self._has_w = True

    def _need_weights(self) -> None:
        if not self._has_w:
            raise RuntimeError("call refresh(param) before the first pass")

    def forward(self, x, out, rng=None) -> None:
        """out [count, tokens, rows] = dropout(x) W^T; x [count, tokens, cols].
        rng is needed where p > 0."""
        count, rows, cols = self.shape
        self._check(x, (count, self.tokens, cols), "x")
        self._check(out, (count, self.tokens, rows), "out")
        self._need_weights()
        mb.mxfp4_quantize(x, self.x, self.x_t, dropout=self.p, rng=rng if self.p > 0 else None, site=self.site)
        self._has_x = True
        mb.mxfp4_matmul(self.x, self.w, out, self.ws_y)

    def infer(self, x, out) -> None:
        """out = x W^T without dropout; any number of tokens up to the layer's,
        in particular one. Leaves what the last forward pass kept for its
        backward pass. It uses the forward pass's workspace, so the two must not
        overlap on the device, nor two calls of it."""
        count, rows, cols = self.shape
        tokens = x.shape[-2]
        if not 1 <= tokens <= self.tokens:
            raise ValueError(f"x must have 1 to {self.tokens} tokens")
        self._check(x, (count, tokens, cols), "x")
        self._check(out, (count, tokens, rows), "out")
        self._need_weights()
        q = self._first_tokens(tokens)
        mb.mxfp4_quantize(x, q)
        mb.mxfp4_matmul(q, self.w, out, self.ws_y)

    def _first_tokens(self, tokens: int) -> "mb.Mxfp4":
        """The storage of `x` used for fewer tokens."""
        if tokens == self.tokens:
            return self.x
        count, _, cols = self.shape
        n, m = mb.mxfp4_storage((count, tokens, cols))
        return mb.Mxfp4(self.x.data.view(-1)[:n], self.x.scales.view(-1)[:m], (count, tokens, cols))

    def backward(self, dy, grad, dx=None, rng=None, accumulate: bool = False) -> None:
        """grad [count, rows, cols] = (or, accumulate, +=) dy^T dropout(x) and,
        if given, dx [count, tokens, cols] = dropout'(dy W), for the x of the last
        forward pass; dy [count, tokens, rows]. rng as in the forward pass (the
        offset unchanged), and needed for the rounding of dy."""
        count, rows, cols = self.shape
        self._check(dy, (count, self.tokens, rows), "dy")
        self._check(grad, self.shape, "grad")
        if dx is not None:
            self._check(dx, (count, self.tokens, cols), "dx")
        if rng is None:
            raise ValueError("backward needs rng")
        self._need_weights()
        if not self._has_x:
            raise RuntimeError("backward needs a forward pass")
        mb.mxfp4_quantize(dy, self.dy if dx is not None else None, self.dy_t, stochastic=True, rng=rng, site=self.site)
        mb.mxfp4_matmul(self.dy_t, self.x_t, grad, self.ws_dw, add=grad if accumulate else None)
        if dx is not None:
            mb.mxfp4_matmul(self.dy, self.w_t, dx, self.ws_dx)
            if self.p > 0:
                mb.dropout(dx, dx, self.p, rng, site=self.site)

    def device_status(self, clear: bool = False) -> int:
        """The first error that a product of this layer recorded (it synchronises
        the current stream). Until it is cleared, products that are split along
        their contraction leave their outputs as they were."""
        codes = [mb.device_status(ws, clear=clear) for ws in (self.ws_y, self.ws_dx, self.ws_dw)]
        return next((code for code in codes if code), 0)


def advance(rng, layers: Sequence[Mxfp4Linear]) -> None:
    """Moves rng's offset past the numbers that a forward and backward pass of
    these layers used; layers: all that draw from rng."""
    sites = [lin.site for lin in layers]
    if len(set(sites)) != len(sites):
        raise ValueError("layers of a step need different sites")
    mb.advance_rng(rng, max(sites, default=0) + 1)
