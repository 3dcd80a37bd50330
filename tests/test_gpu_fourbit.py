"""Linear layers in 4 bits on the GPU: the products of a training step against
the plain float64 forms of the quantised operands, gradients by differences,
whole steps with the optimizer, eager and captured."""
import numpy as np
import pytest
import torch

import _lowbit_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mb():
    import muon_newton_schulz_05_b200 as m
    torch.cuda.set_device(0)
    return m


def _f64(t):
    return t.detach().double().cpu().numpy()


def _quantized(x, numbers=None):
    """Values of the quantised x [count, rows, cols] (float64)."""
    out = []
    for m in range(x.shape[0]):
        codes, scales = ref.quantize(x[m], None if numbers is None else numbers[m])
        out.append(ref.values(codes, scales, x.shape[2]))
    return np.stack(out)


def _t(x):
    return x.transpose(0, 2, 1)


def _close(got, want, mag, terms, dtype):
    """A sum of `terms` products in fp32 (64 per step, a step off by at most
    2^-22 of the magnitudes), rounded once to dtype."""
    half = 2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -24
    tol = -(-terms // 64) * 2.0 ** -22 * mag + half * np.abs(want) * 1.001
    return np.all(np.abs(_f64(got) - want) <= tol)


@pytest.mark.parametrize("shape,tokens", [((1, 96, 160), 200), ((3, 40, 72), 33), ((2, 130, 64), 1), ((1, 768, 256), 520)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_products_of_a_step(mb, shape, tokens, dtype, p):
    from muon_newton_schulz_05_b200.fourbit import Mxfp4Linear
    count, rows, cols = shape
    g = torch.Generator().manual_seed(5)
    w = (0.05 * torch.randn(shape, generator=g)).to(dtype).cuda()
    x = torch.randn((count, tokens, cols), generator=g).to(dtype).cuda()
    dy = (1e-3 * torch.randn((count, tokens, rows), generator=g)).to(dtype).cuda()
    seed, offset, site = 99, 1 << 33, 6
    rng = torch.tensor([seed, offset], dtype=torch.int64, device="cuda")
    lin = Mxfp4Linear(shape, tokens, p=p, site=site)
    y = torch.empty(count, tokens, rows, dtype=dtype, device="cuda")
    dx, grad = torch.empty_like(x), torch.empty_like(w)
    lin.refresh(w)
    lin.forward(x, y, rng)
    lin.backward(dy, grad, dx, rng)
    assert lin.device_status() == 0

    xd = _f64(x)
    if p:
        xd = ref.dropped_f32(xd.reshape(-1, cols), p, (seed, offset), site).reshape(xd.shape)
    nr = ref.numbers16(seed, offset, site, 1, count * tokens, rows).reshape(count, tokens, rows)
    nc = ref.numbers16(seed, offset, site, 2, count * rows, tokens).reshape(count, rows, tokens)
    qx, qxt = _quantized(xd), _quantized(_t(xd))
    qw, qwt = _quantized(_f64(w)), _quantized(_t(_f64(w)))
    qdy, qdyt = _quantized(_f64(dy), nr), _quantized(_t(_f64(dy)), nc)
    for got, a, b, terms in ((y, qx, qw, cols), (grad, qdyt, qxt, tokens)):
        assert _close(got, a @ _t(b), np.abs(a) @ _t(np.abs(b)), terms, dtype)
    pre = qdy @ _t(qwt)
    mag = np.abs(qdy) @ _t(np.abs(qwt))
    if not p:
        assert _close(dx, pre, mag, rows, dtype)
    else:
        t, scale = ref.dropout_terms(p)
        keep = (ref.numbers16(seed, offset, site, 0, count * tokens, cols) >= t).reshape(pre.shape)
        # stored before the mask (one rounding), then scaled (fp32) and stored again
        half = 2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -24
        tol = scale * (-(-rows // 64) * 2.0 ** -22 * mag + (2.01 * half + 2.0 ** -23) * np.abs(pre))
        assert np.all(np.abs(_f64(dx) - np.where(keep, pre * scale, 0.0)) <= tol)
    before = grad.clone()
    lin.backward(dy, grad, None, rng, accumulate=True)
    want = qdyt @ _t(qxt) + _f64(before)
    assert _close(grad, want, np.abs(qdyt) @ _t(np.abs(qxt)) + np.abs(_f64(before)), tokens + 64, dtype)


def test_gradients_by_differences(mb):
    """With operands that 4 bits hold exactly (every block's largest magnitude is
    6, so its scale is 1), the layer is linear and its gradients are difference
    quotients of sum(dy * y), exactly."""
    from muon_newton_schulz_05_b200.fourbit import Mxfp4Linear
    g = np.random.default_rng(3)
    T, R, C = 32, 64, 96

    def grid(rows, cols):
        v = g.choice(ref.LEVELS[:7], (rows, cols)) * g.choice([-1.0, 1.0], (rows, cols))
        v[::32, :] = 6.0     # every block of 32 holds a 6, in both directions
        v[:, ::32] = 6.0
        return torch.from_numpy(v).float().cuda()
    w, x, dy = grid(R, C), grid(T, C), grid(T, R)
    rng = torch.tensor([1, 2], dtype=torch.int64, device="cuda")
    lin = Mxfp4Linear((1, R, C), T)
    y, dx, grad = (torch.empty(s, device="cuda") for s in ((T, R), (T, C), (R, C)))

    def loss(wv, xv):
        lin.refresh(wv.view(1, R, C))
        lin.forward(xv, y)
        return float((y.double() * dy.double()).sum())
    loss(w, x)
    lin.backward(dy, grad.view(1, R, C), dx, rng)
    for i, j in ((1, 1), (5, 37), (31, 95), (17, 64 + 3)):
        for t, d, base in ((x, dx, lambda v: loss(w, v)), (w, grad, lambda v: loss(v, x))):
            lo, hi = t.clone(), t.clone()
            lo[i, j], hi[i, j] = -1.0, 1.5
            assert (base(hi) - base(lo)) / 2.5 == float(d[i, j])


def test_infer_one_token_between_the_passes(mb):
    """Single tokens through the layer: the rows of a whole pass without
    dropout, and the backward pass is not disturbed."""
    from muon_newton_schulz_05_b200.fourbit import Mxfp4Linear
    shape, tokens = (2, 200, 320), 300
    g = torch.Generator().manual_seed(8)
    w = torch.randn(shape, generator=g).cuda()
    x = torch.randn((2, tokens, 320), generator=g).cuda()
    dy = torch.randn((2, tokens, 200), generator=g).cuda()
    rng = torch.tensor([4, 4], dtype=torch.int64, device="cuda")
    lin = Mxfp4Linear(shape, tokens)
    y = torch.empty(2, tokens, 200, device="cuda")
    lin.refresh(w)
    lin.forward(x, y)
    grads = []
    for disturb in (False, True):
        if disturb:
            for n in (1, 7, 300):
                out = torch.empty(2, n, 200, device="cuda")
                lin.infer(x[:, :n].contiguous(), out)
                # another kernel may add in another order: 64-term steps off by 2^-22 of the magnitudes
                mag = 5 * 2.0 ** -21 * (x[:, :n].abs().double() @ w.abs().double().transpose(1, 2)) * 4
                assert bool(((out - y[:, :n]).double().abs() <= mag).all())
        grad, dx = torch.empty(shape, device="cuda"), torch.empty_like(x)
        lin.backward(dy, grad, dx, rng)
        grads.append((grad, dx))
    assert torch.equal(grads[0][0], grads[1][0]) and torch.equal(grads[0][1], grads[1][1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_averaged_weights(mb, dtype):
    """refresh with an average gives the layer the blend: the codes of
    readout_blend's fp32 result, in both orientations."""
    from muon_newton_schulz_05_b200.fourbit import Mxfp4Linear
    shape = (2, 130, 96)
    g = torch.Generator().manual_seed(12)
    w = torch.randn(shape, generator=g).to(dtype).cuda()
    ema, blend = torch.randn(shape, generator=g).cuda(), torch.empty(shape, device="cuda")
    mb.readout_blend(w, ema, blend, w_final=0.25)
    a, b = Mxfp4Linear(shape, 3), Mxfp4Linear(shape, 3)
    a.refresh(w, ema, w_final=0.25)
    b.refresh(blend)
    for q, r in ((a.w, b.w), (a.w_t, b.w_t)):
        assert torch.equal(q.data, r.data) and torch.equal(q.scales, r.scales)
    x = torch.randn((2, 3, 96), generator=g).cuda()
    ya, yb = torch.empty(2, 3, 130, device="cuda"), torch.empty(2, 3, 130, device="cuda")
    a.infer(x, ya)
    b.infer(x, yb)
    assert torch.equal(ya, yb)


def test_first_calls_of_a_process_can_be_captured():
    """Nothing has to run before a capture: the library's first call of each
    kind in a process is one inside it, and the replay gives the eager result."""
    import subprocess
    import sys
    code = """
import torch, muon_newton_schulz_05_b200 as mb
from muon_newton_schulz_05_b200.fourbit import Mxfp4Linear
lin = Mxfp4Linear((1, 96, 160), 200, p=0.25)
w, x, dy = torch.randn(1, 96, 160, device="cuda"), torch.randn(1, 200, 160, device="cuda"), torch.randn(1, 200, 96, device="cuda")
y, grad, dx, back = (torch.zeros_like(t) for t in (dy, w, x, w))
rng = torch.tensor([1, 2], device="cuda")
def step():
    lin.refresh(w)
    lin.forward(x, y, rng)
    lin.backward(dy, grad, dx, rng)
    mb.mxfp4_dequantize(lin.w, back)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
got = [t.clone() for t in (y, grad, dx, back)]
step()
assert lin.device_status() == 0
assert all(torch.equal(a, b) and bool(a.any()) for a, b in zip(got, (y, grad, dx, back)))
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def _training(mb, seed=0):
    """Two layers with dropout between them, a bank per layer, Muon on both."""
    from muon_newton_schulz_05_b200.fourbit import Mxfp4Linear
    T, D, H = 192, 128, 256
    g = torch.Generator().manual_seed(seed)
    banks = []
    for r, c in ((H, D), (D, H)):
        p = (0.1 * torch.randn((1, r, c), generator=g)).bfloat16().cuda()
        banks.append(mb.Bank(p, torch.zeros_like(p), torch.zeros((1, r, c), device="cuda")))
    lins = [Mxfp4Linear((1, H, D), T, site=0), Mxfp4Linear((1, D, H), T, p=0.1, site=1)]
    x = torch.randn((T, D), generator=g).bfloat16().cuda()
    target = torch.randn((T, D), generator=g).bfloat16().cuda()
    rng = torch.tensor([seed, 0], dtype=torch.int64, device="cuda")
    h, y = (torch.empty(T, n, dtype=torch.bfloat16, device="cuda") for n in (H, D))
    dh, dy = torch.empty_like(h), torch.empty_like(y)
    a = torch.empty_like(h)
    ws = mb.alloc_workspace([b.shape for b in banks])
    hp = mb.Hparams(lr=0.02)
    for lin, b in zip(lins, banks):
        lin.refresh(b.param)

    def step():
        lins[0].forward(x, h)
        torch.relu_(h)
        lins[1].forward(h, y, rng)
        torch.sub(y, target, out=dy)
        lins[1].backward(dy, banks[1].grad, dh, rng)
        torch.mul(dh, (h > 0), out=a)
        lins[0].backward(a, banks[0].grad, None, rng)
        mb.muon_step(banks, hp, ws)
        for lin, b in zip(lins, banks):
            lin.refresh(b.param)
        rng[1] += 1
    return step, banks, lins, ws


def test_training_steps_eager_and_captured_agree(mb):
    step, banks, lins, ws = _training(mb)
    for _ in range(4):
        step()
    eager = [b.param.clone() for b in banks] + [b.momentum.clone() for b in banks]
    step2, banks2, lins2, ws2 = _training(mb)
    step2()                                    # also the warm-up before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step2()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager, [b.param for b in banks2] + [b.momentum for b in banks2]):
        assert torch.equal(a, b) and bool(torch.isfinite(a.float()).all())
    for lin in lins + lins2:
        assert lin.device_status() == 0
    assert mb.device_status(ws) == 0 and mb.device_status(ws2) == 0


def test_two_layers_on_two_streams(mb):
    """Layers own their workspaces: two of them run at the same time."""
    from muon_newton_schulz_05_b200.fourbit import Mxfp4Linear
    shape, tokens = (1, 300, 4096), 260
    g = torch.Generator().manual_seed(2)
    work = []
    for i in range(2):
        lin = Mxfp4Linear(shape, tokens)
        lin.refresh(torch.randn(shape, generator=g).cuda())
        x = torch.randn((tokens, 4096), generator=g).cuda()
        y = torch.empty(tokens, 300, device="cuda")
        lin.forward(x, y)
        work.append((lin, x, y, y.clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for s, (lin, x, y, want) in zip(streams, work):
            with torch.cuda.stream(s):
                lin.forward(x, y)
    torch.cuda.synchronize()
    for lin, x, y, want in work:
        assert torch.equal(y, want) and lin.device_status() == 0
