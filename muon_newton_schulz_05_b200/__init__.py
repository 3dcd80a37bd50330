"""Python binding of libmuonb200.so (B200 / sm_100a Muon optimizer step).

Argument marshalling only: every step of the optimizer runs in the library's
CUDA kernels. PyTorch provides device memory and streams; the C ABI takes raw
pointers (``tensor.data_ptr()``) and a ``cudaStream_t`` (the current torch
stream unless one is given). Importing this module fails if the compiled
library is missing; build it with ``python muon_newton_schulz_05_b200/build.py``.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass, field
from typing import List, Optional, Sequence, Tuple

_PKG = os.path.dirname(os.path.abspath(__file__))
# MUON_B200_CHECK=1 selects the debug build with device-side bounds checks
# (`build.py --check`); the default is the release library.
LIB_PATH = os.path.join(_PKG, "libmuonb200_check.so" if os.environ.get("MUON_B200_CHECK") == "1"
                        else "libmuonb200.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python muon_newton_schulz_05_b200/build.py"
        f"{' --check' if LIB_PATH.endswith('_check.so') else ''}` "
        "(this package has no fallback implementation)")

_lib = ctypes.CDLL(LIB_PATH)

MAX_NS_STEPS = 16
MAX_BANKS = 8
F32, BF16 = 0, 1

STATUS_NAMES = {
    0: "MUON_OK", 1: "MUON_ERR_NULL", 2: "MUON_ERR_SHAPE", 3: "MUON_ERR_DTYPE",
    4: "MUON_ERR_ALIGN", 5: "MUON_ERR_HPARAM", 6: "MUON_ERR_WORKSPACE", 7: "MUON_ERR_CUDA",
    8: "MUON_ERR_TIMEOUT", 9: "MUON_ERR_ALIAS", 10: "MUON_ERR_BOUNDS",
}

EXPORTED = ("muon_abi_version", "muon_status_string", "muon_workspace_size", "muon_step",
            "anvil_step", "muon_orthogonalize", "ema_update", "readout_blend",
            "muon_device_status", "muon_set_debug", "muon_set_ns_events",
            "muon_orthogonalize_static", "muon_chain_plan",
            "muon_dropout", "muon_mxfp4_data_size", "muon_mxfp4_scales_size", "muon_mxfp4_quantize",
            "muon_mxfp4_readout", "muon_mxfp4_dequantize", "muon_mxfp4_matmul_workspace_size",
            "muon_mxfp4_matmul")


class MuonError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {status_string(code)}")


class CBank(ctypes.Structure):
    _fields_ = [("count", ctypes.c_int64), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("param", ctypes.c_void_p), ("param_dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("grad", ctypes.c_void_p),
                ("momentum", ctypes.c_void_p), ("momentum_slow", ctypes.c_void_p),
                ("ema", ctypes.c_void_p)]


class CHparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("mu", ctypes.c_float),
                ("weight_decay", ctypes.c_float), ("eps", ctypes.c_float),
                ("nesterov", ctypes.c_int32), ("ns_steps", ctypes.c_int32),
                ("coeffs", ctypes.c_float * (3 * MAX_NS_STEPS)), ("ema_beta", ctypes.c_float),
                ("beta_fast", ctypes.c_float), ("beta_slow", ctypes.c_float),
                ("sgd_momentum", ctypes.c_int32)]


class CMxfp4(ctypes.Structure):
    _fields_ = [("count", ctypes.c_int64), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("data", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


_vp, _i32, _i64, _sz, _f = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
_sig = {
    "muon_abi_version": (_i32, []),
    "muon_status_string": (ctypes.c_char_p, [_i32]),
    "muon_workspace_size": (_sz, [ctypes.POINTER(CBank), _i32]),
    "muon_step": (_i32, [ctypes.POINTER(CBank), _i32, ctypes.POINTER(CHparams), _vp, _sz, _vp]),
    "anvil_step": (_i32, [ctypes.POINTER(CBank), _i32, ctypes.POINTER(CHparams), _vp, _sz, _vp]),
    "muon_orthogonalize": (_i32, [_vp, _i32, _vp, _i32, _i64, _i64, _i64,
                                  ctypes.POINTER(CHparams), _vp, _sz, _vp]),
    "ema_update": (_i32, [ctypes.POINTER(CBank), _i32, _f, _vp]),
    "readout_blend": (_i32, [_vp, _i32, _vp, _vp, _i32, _i64, _f, _vp]),
    "muon_device_status": (_i32, [_vp, _sz, _vp, _i32]),
    "muon_set_debug": (_i32, [_i32, ctypes.c_double]),
    "muon_set_ns_events": (_i32, [_vp, _vp]),
    "muon_chain_plan": (_i64, [ctypes.POINTER(_i64), _i32, _i32, ctypes.POINTER(_i32), _i64]),
    "muon_orthogonalize_static": (_i32, [_vp, _i32, _vp, _i32, _i64, _i64, _i64,
                                         ctypes.POINTER(CHparams), _vp]),
    "muon_dropout": (_i32, [_vp, _vp, _vp, _i32, _i64, _i64, ctypes.c_double, _vp, ctypes.c_uint64, _vp]),
    "muon_mxfp4_data_size": (_sz, [_i64, _i64, _i64]),
    "muon_mxfp4_scales_size": (_sz, [_i64, _i64, _i64]),
    "muon_mxfp4_quantize": (_i32, [_vp, _i32, _i64, _i64, _i64, ctypes.POINTER(CMxfp4),
                                   ctypes.POINTER(CMxfp4), ctypes.c_double, _i32, _vp, ctypes.c_uint64, _vp]),
    "muon_mxfp4_readout": (_i32, [_vp, _i32, _vp, _f, _i64, _i64, _i64, ctypes.POINTER(CMxfp4),
                                  ctypes.POINTER(CMxfp4), _vp]),
    "muon_mxfp4_dequantize": (_i32, [ctypes.POINTER(CMxfp4), _vp, _i32, _vp]),
    "muon_mxfp4_matmul_workspace_size": (_sz, [_i64, _i64, _i64, _i64]),
    "muon_mxfp4_matmul": (_i32, [ctypes.POINTER(CMxfp4), ctypes.POINTER(CMxfp4), _vp, _vp, _i32, _vp, _sz,
                                 _vp]),
}
for _name, (_res, _args) in _sig.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def status_string(code: int) -> str:
    return _lib.muon_status_string(int(code)).decode()


def abi_version() -> int:
    return int(_lib.muon_abi_version())


def _check(code: int, what: str) -> None:
    if code != 0:
        raise MuonError(code, what)


# ---------------------------------------------------------------- data types
@dataclass
class Bank:
    """A bank of same-shape matrices: tensors [count, rows, cols] on one device.

    param: bf16 or fp32; grad: bf16 or fp32; momentum (M or ANVIL's M_fast),
    momentum_slow and ema: fp32 (the last two optional)."""
    param: "object"
    grad: "object"
    momentum: "object"
    momentum_slow: Optional["object"] = None
    ema: Optional["object"] = None

    @property
    def shape(self) -> Tuple[int, int, int]:
        s = tuple(self.param.shape)
        return (1, s[0], s[1]) if len(s) == 2 else s  # type: ignore[return-value]


@dataclass
class Hparams:
    lr: float = 0.02
    mu: float = 0.95
    weight_decay: float = 0.0
    eps: float = 1e-7
    nesterov: bool = True
    coeffs: Sequence[Sequence[float]] = field(default_factory=lambda: [(3.4445, -4.7750, 2.0315)] * 5)
    ema_beta: float = 0.99
    beta_fast: float = 0.9
    beta_slow: float = 0.99
    sgd_momentum: bool = False

    @classmethod
    def from_dict(cls, d: dict) -> "Hparams":
        keys = {k: d[k] for k in ("lr", "mu", "weight_decay", "eps", "nesterov", "coeffs",
                                  "ema_beta", "beta_fast", "beta_slow", "sgd_momentum") if k in d}
        return cls(**keys)

    def to_c(self) -> CHparams:
        h = CHparams()
        h.lr, h.mu, h.weight_decay, h.eps = self.lr, self.mu, self.weight_decay, self.eps
        h.nesterov = 1 if self.nesterov else 0
        h.ns_steps = len(self.coeffs)  # range checked by the library (MUON_ERR_HPARAM)
        for i, (a, b, c) in enumerate(list(self.coeffs)[:MAX_NS_STEPS]):
            h.coeffs[3 * i], h.coeffs[3 * i + 1], h.coeffs[3 * i + 2] = a, b, c
        h.ema_beta, h.beta_fast, h.beta_slow = self.ema_beta, self.beta_fast, self.beta_slow
        h.sgd_momentum = 1 if self.sgd_momentum else 0
        return h


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    return 99  # rejected by the library with MUON_ERR_DTYPE


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous")
    return t.data_ptr()


def _cbanks(banks: Sequence[Bank]):
    arr = (CBank * max(1, len(banks)))()
    for i, b in enumerate(banks):
        cnt, r, c = b.shape
        arr[i].count, arr[i].rows, arr[i].cols = cnt, r, c
        arr[i].param = _ptr(b.param)
        arr[i].param_dtype = _dtype_code(b.param)
        arr[i].grad = _ptr(b.grad)
        arr[i].grad_dtype = _dtype_code(b.grad)
        arr[i].momentum = _ptr(b.momentum)
        arr[i].momentum_slow = _ptr(b.momentum_slow)
        arr[i].ema = _ptr(b.ema)
        for t in (b.momentum, b.momentum_slow, b.ema):
            if t is not None and _dtype_code(t) != F32:
                raise ValueError("momentum buffers and the EMA must be float32")
    return arr


def _stream_handle(stream) -> Optional[int]:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


# ---------------------------------------------------------------- entry points
def workspace_size(banks_or_shapes) -> int:
    """Bytes of workspace for a list of Banks or (count, rows, cols) tuples."""
    shapes = [b.shape if isinstance(b, Bank) else tuple(b) for b in banks_or_shapes]
    arr = (CBank * max(1, len(shapes)))()
    for i, (cnt, r, c) in enumerate(shapes):
        arr[i].count, arr[i].rows, arr[i].cols = cnt, r, c
    return int(_lib.muon_workspace_size(arr, len(shapes)))


def alloc_workspace(banks_or_shapes, device="cuda"):
    """A zero-filled uint8 workspace tensor of the right size."""
    import torch
    n = workspace_size(banks_or_shapes)
    if n == 0:
        raise MuonError(2, "workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def muon_step(banks: Sequence[Bank], hp: Hparams, workspace, stream=None) -> None:
    arr = _cbanks(banks)
    h = hp.to_c()
    _check(_lib.muon_step(arr, len(banks), ctypes.byref(h), _ptr(workspace),
                          workspace.numel() * workspace.element_size(), _stream_handle(stream)),
           "muon_step")


def anvil_step(banks: Sequence[Bank], hp: Hparams, workspace, stream=None) -> None:
    arr = _cbanks(banks)
    h = hp.to_c()
    _check(_lib.anvil_step(arr, len(banks), ctypes.byref(h), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), _stream_handle(stream)),
           "anvil_step")


def orthogonalize(x, out, hp: Hparams, workspace, stream=None) -> None:
    """out = NS(x / (||x||_F + eps)) per matrix; x, out: [count, rows, cols]."""
    s = tuple(x.shape)
    cnt, r, c = (1, s[0], s[1]) if len(s) == 2 else s
    h = hp.to_c()
    _check(_lib.muon_orthogonalize(_ptr(x), _dtype_code(x), _ptr(out), _dtype_code(out), cnt, r, c,
                                   ctypes.byref(h), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(),
                                   _stream_handle(stream)), "muon_orthogonalize")


def ema_update(banks: Sequence[Bank], beta: float, stream=None) -> None:
    arr = _cbanks(banks)
    _check(_lib.ema_update(arr, len(banks), beta, _stream_handle(stream)), "ema_update")


def checkpoint_average_betas(weights: Sequence[float]) -> List[float]:
    """The beta of each ema_update call that turns the EMA recurrence into a
    weighted checkpoint average sum_i w_i theta_i / sum_i w_i: checkpoint n
    uses beta_n = 1 - w_n / (w_1 + ... + w_n) (so beta_1 = 0: the average
    starts at the first checkpoint). A checkpoint with weight 0 gets beta = 1,
    which ema_update rejects: skip its call instead. Host scalars only; the
    averaging itself is ema_update's kernel."""
    out, total = [], 0.0
    for w in weights:
        w = float(w)
        if w < 0.0:
            raise ValueError("checkpoint weights must be non-negative")
        total += w
        if total <= 0.0:
            raise ValueError("the first checkpoint needs a positive weight")
        out.append(1.0 - w / total)
    return out


def readout_blend(theta, ema, out, w_final: float = 0.35, stream=None) -> None:
    _check(_lib.readout_blend(_ptr(theta), _dtype_code(theta), _ptr(ema), _ptr(out),
                              _dtype_code(out), theta.numel(), w_final, _stream_handle(stream)),
           "readout_blend")


# ------------------------------------------------------- dropout and 4 bits
# These calls are short (a few microseconds on the device), so their host side
# is kept short too: no per-call imports, one pass over the tensors.
_torch = _u8 = None
_codes = {}


def _need_torch() -> None:
    global _torch, _u8, _codes
    if _torch is None:
        import torch
        _torch, _u8, _codes = torch, torch.uint8, {torch.float32: F32, torch.bfloat16: BF16}


def _code(t) -> int:
    """_dtype_code after _need_torch()."""
    return _codes.get(t.dtype, 99)


class Mxfp4:
    """Matrices (count, rows, cols) in microscaled 4-bit floating point, blocks
    of 32 along cols. data: the codes, scales: one byte per block in tiles of
    128 rows x 4 blocks (both uint8; the header describes the layout)."""
    __slots__ = ("data", "scales", "_shape", "_bytes", "_c", "_ref")

    def __init__(self, data, scales, shape):
        _need_torch()
        self.data, self.scales = data, scales
        self._shape = _shape3(shape)
        self._bytes = (int(_lib.muon_mxfp4_data_size(*self._shape)), int(_lib.muon_mxfp4_scales_size(*self._shape)))
        self._c = CMxfp4(*self._shape, None, None)   # the pointers are set at each call
        self._ref = ctypes.byref(self._c)

    @property
    def shape(self) -> Tuple[int, int, int]:
        return self._shape

    def __repr__(self) -> str:
        return f"Mxfp4(shape={self._shape}, device={self.data.device})"


def _shape3(shape) -> Tuple[int, int, int]:
    s = tuple(shape)
    if len(s) == 2:
        return (1, int(s[0]), int(s[1]))
    if len(s) != 3:
        raise ValueError("expected (rows, cols) or (count, rows, cols)")
    return (int(s[0]), int(s[1]), int(s[2]))


def mxfp4_storage(shape) -> Tuple[int, int]:
    """Bytes of the codes and of the scales of matrices of this shape."""
    c, r, k = _shape3(shape)
    n = int(_lib.muon_mxfp4_data_size(c, r, k))
    if n == 0:
        raise MuonError(2, "mxfp4_storage")
    return n, int(_lib.muon_mxfp4_scales_size(c, r, k))


def alloc_mxfp4(shape, device="cuda") -> Mxfp4:
    """Storage for matrices (count, rows, cols) or (rows, cols) in 4 bits."""
    import torch
    c, r, k = _shape3(shape)
    n = int(_lib.muon_mxfp4_data_size(c, r, k))
    if n == 0:
        raise MuonError(2, "alloc_mxfp4")
    data = torch.empty((c, r, n // (c * r)), dtype=torch.uint8, device=device)
    scales = torch.empty((c, -(-r // 128), -(-k // 128), 512), dtype=torch.uint8, device=device)
    return Mxfp4(data, scales, (c, r, k))


def _cmx(q: Optional[Mxfp4], what: str):
    """The C view of q, which its tensors must still fit."""
    if q is None:
        return None
    d, s, c = q.data, q.scales, q._c
    if d.dtype is not _u8 or s.dtype is not _u8:
        raise ValueError(f"{what}: data and scales must be uint8")
    n, m = q._bytes
    if n and (d.numel() != n or s.numel() != m):
        raise ValueError(f"{what}: storage of {d.numel()} + {s.numel()} bytes for {n} + {m}")
    if not d.is_contiguous() or not s.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous")
    c.data, c.scales = d.data_ptr(), s.data_ptr()
    return q._ref


def _launch(stream, fn, what, x, others, *args) -> None:
    """fn(*args, stream) with the device of the call's tensors current, on the
    given stream or that device's current one."""
    dev = x.get_device()
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError("the tensors of a call must be on one CUDA device")
    if dev < 0:
        raise ValueError("the tensors of a call must be on one CUDA device")
    if dev == _torch._C._cuda_getDevice():
        code = fn(*args, _torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream_handle(stream))
    else:
        with _torch.cuda.device(dev):
            code = fn(*args, _stream_handle(stream))
    if code != 0:
        raise MuonError(code, what)


def _rng_ptr(rng):
    if rng is None:
        return None
    _need_torch()
    if rng.dtype is not _torch.int64 or rng.numel() != 2:
        raise ValueError("rng must be two int64: (seed, offset)")
    return _ptr(rng)


def advance_rng(rng, sites: int) -> None:
    """Moves rng's offset past the numbers of a forward and backward pass whose
    calls use the sites 0 .. sites - 1. The numbers of a call depend on
    offset + site: with a smaller move, a call of the next pass repeats the
    numbers of another site's call of this one. Enqueued on the current stream
    (it can be captured)."""
    _rng_ptr(rng)
    if isinstance(sites, bool) or not isinstance(sites, int) or sites < 1:
        raise ValueError("sites must be a positive integer")
    rng[1] += sites


def dropout(x, out, p: float, rng, site: int = 0, residual=None, stream=None) -> None:
    """out = [residual +] dropout(x): elements are dropped with probability p
    (to the nearest 2^-16), the others scaled by 1 / (1 - p). x: [..., cols],
    bf16 or fp32; out may be x or residual. rng: int64 (seed, offset) on the
    device, site: the call's place within the step. The mask depends on the
    seed, offset + site, the row and the column only (see advance_rng); the
    gradient's pass is the same call on the output's gradient."""
    _need_torch()
    shape = x.shape
    if out.shape != shape or out.dtype != x.dtype:
        raise ValueError("out must have x's shape and dtype")
    if residual is not None and (residual.shape != shape or residual.dtype != x.dtype):
        raise ValueError("residual must have x's shape and dtype")
    r = _rng_ptr(rng)
    cols = shape[-1] if len(shape) else 1
    rows = x.numel() // cols if cols else 0
    _launch(stream, _lib.muon_dropout, "dropout", x, (out, rng, residual), _ptr(x), _ptr(residual), _ptr(out),
            _code(x), rows, cols, p, r, site)


def mxfp4_quantize(x, out: Optional[Mxfp4] = None, out_t: Optional[Mxfp4] = None, dropout: float = 0.0,
                   stochastic: bool = False, rng=None, site: int = 0, stream=None) -> None:
    """Quantises x ([count, rows, cols] or [rows, cols], bf16 or fp32) into out
    (blocks along cols), and its transpose into out_t (blocks along rows), from
    one read. dropout > 0 first applies dropout()'s mask and factor (of the
    same rng and site, x seen as [count * rows, cols]); stochastic rounds
    without bias, out and out_t independently. A block with an infinity or a
    NaN stands for NaN."""
    _need_torch()
    c, r, k = _shape3(x.shape)
    q, qt, g = _cmx(out, "out"), _cmx(out_t, "out_t"), _rng_ptr(rng)
    _launch(stream, _lib.muon_mxfp4_quantize, "mxfp4_quantize", x, (rng, *_storage(out), *_storage(out_t)),
            _ptr(x), _code(x), c, r, k, q, qt, dropout, 1 if stochastic else 0, g, site)


def _storage(q: Optional[Mxfp4]):
    return () if q is None else (q.data, q.scales)


def mxfp4_readout(theta, ema, out: Optional[Mxfp4] = None, out_t: Optional[Mxfp4] = None,
                  w_final: float = 0.35, stream=None) -> None:
    """Quantises the readout blend w_final theta + (1 - w_final) ema without
    storing it: the codes of readout_blend's fp32 result."""
    _need_torch()
    if ema.shape != theta.shape or _code(ema) != F32:
        raise ValueError("ema must be float32 of theta's shape")
    c, r, k = _shape3(theta.shape)
    q, qt = _cmx(out, "out"), _cmx(out_t, "out_t")
    _launch(stream, _lib.muon_mxfp4_readout, "mxfp4_readout", theta, (ema, *_storage(out), *_storage(out_t)),
            _ptr(theta), _code(theta), _ptr(ema), w_final, c, r, k, q, qt)


def mxfp4_dequantize(q: Mxfp4, out, stream=None) -> None:
    """out ([count, rows, cols] or [rows, cols], bf16 or fp32) = the values of
    q, exactly (2^128 and above become infinity)."""
    cq = _cmx(q, "q")
    shape = tuple(out.shape)
    if shape != q._shape and (q._shape[0] != 1 or shape != q._shape[1:]):
        raise ValueError("out must have q's shape")
    _launch(stream, _lib.muon_mxfp4_dequantize, "mxfp4_dequantize", out, (q.data, q.scales), cq, _ptr(out),
            _code(out))


def matmul_workspace_size(a_shape, b_shape) -> int:
    """Bytes of workspace for mxfp4_matmul of (count, m, k) and (count, n, k)."""
    (ca, m, k), (cb, n, kb) = _shape3(a_shape), _shape3(b_shape)
    if k != kb or (ca != cb and 1 not in (ca, cb)):
        return 0
    return int(_lib.muon_mxfp4_matmul_workspace_size(max(ca, cb), m, n, k))


def alloc_matmul_workspace(a_shape, b_shape, device="cuda"):
    """A zero-filled uint8 workspace for mxfp4_matmul of these shapes."""
    import torch
    n = matmul_workspace_size(a_shape, b_shape)
    if n == 0:
        raise MuonError(2, "matmul_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def mxfp4_matmul(a: Mxfp4, b: Mxfp4, out, workspace, add=None, stream=None) -> None:
    """out = [add +] a b^T: a (count, m, k), b (count, n, k), out and add
    [count, m, n] in bf16 or fp32 (out may be add). a or b with count 1 serves
    every product. Accumulates in fp32 and rounds once. The workspace may not
    be shared by calls that overlap on the device; device_status(workspace)
    reports a device-side wait that ran out."""
    ca, cb = _cmx(a, "a"), _cmx(b, "b")
    (na, m, _), (nb, n, _) = a._shape, b._shape
    shape, count = out.shape, na if na > nb else nb
    if shape != (count, m, n) and (count != 1 or shape != (m, n)):
        raise ValueError("out must be [count, a's rows, b's rows]")
    if add is not None and (add.shape != shape or add.dtype != out.dtype):
        raise ValueError("add must have out's shape and dtype")
    _launch(stream, _lib.muon_mxfp4_matmul, "mxfp4_matmul", out,
            (a.data, a.scales, b.data, b.scales, workspace, add), ca, cb, _ptr(add), _ptr(out), _code(out),
            _ptr(workspace), workspace.nbytes)


def device_status(workspace, stream=None, clear: bool = False) -> int:
    """Synchronises the stream (default: the current one of the workspace's
    device) and returns the workspace's device status code."""
    if stream is None:
        import torch
        stream = torch.cuda.current_stream(workspace.device)
    return int(_lib.muon_device_status(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                       _stream_handle(stream), 1 if clear else 0))


def set_debug(fault_mode: int = 0, wait_limit_seconds: float = 0.0) -> None:
    _check(_lib.muon_set_debug(fault_mode, wait_limit_seconds), "muon_set_debug")


def set_ns_events(before, after) -> None:
    """The next step call records these torch.cuda.Events around its
    Newton-Schulz launches (instrumentation for the benchmark)."""
    _check(_lib.muon_set_ns_events(before.cuda_event if before is not None else None,
                                   after.cuda_event if after is not None else None),
           "muon_set_ns_events")


def raw_library():
    """The ctypes handle (used by tests that call the C ABI directly)."""
    return _lib


def loaded_library_path() -> str:
    return LIB_PATH


__all__: List[str] = ["Bank", "Hparams", "MuonError", "workspace_size", "alloc_workspace",
                      "muon_step", "anvil_step", "orthogonalize", "ema_update", "readout_blend",
                      "checkpoint_average_betas",
                      "Mxfp4", "alloc_mxfp4", "mxfp4_storage", "advance_rng", "dropout", "mxfp4_quantize", "mxfp4_readout",
                      "mxfp4_dequantize", "mxfp4_matmul", "matmul_workspace_size",
                      "alloc_matmul_workspace", "CMxfp4",
                      "device_status", "set_debug", "set_ns_events", "status_string", "abi_version",
                      "raw_library", "CBank", "CHparams", "EXPORTED", "F32", "BF16"]
