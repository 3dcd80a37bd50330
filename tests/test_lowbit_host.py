"""Dropout and the 4-bit operators on the host (no GPU needed): storage sizes,
refusals of the C ABI and of the binding, and the plain forms' own pins."""
import ctypes

import numpy as np
import pytest
import torch

import muon_newton_schulz_05_b200 as mb
import _lowbit_reference as ref

FAKE = 0x10000  # aligned, never dereferenced: validation fails first
OK, NULL, SHAPE, DTYPE, ALIGN, HPARAM, WORKSPACE, CUDA, _, ALIAS = range(10)


def test_philox_known_answers():
    """The published known-answer vectors of Philox4x32-10 (zero, ones, digits of pi)."""
    assert ref.philox([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert ref.philox([ref.M32] * 4, [ref.M32] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert ref.philox([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0]) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_numbers_are_the_documented_counters():
    seed, offset, site, domain = 0x0123456789ABCDEF, 2 ** 64 - 3, 11, 2
    got = ref.numbers16(seed, offset, site, domain, 3, 21)
    n = (offset + site) % 2 ** 64
    for r in range(3):
        for c in range(21):
            w = ref.philox([c >> 3, r, n & ref.M32, (n >> 32) & 0x3FFFFFFF | domain << 30],
                           [seed & ref.M32, seed >> 32])[(c >> 1) & 3]
            assert got[r, c] == (w >> 16 if c & 1 else w & 0xFFFF)


def test_reference_quantiser_pins():
    x = np.zeros((1, 40))
    x[0, :8] = [6.0, -0.25, 0.75, 1.25, 1.75, 2.5, -3.5, 5.0]   # ties go to the even code
    codes, scales = ref.quantize(x)
    assert scales.tolist() == [[127, 0]]
    assert ref.values(codes, scales, 8)[0].tolist() == [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, -4.0, 4.0]
    for amax, e in ((6.0, 0), (np.nextafter(6.0, 7), 1), (12.0, 1), (4.0, 0), (3.0, -1), (2.0 ** -140, -127), (0, -127)):
        assert ref.block_scale_exponent(amax) == e, amax


def test_sizes():
    lib = mb.raw_library()
    assert lib.muon_mxfp4_data_size(3, 5, 70) == 3 * 5 * 3 * 16
    assert lib.muon_mxfp4_scales_size(3, 129, 129) == 3 * 2 * 2 * 512
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, -1), (1 << 40, 1, 1), (1, 1 << 24, 1), (1, 1, 1 << 24),
                (1 << 20, 1 << 20, 1), (1 << 20, 1, 1 << 20), (1 << 12, 1 << 18, 1 << 18)):
        assert lib.muon_mxfp4_data_size(*bad) == 0 and lib.muon_mxfp4_scales_size(*bad) == 0
        with pytest.raises(mb.MuonError):
            mb.alloc_mxfp4(bad, device="cpu")
    q = mb.alloc_mxfp4((2, 5, 70), device="cpu")
    assert q.data.shape == (2, 5, 48) and q.scales.shape == (2, 1, 1, 512) and q.shape == (2, 5, 70)
    assert mb.alloc_mxfp4((5, 70), device="cpu").shape == (1, 5, 70)
    # a product's workspace: the header alone, or with partial tiles when few tiles meet a long k
    assert mb.matmul_workspace_size((1, 4096, 512), (1, 4096, 512)) == 4096
    assert mb.matmul_workspace_size((1, 200, 1 << 16), (1, 200, 1 << 16)) > 4096
    assert mb.matmul_workspace_size((2, 8, 64), (3, 8, 64)) == 0
    assert mb.matmul_workspace_size((1, 8, 64), (1, 8, 65)) == 0
    assert mb.matmul_workspace_size((1, 0, 64), (1, 8, 64)) == 0


def _mx(count=1, rows=8, cols=64, data=FAKE, scales=FAKE + 0x8000):
    return mb.CMxfp4(count, rows, cols, data, scales)


def test_dropout_refusals():
    f = mb.raw_library().muon_dropout
    x, res, out, rng = FAKE, FAKE * 2, FAKE * 3, FAKE * 4

    def call(x=x, res=None, out=out, dtype=1, rows=4, cols=8, p=0.1, rng=rng):
        return f(x, res, out, dtype, rows, cols, p, rng, 0, None)
    assert call(x=None) == NULL and call(out=None) == NULL and call(rng=None) == NULL
    for kw in (dict(rows=0), dict(cols=0), dict(rows=-1), dict(rows=1 << 31), dict(cols=1 << 24),
               dict(rows=1 << 30, cols=1 << 10)):
        assert call(**kw) == SHAPE, kw
    assert call(dtype=2) == DTYPE
    for kw in (dict(x=FAKE + 2), dict(out=FAKE * 3 + 8), dict(res=FAKE * 2 + 4), dict(rng=FAKE * 4 + 8)):
        assert call(**kw) == ALIGN, kw
    for p in (-0.1, 1.0, 1.5, float("nan"), float("inf"), 1 - 2.0 ** -18):
        assert call(p=p) == HPARAM, p
    assert call(out=FAKE + 16) == ALIAS                      # out over a part of x
    assert call(res=FAKE * 3 + 16) == ALIAS
    assert call(rng=FAKE * 3 + 16) == ALIAS
    if not torch.cuda.is_available():                        # valid: fails on the missing GPU
        assert call() == CUDA and call(out=x) == CUDA and call(res=res, out=res) == CUDA


def test_quantize_refusals():
    lib = mb.raw_library()
    q, qt = _mx(), _mx(rows=64, cols=8, data=FAKE * 2, scales=FAKE * 2 + 0x8000)

    def call(x=FAKE * 8, dtype=1, shape=(1, 8, 64), out=q, out_t=None, p=0.0, st=0, rng=None):
        return lib.muon_mxfp4_quantize(x, dtype, *shape, out, out_t, p, st, rng, 0, None)
    assert call(x=None) == NULL and call(out=None) == NULL
    assert call(p=0.1) == NULL and call(st=1) == NULL        # rng missing
    assert call(shape=(0, 8, 64)) == SHAPE and call(shape=(1, 9, 64)) == SHAPE
    assert call(out=None, out_t=q) == SHAPE                  # not the transposed shape
    assert call(shape=(1, 1 << 24, 64)) == SHAPE
    assert call(dtype=3) == DTYPE
    assert call(x=FAKE * 8 + 4) == ALIGN and call(out=_mx(data=FAKE + 8)) == ALIGN
    assert call(p=0.1, rng=FAKE * 16 + 4) == ALIGN
    assert call(p=1.0, rng=FAKE * 16) == HPARAM and call(st=2, rng=FAKE * 16) == HPARAM
    assert call(out=_mx(data=None)) == NULL and call(out=_mx(scales=None)) == NULL
    assert call(out=_mx(data=FAKE * 8 + 64)) == ALIAS        # over the source
    assert call(out=_mx(scales=FAKE + 16)) == ALIAS          # scales over the codes
    assert call(out_t=_mx(rows=64, cols=8, data=FAKE + 16, scales=FAKE * 3)) == ALIAS
    assert call(p=0.1, rng=FAKE + 16) == ALIAS
    if not torch.cuda.is_available():
        assert call(out_t=qt) == CUDA

    def readout(theta=FAKE * 8, ema=FAKE * 9, w=0.35, out=q):
        return lib.muon_mxfp4_readout(theta, 1, ema, w, 1, 8, 64, out, None, None)
    assert readout(theta=None) == NULL and readout(ema=None) == NULL and readout(out=None) == NULL
    assert readout(w=float("nan")) == HPARAM and readout(ema=FAKE * 9 + 4) == ALIGN
    assert readout(out=_mx(data=FAKE * 9 + 16)) == ALIAS

    def back(q=q, out=FAKE * 8, dtype=1):
        return lib.muon_mxfp4_dequantize(q, out, dtype, None)
    assert back(q=None) == NULL and back(out=None) == NULL and back(dtype=9) == DTYPE
    assert back(out=FAKE * 8 + 2) == ALIGN and back(out=FAKE + 16) == ALIAS
    assert back(q=_mx(rows=0)) == SHAPE


def test_matmul_refusals():
    f = mb.raw_library().muon_mxfp4_matmul
    a, b = _mx(), _mx(rows=16, data=FAKE * 2, scales=FAKE * 2 + 0x8000)

    def call(a=a, b=b, add=None, out=FAKE * 8, dtype=1, ws=FAKE * 16, n=1 << 16):
        return f(a, b, add, out, dtype, ws, n, None)
    assert call(a=None) == NULL and call(b=None) == NULL and call(out=None) == NULL
    assert call(a=_mx(cols=65)) == SHAPE                     # k differs
    assert call(a=_mx(count=2), b=_mx(count=3)) == SHAPE
    assert call(a=_mx(rows=0)) == SHAPE
    assert call(a=_mx(rows=(1 << 24) - 1), b=_mx(rows=(1 << 24) - 1)) == SHAPE   # too many tiles
    assert call(dtype=2) == DTYPE
    assert call(out=FAKE * 8 + 8) == ALIGN and call(add=FAKE * 9 + 4) == ALIGN and call(ws=FAKE * 16 + 8) == ALIGN
    assert call(ws=None) == WORKSPACE and call(n=4095) == WORKSPACE
    long = dict(a=_mx(rows=200, cols=1 << 16), b=_mx(rows=200, cols=1 << 16, data=FAKE << 12, scales=FAKE << 14))
    assert call(**long, ws=FAKE << 15, n=4096) == WORKSPACE  # split along k: needs room for the parts
    assert call(out=FAKE + 16) == ALIAS and call(add=FAKE * 8 + 16) == ALIAS
    assert call(ws=FAKE) == ALIAS and call(out=FAKE * 16 + 4096) == ALIAS and call(add=FAKE * 16) == ALIAS
    if not torch.cuda.is_available():
        assert call() == CUDA and call(add=FAKE * 8) == CUDA


def test_binding_refusals():
    x = torch.zeros(4, 64)
    rng = torch.zeros(2, dtype=torch.int64)
    q = mb.alloc_mxfp4((4, 64), device="cpu")
    ws = torch.zeros(4096, dtype=torch.uint8)
    cases = [
        lambda: mb.dropout(x, torch.zeros(4, 63), 0.1, rng),
        lambda: mb.dropout(x, x.bfloat16(), 0.1, rng),
        lambda: mb.dropout(x, x, 0.1, rng.int()),
        lambda: mb.dropout(x, x, 0.1, torch.zeros(3, dtype=torch.int64)),
        lambda: mb.dropout(x, x, 0.1, rng, residual=torch.zeros(4, 8)),
        lambda: mb.dropout(x, x, 0.1, rng),                                   # not on a CUDA device
        lambda: mb.mxfp4_quantize(torch.zeros(64), out=q),
        lambda: mb.mxfp4_quantize(x, out=q),
        lambda: mb.mxfp4_quantize(x, out=mb.Mxfp4(q.data[:2], q.scales, (4, 64))),
        lambda: mb.mxfp4_quantize(x, out=mb.Mxfp4(q.data.char(), q.scales, (4, 64))),
        lambda: mb.mxfp4_readout(x, x.bfloat16(), out=q),
        lambda: mb.mxfp4_dequantize(q, torch.zeros(4, 65)),
        lambda: mb.mxfp4_matmul(q, q, torch.zeros(4, 5), ws),
        lambda: mb.mxfp4_matmul(q, q, torch.zeros(4, 4), ws, add=torch.zeros(4, 4).bfloat16()),
        lambda: mb.mxfp4_matmul(q, q, torch.zeros(4, 4), ws),
    ]
    for f in cases:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(mb.MuonError):
        mb.alloc_matmul_workspace((1, 4, 64), (1, 4, 63), device="cpu")


def test_struct_layout():
    assert ctypes.sizeof(mb.CMxfp4) == 40 and mb.CMxfp4.data.offset == 24


def test_linear_layer_refusals():
    from muon_newton_schulz_05_b200.fourbit import Mxfp4Linear
    lin = Mxfp4Linear((2, 24, 40), tokens=7, p=0.1, device="cpu")
    assert lin.w.shape == (2, 24, 40) and lin.w_t.shape == (2, 40, 24) and lin.dy_t.shape == (2, 24, 7)
    x, y, w = torch.zeros(2, 7, 40), torch.zeros(2, 7, 24), torch.zeros(2, 24, 40)
    cases = [
        lambda: Mxfp4Linear((2, 24, 40), tokens=0, device="cpu"),
        lambda: lin.refresh(torch.zeros(24, 40)),
        lambda: lin.forward(x[:, :6], y),
        lambda: lin.forward(x, y[:1]),
        lambda: lin.infer(torch.zeros(2, 8, 40), torch.zeros(2, 8, 24)),
        lambda: lin.infer(torch.zeros(2, 0, 40), torch.zeros(2, 0, 24)),
        lambda: lin.backward(y, w),                                          # rng missing
        lambda: lin.backward(x, w, rng=torch.zeros(2, dtype=torch.int64)),
        lambda: lin.backward(y, w, dx=y, rng=torch.zeros(2, dtype=torch.int64)),
    ]
    for f in cases:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(mb.MuonError):
        Mxfp4Linear((0, 24, 40), tokens=7, device="cpu")
    # the forward workspace serves fewer tokens too: 256 rows of 80 tiles' worth are split along cols
    lin = Mxfp4Linear((1, 256, 16384), tokens=20480, device="cpu")
    for tokens in (1, 64, 65, 256, 257, 1000, 20480):
        assert lin.ws_y.numel() >= mb.matmul_workspace_size((1, tokens, 16384), lin.w.shape)


def test_linear_layer_refuses_passes_out_of_order():
    from muon_newton_schulz_05_b200.fourbit import Mxfp4Linear
    lin = Mxfp4Linear((2, 24, 40), tokens=7, device="cpu")
    x, y, w, rng = torch.zeros(2, 7, 40), torch.zeros(2, 7, 24), torch.zeros(2, 24, 40), torch.zeros(2, dtype=torch.int64)
    for f in (lambda: lin.forward(x, y), lambda: lin.infer(x[:, :1], y[:, :1]), lambda: lin.backward(y, w, rng=rng)):
        with pytest.raises(RuntimeError, match="refresh"):
            f()
    with pytest.raises(ValueError):
        lin.refresh(w, ema=x)
