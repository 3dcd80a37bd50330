"""Dropout, 4-bit quantisation and its product on the GPU against plain float64 forms.

Codes, scales, dropout masks and read-back values have to be equal bit for
bit: every intermediate is exact or rounded in a defined place. Products of
codes whose scales lie within a factor of 4 are sums of multiples of 2^-4 that
fp32 holds exactly (36 * 16 * 16 K < 2^24 up to K = 1820; the codes drawn here
average far less, and every case asserts the bound on its own data), so they
are compared for equality too. With scales of any size an fp32 sum of S = ceil(K / 64)
steps is off by at most S 2^-22 sum |a b| (each step rounds the aligned
products and the running sum, twice a bit), plus the output's half step.
"""
import ctypes

import numpy as np
import pytest
import torch

import _lowbit_reference as ref

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def mb():
    import muon_newton_schulz_05_b200 as m
    torch.cuda.set_device(0)
    return m


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _rng(seed=0x1234567890ABCDEF, offset=77):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda"), (seed, offset)


def _f64(t):
    return t.detach().double().cpu().numpy()


def _source(rows, cols, dtype, seed, spread=1.0):
    g = np.random.default_rng(seed)
    x = g.standard_normal((rows, cols)) * np.exp(spread * g.standard_normal((1, cols)))
    return torch.from_numpy(x).to(DTYPES[dtype])


# -------------------------------------------------------------------- dropout
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (3, 8), (5, 64), (33, 71), (257, 1001), (512, 1024),
                                   (700, 17), (301, 18), (129, 23), (90, 33), (1, 2050), (40, 2047), (700, 9)])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout(mb, shape, dtype, residual):
    x, r = _source(*shape, dtype, 1), _source(*shape, dtype, 2)
    rng, key = _rng()
    for p, site in ((0.0, 0), (0.1, 3), (0.75, 2 ** 63)):
        out = torch.full(shape, float("nan"), dtype=DTYPES[dtype], device="cuda")
        mb.dropout(x.cuda(), out, p, rng, site, residual=r.cuda() if residual else None)
        want = ref.dropped(_f64(x), p, key, site)
        mag = np.abs(want)
        if residual:
            want = want + _f64(r)
            mag = mag + np.abs(_f64(r))
        # the scaled value and the sum round once each in fp32, the result once more
        tol = 2.0 ** -23 * mag + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * np.abs(want) * (1 + 2.0 ** -20)
        got = _f64(out)
        assert np.all(np.abs(got - want) <= tol)
        if not residual:
            assert np.array_equal(got == 0, want == 0)


def test_dropout_in_place_and_gradient(mb):
    """The gradient of sum(w * dropout(x)) is the same call on w; by differences
    too (dropout is linear, so a difference quotient in fp64 of the plain form is exact)."""
    rng, key = _rng(5, 2 ** 40)
    x, w = _source(40, 130, "f32", 3), _source(40, 130, "f32", 4)
    gx = w.cuda().clone()
    mb.dropout(gx, gx, 0.3, rng, site=9)                    # in place
    e = 0.25
    plus = ref.dropped(_f64(x) + e, 0.3, key, 9) * _f64(w)
    minus = ref.dropped(_f64(x) - e, 0.3, key, 9) * _f64(w)
    assert np.all(np.abs(_f64(gx) - (plus - minus) / (2 * e)) <= 2.0 ** -22 * np.abs(_f64(w)) * 2)
    y = x.cuda().clone()
    mb.dropout(w.cuda(), y, 0.3, rng, site=9, residual=y)   # onto the residual
    assert np.all(np.abs(_f64(y) - (_f64(x) + _f64(gx))) <= 2.0 ** -23 * (np.abs(_f64(x)) + np.abs(_f64(gx))))


def test_dropout_rate_and_independence(mb):
    rng, _ = _rng(99, 0)
    n = 1 << 22
    x = torch.ones(1024, n // 1024, device="cuda")
    masks = []
    for site in (0, 1):
        out = torch.empty_like(x)
        mb.dropout(x, out, 0.1, rng, site)
        masks.append(out != 0)
        kept = masks[-1].double().mean().item()
        p = round(0.1 * 65536) / 65536
        assert abs(kept - (1 - p)) < 6 * (p * (1 - p) / n) ** 0.5      # six standard deviations
    both = (masks[0] & masks[1]).double().mean().item()
    assert abs(both - (1 - p) ** 2) < 6 * (0.25 / n) ** 0.5


def test_dropout_passes_infinities_and_nans(mb):
    rng, key = _rng()
    x = torch.tensor([[float("inf"), float("-inf"), float("nan")] * 40], device="cuda")
    out = torch.empty_like(x)
    mb.dropout(x, out, 0.5, rng)
    keep = torch.from_numpy(ref.numbers16(*key, 0, 0, 1, 120) >= 32768).cuda()
    assert torch.equal(torch.isnan(out), torch.isnan(x) & keep)
    assert bool((out[~keep] == 0).all()) and torch.equal(torch.isinf(out), torch.isinf(x) & keep)


# ---------------------------------------------------------------- quantisation
def _check_stored(mb, q, x, numbers=None):
    """q's bytes against the plain form of x [count, rows, cols] (float64)."""
    c = x.shape[0]
    for m in range(c):
        codes, scales = ref.quantize(x[m], None if numbers is None else numbers[m])
        data, flat = ref.pack(codes, scales)
        assert np.array_equal(q.scales[m].cpu().numpy().reshape(-1), flat)
        got = q.data[m].cpu().numpy()
        bad = np.repeat(scales == 255, 16, axis=1)
        assert np.array_equal(np.where(bad, 0, got), np.where(bad, 0, data))


SHAPES = [(1, 1, 1), (1, 1, 40), (1, 40, 1), (2, 33, 31), (1, 128, 128), (3, 129, 72), (1, 5, 300), (2, 260, 136),
          (1, 131, 1023), (2, 300, 9), (1, 200, 17), (3, 70, 35)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mode", ["nearest", "stochastic", "dropout", "both"])
def test_quantize(mb, shape, dtype, mode):
    c, r, k = shape
    x = _source(c * r, k, dtype, 11, 2.0)
    rng, key = _rng(-3, -5)
    key = (key[0] % 2 ** 64, key[1] % 2 ** 64)
    p = 0.2 if mode in ("dropout", "both") else 0.0
    st = mode in ("stochastic", "both")
    q, qt = mb.alloc_mxfp4(shape), mb.alloc_mxfp4((c, k, r))
    for t in (q.data, q.scales, qt.data, qt.scales):
        t.fill_(0xEE)
    mb.mxfp4_quantize(x.cuda().view(shape), q, qt, dropout=p, stochastic=st, rng=rng if p or st else None, site=4)
    v = _f64(x)
    if p:
        v = ref.dropped_f32(v, p, key, 4)
    v = v.reshape(shape)
    rows = ref.numbers16(*key, 4, 1, c * r, k).reshape(shape) if st else None
    cols = ref.numbers16(*key, 4, 2, c * k, r).reshape(c, k, r) if st else None
    _check_stored(mb, q, v, rows)
    _check_stored(mb, qt, v.transpose(0, 2, 1), cols)
    # one orientation alone gives the same bytes
    q1, qt1 = mb.alloc_mxfp4(shape), mb.alloc_mxfp4((c, k, r))
    kw = dict(dropout=p, stochastic=st, rng=rng if p or st else None, site=4)
    mb.mxfp4_quantize(x.cuda().view(shape), q1, **kw)
    mb.mxfp4_quantize(x.cuda().view(shape), out_t=qt1, **kw)
    assert torch.equal(q1.data, q.data) and torch.equal(q1.scales, q.scales)
    assert torch.equal(qt1.data, qt.data) and torch.equal(qt1.scales, qt.scales)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_borders_and_extremes(mb, dtype):
    """Ties, the border of two scales, zeros of both signs, values next to the
    type's ends, subnormals; infinities and NaNs make their own block NaN only."""
    lv = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    rows = []
    for e in (-126, -100, -1, 0, 5, 100, 124):
        rows.append(([6.0] + lv + [-v for v in lv] + [0.0, -0.0] + [0.1] * 15) * 1)
        rows[-1] = [v * 2.0 ** e for v in rows[-1]][:32]
    big = float(torch.finfo(DTYPES[dtype]).max)
    rows += [[0.0] * 32, [-0.0] * 32, [big] + [-big] * 31, [2.0 ** -126] * 32, [2.0 ** -133] * 32,
             [float("inf")] + [1.0] * 31, [1.0] * 31 + [float("nan")], [1.0] * 16 + [float("-inf")] + [2.0] * 15,
             [6.0 * (1 + 2.0 ** -7)] + [1.0] * 31, [1.5] * 32, [1.5 * (1 + 2.0 ** -7)] * 32]
    rows += [[1.0] * 32] * (32 - len(rows))
    x = torch.tensor(rows, dtype=torch.float64).to(DTYPES[dtype])
    q, qt = mb.alloc_mxfp4((32, 32)), mb.alloc_mxfp4((32, 32))
    mb.mxfp4_quantize(x.cuda(), q, qt)
    _check_stored(mb, q, _f64(x)[None])
    _check_stored(mb, qt, _f64(x).T[None])
    back = torch.empty(32, 32, device="cuda")
    mb.mxfp4_dequantize(q, back)
    codes, scales = ref.quantize(_f64(x))
    # the type's largest value is 1.99 * 2^127 = 3.98 * 2^126: its code stands for 4 * 2^126 = 2^128,
    # which the read-back, rounded to fp32, gives as infinity
    with np.errstate(over="ignore"):
        want = ref.values(codes, scales, 32).astype(np.float32)
    assert np.isinf(want).sum() == 32
    assert np.array_equal(back.cpu().numpy(), want, equal_nan=True)
    # dropping the only bad element leaves an ordinary block
    y = torch.ones(1, 32, device="cuda")
    y[0, 3] = float("nan")
    for off in range(64):
        rng, key = _rng(1, off)
        keep = ref.numbers16(*key, 0, 0, 1, 32)[0, 3] >= 32768
        q1 = mb.alloc_mxfp4((1, 32))
        mb.mxfp4_quantize(y, q1, dropout=0.5, rng=rng)
        assert (q1.scales.view(-1)[0].item() == 255) == bool(keep)


def test_stochastic_rounding_keeps_the_mean(mb):
    """4096 draws of one row: the mean of each element is within six standard
    deviations of the value (a draw's deviation is at most half a gap: 1)."""
    n = 4096
    row = torch.cat([torch.tensor([6.0]), torch.rand(31, generator=torch.Generator().manual_seed(1)) * 6])
    x = row.expand(n, 32).contiguous().cuda()
    rng, _ = _rng(7, 0)
    q = mb.alloc_mxfp4((n, 32))
    mb.mxfp4_quantize(x, q, stochastic=True, rng=rng)
    v = torch.empty(n, 32, device="cuda")
    mb.mxfp4_dequantize(q, v)
    assert (v.double().mean(0).cpu() - row.double()).abs().max().item() < 6 * 1.0 / n ** 0.5 + 2.0 ** -15


@pytest.mark.parametrize("shape", [(1, 768, 300), (2, 65, 129), (1, 1, 1)], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_readout(mb, shape, dtype):
    """The quantised blend is the quantised readout_blend, bit for bit."""
    c, r, k = shape
    theta = _source(c * r, k, dtype, 21).cuda().view(shape)
    ema = _source(c * r, k, "f32", 22).cuda().view(shape)
    for w in (0.35, 0.0, 1.0):
        q, qt = mb.alloc_mxfp4(shape), mb.alloc_mxfp4((c, k, r))
        mb.mxfp4_readout(theta, ema, q, qt, w_final=w)
        blend = torch.empty(shape, device="cuda")
        mb.readout_blend(theta, ema, blend, w_final=w)
        q2, qt2 = mb.alloc_mxfp4(shape), mb.alloc_mxfp4((c, k, r))
        mb.mxfp4_quantize(blend, q2, qt2)
        for a, b in ((q, q2), (qt, qt2)):
            assert torch.equal(a.data, b.data) and torch.equal(a.scales, b.scales)
        wf = float(np.float32(w))
        want = wf * _f64(theta) + (1 - wf) * _f64(ema)
        assert np.all(np.abs(_f64(blend) - want) <= 2.0 ** -22 * (np.abs(wf * _f64(theta)) + np.abs(_f64(ema))))


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dequantize(mb, shape, dtype):
    """Any codes and any scales, 0 and 255 among them, read back exactly."""
    c, r, k = shape
    g = np.random.default_rng(5)
    b = (k + 31) // 32
    codes = g.integers(0, 16, (c, r, b * 32), dtype=np.uint8)
    codes[:, :, k:] = 0
    scales = g.integers(0, 251, (c, r, b), dtype=np.uint8)
    scales[0, 0, 0] = 255
    scales[-1, -1, -1] = 0
    q = _stored(mb, codes, scales, shape)
    out = torch.empty(shape, dtype=DTYPES[dtype], device="cuda")
    mb.mxfp4_dequantize(q, out)
    want = np.stack([ref.values(codes[m], scales[m], k) for m in range(c)])
    assert np.array_equal(_f64(out), want, equal_nan=True)


# --------------------------------------------------------------------- product
def _stored(mb, codes, scales, shape):
    parts = [ref.pack(codes[m], scales[m]) for m in range(shape[0])]
    return mb.Mxfp4(_dev(np.stack([p[0] for p in parts])), _dev(np.stack([p[1] for p in parts])), shape)


def _operand(mb, count, rows, k, seed, lo=126, hi=129):
    g = np.random.default_rng(seed)
    b = (k + 31) // 32
    codes = g.integers(0, 16, (count, rows, b * 32), dtype=np.uint8)
    codes[:, :, k:] = 0
    scales = g.integers(lo, hi, (count, rows, b), dtype=np.uint8)
    v = np.stack([ref.values(codes[m], scales[m], k) for m in range(count)])
    return _stored(mb, codes, scales, (count, rows, k)), v


FEW = [(1, 1, 1, 1), (1, 1, 128, 32), (1, 1, 1000, 96), (1, 3, 129, 257), (2, 16, 300, 768), (1, 17, 64, 512),
       (1, 33, 500, 1000), (3, 64, 200, 800), (1, 128, 400, 1100), (1, 300, 5, 640), (1, 100, 100, 1800),
       (1, 7, 2000, 1024), (1, 2, 60, 1664)]
PAIR = [(1, 129, 129, 64), (1, 256, 256, 256), (1, 300, 200, 520), (2, 257, 511, 300), (1, 1000, 771, 1001),
        (1, 512, 512, 1800), (4, 130, 260, 96), (1, 2600, 2600, 160), (1, 5000, 2048, 320),
        # many tiles per CTA pair with one K stage each: the epilogue is behind the MMAs all the time
        (1, 6000, 6016, 64), (1, 5000, 5001, 32)]


def _want(a, b):
    """a b^T in float64, with a check that fp32 holds every partial sum exactly."""
    assert np.max(np.einsum("cmk,cnk->cmn", np.abs(a), np.abs(b))) * 16 < 2 ** 24
    return np.einsum("cmk,cnk->cmn", a, b)


@pytest.mark.parametrize("shape", FEW + PAIR, ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_matmul_is_exact(mb, shape, dtype):
    c, m, n, k = shape
    qa, a = _operand(mb, c, m, k, 1)
    qb, b = _operand(mb, c, n, k, 2)
    ws = mb.alloc_matmul_workspace(qa.shape, qb.shape)
    out = torch.full((c, m, n), float("nan"), dtype=DTYPES[dtype], device="cuda")
    mb.mxfp4_matmul(qa, qb, out, ws)
    assert mb.device_status(ws) == 0
    want = torch.from_numpy(_want(a, b)).to(DTYPES[dtype])
    assert torch.equal(out.cpu(), want)
    add = torch.randint(-8, 8, (c, m, n), generator=torch.Generator().manual_seed(3)).to(DTYPES[dtype])
    both = torch.from_numpy(_want(a, b) + _f64(add)).to(DTYPES[dtype])
    mb.mxfp4_matmul(qa, qb, out, ws, add=add.cuda())
    assert torch.equal(out.cpu(), both)
    inplace = add.cuda()
    mb.mxfp4_matmul(qa, qb, inplace, ws, add=inplace)
    assert torch.equal(inplace.cpu(), both) and mb.device_status(ws) == 0


@pytest.mark.parametrize("shape", [(1, 4096, 4096, 1792), (1, 8192, 2560, 1024), (16, 1024, 768, 768), (1, 16, 8192, 1792)], ids=str)
def test_repeated_products_are_bitwise_right(mb, shape):
    """The same large product many times, with scales that differ from row to row
    and block to block: no call may read a scale or a code too early or too late."""
    c, m, n, k = shape
    g = torch.Generator(device="cuda").manual_seed(7)

    def operand(rows):
        data = torch.randint(0, 256, (c, rows, k // 2), generator=g, device="cuda", dtype=torch.int64).to(torch.uint8)
        tiles = (c, -(-rows // 128), -(-k // 128), 512)
        scales = torch.randint(126, 129, tiles, generator=g, device="cuda", dtype=torch.int64).to(torch.uint8)
        return mb.Mxfp4(data, scales, (c, rows, k))
    qa, qb = operand(m), operand(n)
    a, b = torch.empty(c, m, k, device="cuda"), torch.empty(c, n, k, device="cuda")
    mb.mxfp4_dequantize(qa, a)
    mb.mxfp4_dequantize(qb, b)
    # sums of 2^-4 units below 2^24 of them are exact in fp32
    assert float((a.abs().double() @ b.abs().double().transpose(1, 2)).max()) * 16 < 2 ** 24
    want = (a.double() @ b.double().transpose(1, 2)).float()
    ws = mb.alloc_matmul_workspace(qa.shape, qb.shape)
    for dt in (torch.float32, torch.bfloat16):
        w = want.to(dt)
        out = torch.empty(c, m, n, dtype=dt, device="cuda")
        for i in range(60):
            out.fill_(float("nan"))
            mb.mxfp4_matmul(qa, qb, out, ws)
            assert torch.equal(out, w), i
    assert mb.device_status(ws) == 0


@pytest.mark.parametrize("shape", [(1, 4096, 4096, 1792), (5, 1000, 776, 300), (3, 600, 516, 64), (2, 300, 1001, 700)], ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_repeated_products_with_an_addend(mb, shape, dtype):
    """Addends of their own and in place, many times over; ones and minus ones,
    so that every sum is exact in fp32."""
    c, m, n, k = shape
    g = torch.Generator(device="cuda").manual_seed(11)
    a, b = (torch.randint(0, 2, (c, r, k), generator=g, device="cuda").mul_(2).sub_(1).float() for r in (m, n))
    qa, qb = mb.alloc_mxfp4((c, m, k)), mb.alloc_mxfp4((c, n, k))
    mb.mxfp4_quantize(a, qa)
    mb.mxfp4_quantize(b, qb)
    add = torch.randint(-100, 101, (c, m, n), generator=g, device="cuda").to(dtype)
    want = ((a.double() @ b.double().transpose(1, 2)) + add.double()).float().to(dtype)
    ws = mb.alloc_matmul_workspace(qa.shape, qb.shape)
    out = torch.empty_like(add)
    for i in range(30):
        if i % 2:
            out.copy_(add)
            mb.mxfp4_matmul(qa, qb, out, ws, add=out)
        else:
            out.fill_(float("nan"))
            mb.mxfp4_matmul(qa, qb, out, ws, add=add)
        assert torch.equal(out, want), i
    assert mb.device_status(ws) == 0


LONG = [(1, 200, 200, 16384), (1, 64, 768, 20000), (2, 150, 300, 9000), (1, 768, 768, 32768), (1, 1, 300, 40000)]


@pytest.mark.parametrize("shape", LONG, ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_matmul_long_k(mb, shape, dtype):
    """Long sums, split over CTAs or not, with scales of many sizes."""
    c, m, n, k = shape
    qa, a = _operand(mb, c, m, k, 3, 120, 135)
    qb, b = _operand(mb, c, n, k, 4, 100, 120)
    ws = mb.alloc_matmul_workspace(qa.shape, qb.shape)
    out = torch.empty((c, m, n), dtype=DTYPES[dtype], device="cuda")
    mb.mxfp4_matmul(qa, qb, out, ws)
    assert mb.device_status(ws) == 0
    ta, tb = _dev(a), _dev(b)
    want = torch.einsum("cmk,cnk->cmn", ta, tb)
    mag = torch.einsum("cmk,cnk->cmn", ta.abs(), tb.abs())
    tol = -(-k // 64) * 2.0 ** -22 * mag + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * want.abs() * 1.001
    assert bool(((out.double() - want).abs() <= tol).all())
    again = torch.empty_like(out)
    mb.mxfp4_matmul(qa, qb, again, ws)
    assert torch.equal(out, again)                           # the order of the sums is fixed


@pytest.mark.parametrize("shape", [(3, 5, 200, 96), (3, 300, 260, 96)], ids=str)
def test_matmul_shared_operand(mb, shape):
    c, m, n, k = shape
    qa, a = _operand(mb, 1, m, k, 5)
    qb, b = _operand(mb, c, n, k, 6)
    for l, r, want in ((qa, qb, _want(np.repeat(a, c, 0), b)), (qb, qa, _want(b, np.repeat(a, c, 0)))):
        ws = mb.alloc_matmul_workspace(l.shape, r.shape)
        out = torch.empty((c, l.shape[1], r.shape[1]), device="cuda")
        mb.mxfp4_matmul(l, r, out, ws)
        assert np.array_equal(_f64(out), want)


@pytest.mark.parametrize("m", [4, 200])
def test_matmul_nan_blocks_stay_in_their_rows(mb, m):
    """A block that stands for NaN makes its row's results NaN, and no others."""
    qa, a = _operand(mb, 1, m, 200, 7)
    qb, b = _operand(mb, 1, 300, 200, 8)
    x = _dev(a)[0].float()
    x[2, 70] = float("inf")
    mb.mxfp4_quantize(x, qa)
    back = torch.empty(1, m, 200, device="cuda")
    mb.mxfp4_dequantize(qa, back)
    ws = mb.alloc_matmul_workspace(qa.shape, qb.shape)
    out = torch.empty(1, m, 300, device="cuda")
    mb.mxfp4_matmul(qa, qb, out, ws)
    assert bool(torch.isnan(out[0, 2]).all())
    keep = [i for i in range(m) if i != 2]
    want = torch.einsum("mk,nk->mn", back[0].double(), _dev(b)[0])
    assert torch.equal(out[0, keep].double(), want[keep])


def test_bytes_behind_the_results_stay(mb):
    """Outputs end where they end: the bytes behind them keep their values."""
    guard = 4096
    for c, m, n, k in ((1, 3, 129, 100), (1, 257, 131, 100), (2, 150, 300, 9000)):
        qa, _ = _operand(mb, c, m, k, 9)
        qb, _ = _operand(mb, c, n, k, 10)
        for dt in DTYPES.values():
            flat = torch.full((c * m * n + guard,), 7.0, dtype=dt, device="cuda")
            size = mb.matmul_workspace_size(qa.shape, qb.shape)
            ws = torch.zeros(size + guard, dtype=torch.uint8, device="cuda")
            mb.mxfp4_matmul(qa, qb, flat[:c * m * n].view(c, m, n), ws[:size])
            assert bool((flat[c * m * n:] == 7.0).all()) and int(ws[size:].sum()) == 0
            dq = torch.full((c * m * k + guard,), 7.0, dtype=dt, device="cuda")
            mb.mxfp4_dequantize(qa, dq[:c * m * k].view(c, m, k))
            assert bool((dq[c * m * k:] == 7.0).all())
        x = torch.randn(c, m, k, device="cuda")
        for shape, kw in (((c, m, k), "out"), ((c, k, m), "out_t")):
            q = mb.alloc_mxfp4(shape)
            data = torch.full((q.data.numel() + guard,), 9, dtype=torch.uint8, device="cuda")
            scales = torch.full((q.scales.numel() + guard,), 9, dtype=torch.uint8, device="cuda")
            held = mb.Mxfp4(data[:q.data.numel()], scales[:q.scales.numel()], shape)
            mb.mxfp4_quantize(x, **{kw: held})
            assert bool((data[q.data.numel():] == 9).all()) and bool((scales[q.scales.numel():] == 9).all())


def test_other_stream_and_graph(mb):
    """A captured quantise + product on a side stream; the replay draws new
    numbers once the offset in device memory has moved."""
    x = _source(300, 512, "bf16", 31).cuda()
    qb, b = _operand(mb, 1, 400, 512, 32)
    rng, key = _rng(3, 100)
    q = mb.alloc_mxfp4((300, 512))
    ws = mb.alloc_matmul_workspace(q.shape, qb.shape)
    out = torch.empty(1, 300, 400, device="cuda")

    def step():
        mb.mxfp4_quantize(x, q, dropout=0.1, stochastic=True, rng=rng)
        mb.mxfp4_matmul(q, qb, out, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    eager = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
        rng[1] += 1
    out.zero_()
    graph.replay()
    assert torch.equal(out, eager)
    graph.replay()
    second = out.clone()
    assert not torch.equal(second, eager) and rng[1].item() == key[1] + 2
    rng[1] -= 1
    step()
    assert torch.equal(out, second)


def test_bounded_wait_limit_is_not_reached(mb):
    """The status word of a workspace stays clear over many calls of mixed sizes."""
    ws = torch.zeros(max(mb.matmul_workspace_size((1, m, 4096), (1, 300, 4096)) for m in (1, 40, 300)),
                     dtype=torch.uint8, device="cuda")
    qb, _ = _operand(mb, 1, 300, 4096, 41)
    for m in (1, 40, 300) * 5:
        qa, _ = _operand(mb, 1, m, 4096, m)
        out = torch.empty(1, m, 300, device="cuda")
        mb.mxfp4_matmul(qa, qb, out, ws)
    assert mb.device_status(ws) == 0


# --------------------------------------------------- offsets past 32 bits, graphs
def _rows_numbers(key, site, domain, rows, cols):
    """16-bit numbers of some rows (indices) of a matrix."""
    out = np.empty((len(rows), cols), dtype=np.int64)
    n = (key[1] + site) % 2 ** 64
    for i, r in enumerate(rows):
        for g in range((cols + 7) // 8):
            w = ref.philox([g, int(r), n & ref.M32, (n >> 32) & 0x3FFFFFFF | domain << 30],
                           [key[0] & ref.M32, key[0] >> 32])
            for c in range(8 * g, min(cols, 8 * g + 8)):
                v = w[(c & 7) >> 1]
                out[i, c] = v >> 16 if c & 1 else v & 0xFFFF
    return out


@pytest.mark.parametrize("cols", [520, 523])
def test_elements_past_32_bits(mb, cols):
    """More than 2^31 elements (and, read back in fp32, 2^33 bytes): the last rows,
    and those around the 2^31st element, of dropout, quantisation and read-back."""
    rows = (1 << 31) // cols + 300
    base = _source(64, cols, "bf16", 51).cuda()
    x = base.repeat(-(-rows // 64), 1)[:rows].contiguous()
    assert x.numel() > 1 << 31
    rng, key = _rng(17, 23)
    probe = [0, (1 << 31) // cols - 1, (1 << 31) // cols, (1 << 31) // cols + 1, rows - 1]
    out = torch.empty_like(x)
    mb.dropout(x, out, 0.25, rng)
    keep = _rows_numbers(key, 0, 0, probe, cols) >= 16384
    want = np.where(keep, _f64(x[probe]) * (4.0 / 3.0), 0.0)
    assert np.all(np.abs(_f64(out[probe]) - want) <= np.abs(want) * 2.0 ** -8 * 1.001)
    del out
    q, qt = mb.alloc_mxfp4((rows, cols)), mb.alloc_mxfp4((cols, rows))
    mb.mxfp4_quantize(x, q, qt)
    back = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    mb.mxfp4_dequantize(q, back)
    codes, scales = ref.quantize(_f64(x[probe]))
    assert np.array_equal(_f64(back[probe]), ref.values(codes, scales, cols))
    back = back.view(cols, rows)
    mb.mxfp4_dequantize(qt, back)
    tail = _f64(x[rows - rows % 32 - 64:, [0, cols - 1]]).T       # the last blocks of the first and last column
    codes, scales = ref.quantize(tail)
    got = _f64(back[[0, cols - 1], rows - rows % 32 - 64:])
    assert np.array_equal(got, ref.values(codes, scales, tail.shape[1]))


@pytest.mark.parametrize("n", [46400, 46399])
def test_product_past_32_bits(mb, n):
    """More than 2^31 results."""
    m = 46500
    qa, a = _operand(mb, 1, 128, 64, 61)
    rep = -(-m // 128)
    big_a = mb.Mxfp4(qa.data.repeat(1, rep, 1)[:, :m].contiguous(), qa.scales.view(-1).repeat(rep), (1, m, 64))
    rep = -(-n // 128)
    big_b = mb.Mxfp4(qa.data.repeat(1, rep, 1)[:, :n].contiguous(), qa.scales.view(-1).repeat(rep), (1, n, 64))
    out = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = mb.alloc_matmul_workspace((1, m, 64), (1, n, 64))
    mb.mxfp4_matmul(big_a, big_b, out, ws)
    want = torch.from_numpy(_want(a, a))[0].bfloat16().cuda()
    cols = torch.arange(n, device="cuda") % 128
    for r in (0, (1 << 31) // n, (1 << 31) // n + 1, m - 1):
        assert torch.equal(out[r], want[r % 128, cols])
    assert not bool(torch.isnan(out).any())


def test_two_captured_graphs_replayed_at_once(mb):
    """Split and few-row products captured into two graphs with workspaces of
    their own and replayed on two streams."""
    graphs, outs, wants = [], [], []
    for i, (m, n, k) in enumerate(((300, 260, 16384), (16, 900, 8192))):
        qa, _ = _operand(mb, 1, m, k, 70 + i, 122, 130)
        qb, _ = _operand(mb, 1, n, k, 80 + i, 122, 130)
        ws = mb.alloc_matmul_workspace(qa.shape, qb.shape)
        out = torch.empty(1, m, n, device="cuda")
        mb.mxfp4_matmul(qa, qb, out, ws)
        torch.cuda.synchronize()
        wants.append(out.clone())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(4):
                mb.mxfp4_matmul(qa, qb, out, ws)
        graphs.append((g, qa, qb, ws))
        outs.append(out)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(10):
        for s, g, o in zip(streams, graphs, outs):
            with torch.cuda.stream(s):
                o.zero_()
                g[0].replay()
    torch.cuda.synchronize()
    for o, w, g in zip(outs, wants, graphs):
        assert torch.equal(o, w) and mb.device_status(g[3]) == 0


def test_a_matrix_times_itself(mb):
    """One handle as both operands, and many small matrices in one call."""
    qa, a = _operand(mb, 1, 300, 200, 91)
    ws = mb.alloc_matmul_workspace(qa.shape, qa.shape)
    out = torch.empty(300, 300, device="cuda")
    mb.mxfp4_matmul(qa, qa, out, ws)
    assert np.array_equal(_f64(out), _want(a, a)[0])
    qb, b = _operand(mb, 700, 3, 40, 92)
    qc, c = _operand(mb, 700, 5, 40, 93)
    ws = mb.alloc_matmul_workspace(qb.shape, qc.shape)
    out = torch.empty(700, 3, 5, dtype=torch.bfloat16, device="cuda")
    mb.mxfp4_matmul(qb, qc, out, ws)
    assert torch.equal(out.cpu(), torch.from_numpy(_want(b, c)).bfloat16())
