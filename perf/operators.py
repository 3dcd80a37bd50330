"""Plain forms and workloads of the 4-bit and dropout operators.

Three operators that stand around the optimizer step: dropout from a
counter-based generator, microscaled 4-bit quantisation (MXFP4: e2m1 elements,
one power-of-two scale per 32 of them) with its read-back, and the product of
two such matrices. `run` computes each either in its plain form (elementary
torch operations) or through the package's entry points (`own`).

Definitions
-----------
Random numbers. rng = (seed, offset), two int64 in device memory. With
n = (offset + site) mod 2^64, element (r, c) of the matrix numbered m takes
half (c & 1) of word (c >> 1) & 3 of Philox4x32-10 under key (lo(seed),
hi(seed)) and counter (c >> 3, m * rows + r, lo(n), hi(n) & 0x3fffffff | d << 30),
where d is 0 for dropout, 1 for the rounding of rows, 2 for the rounding of
columns (r and c are then those of the transposed matrix).

Dropout. t = round(p 2^16); out = x * (2^16 / (2^16 - t)) where u16 >= t, else 0.

Quantisation. Blocks of 32 along the last axis; amax = m 2^e with 1 <= m < 2;
scale = 2^(e - 2 + (m > 1.5)), at least 2^-127: the smallest power of two with
amax / scale <= 6. Elements round to {0, .5, 1, 1.5, 2, 3, 4, 6}, to nearest
with ties to the even code, or stochastically: with y between two neighbours
at fraction f, up iff u16 + 1/2 < f 2^16. A block with an infinity or a NaN
has the scale 0xff and stands for NaN.

Storage. Two elements a byte, the first in the low half; rows padded to 32
elements. Scales (exponent + 127) lie in tiles of 128 rows x 4 blocks of 512
bytes, tile (i, j) at (i * ceil(blocks / 4) + j) * 512; in it row r, block b at
(r % 32) * 16 + (r // 32) * 4 + b; the padding is zero.
"""
import torch

own = False

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"


# ------------------------------------------------------------------ workloads
def listed():
    return [
        # re-quantising a bank of weights for the forward and backward products after a step
        dict(name="quantize_weights", op="quantize", count=48, rows=768, cols=768, dtype="bf16",
             both=True, p=0.0, stochastic=False),
        # the activations of a training batch, with the dropout in front of the linear layer
        dict(name="quantize_activations_dropout", op="quantize", count=1, rows=16384, cols=2560, dtype="bf16",
             both=True, p=0.1, stochastic=False),
        # an output gradient of ragged size, rounded stochastically
        dict(name="quantize_gradient_ragged", op="quantize", count=1, rows=4099, cols=1023, dtype="f32",
             both=True, p=0.0, stochastic=True),
        # the averaged readout matrix, laid out for serving: [768, 50304] -> blocks along the 768
        dict(name="readout_blend", op="readout", count=1, rows=768, cols=50304, dtype="bf16", w_final=0.35),
        # residual dropout over a large batch
        dict(name="dropout_residual", op="dropout", rows=32768, cols=2560, dtype="bf16", p=0.1, residual=True),
        # a few odd rows in fp32, where the launch is what counts
        dict(name="dropout_small", op="dropout", rows=257, cols=1001, dtype="f32", p=0.1, residual=False),
        # one token against the readout
        dict(name="matmul_one_token", op="matmul", count=1, m=1, n=50304, k=768, dtype="bf16", add=False),
        # a few tokens against a square layer
        dict(name="matmul_few_tokens", op="matmul", count=1, m=16, n=2560, k=2560, dtype="bf16", add=False),
        # a training batch through the widening layer of the larger bank
        dict(name="matmul_forward", op="matmul", count=1, m=16384, n=10240, k=2560, dtype="bf16", add=False),
        # a weight gradient over the tokens of a batch, added to the gradient that is there
        dict(name="matmul_weight_gradient", op="matmul", count=1, m=768, n=768, k=32768, dtype="f32", add=True),
        # several matrices of ragged sizes at once
        dict(name="matmul_ragged_bank", op="matmul", count=4, m=1000, n=1537, k=771, dtype="bf16", add=False),
    ]


def _log_int(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]; half of them odd or ragged."""
    import math
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v >= 256:
        v -= v % 128
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["quantize", "quantize", "readout", "dropout", "matmul", "matmul", "matmul"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "dropout":
        rows = _log_int(rng, 1, 32768)
        cols = _log_int(rng, 64, min(10240, 16384 * 2560 // rows))
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, p=round(rng.uniform(0.02, 0.6), 3),
                    residual=rng.random() < 0.5)
    if op == "readout":
        rows = _log_int(rng, 64, 2560)
        return dict(op=op, count=rng.choice([1, 1, 3]), rows=rows, cols=_log_int(rng, 64, 12000), dtype=dtype,
                    w_final=round(rng.uniform(0.0, 1.0), 3))
    if op == "quantize":
        count = rng.choice([1, 1, 4, 13])
        cols = _log_int(rng, 33, 10240)
        rows = _log_int(rng, 1, min(16384, 16384 * 2560 // (count * cols)))
        stochastic = rng.random() < 0.4
        return dict(op=op, count=count, rows=rows, cols=cols, dtype=dtype, both=rng.random() < 0.7,
                    p=rng.choice([0.0, 0.0, 0.1, 0.35]), stochastic=stochastic)
    count = rng.choice([1, 1, 1, 3])
    kind = rng.choice(["serve", "train", "gradient"])
    if kind == "serve":
        m, n, k = rng.randint(1, 64), _log_int(rng, 256, 50304), _log_int(rng, 128, 2560)
    elif kind == "train":
        m, n, k = _log_int(rng, 65, 8192), _log_int(rng, 64, 4096), _log_int(rng, 64, 2560)
    else:
        m, n, k = _log_int(rng, 64, 2560), _log_int(rng, 64, 2560), _log_int(rng, 4096, 16384)
    return dict(op=op, count=count, m=m, n=n, k=k, dtype=dtype, add=rng.random() < 0.4)


def _up(x, m):
    return -(-x // m) * m


def _packed_bytes(count, rows, cols):
    """Bytes of codes and scales that a matrix in 4 bits is made of."""
    blocks = -(-cols // 32)
    return count * rows * blocks * 17


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "dropout":
        n = case["rows"] * case["cols"]
        return {"bytes": n * e * (3 if case["residual"] else 2) + 16, "flops": n * (2 if case["residual"] else 1)}
    if case["op"] == "matmul":
        c, m, n, k = case["count"], case["m"], case["n"], case["k"]
        out = c * m * n * e
        return {"bytes": _packed_bytes(c, m, k) + _packed_bytes(c, n, k) + out * (2 if case["add"] else 1),
                "flops": 2 * c * m * n * k}
    c, r, k = case["count"], case["rows"], case["cols"]
    n = c * r * k
    if case["op"] == "readout":  # theta and the fp32 average in; codes, and the values read back, out
        return {"bytes": n * (e + 4) + _packed_bytes(c, k, r) + n * 2, "flops": 6 * n}
    sides = 2 if case["both"] else 1
    bytes_ = n * e + _packed_bytes(c, r, k) + sides * n * 2
    if case["both"]:
        bytes_ += _packed_bytes(c, k, r)
    return {"bytes": bytes_, "flops": 4 * n * sides}


# --------------------------------------------------------------------- inputs
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32)


def _activations(gen, count, rows, cols):
    """Values with features of different sizes and a few large ones, as the layers of a network have them."""
    x = _normal(gen, count, rows, cols)
    x *= torch.exp(0.7 * _normal(gen, count, 1, cols))
    x *= torch.exp(0.3 * _normal(gen, count, rows, 1))
    return x


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    st = dict(case=dict(case))
    dt = DTYPES[case["dtype"]]
    st["rng"] = torch.randint(0, 2 ** 62, (2,), generator=gen, device=DEV, dtype=torch.int64)
    if case["op"] == "dropout":
        st["x"] = _activations(gen, 1, case["rows"], case["cols"])[0].to(dt)
        if case["residual"]:
            st["residual"] = _activations(gen, 1, case["rows"], case["cols"])[0].to(dt)
    elif case["op"] == "quantize":
        st["x"] = (0.02 * _activations(gen, case["count"], case["rows"], case["cols"])).to(dt)
    elif case["op"] == "readout":
        shape = (case["count"], case["rows"], case["cols"])
        theta = 0.02 * _normal(gen, *shape)
        st["theta"] = theta.to(dt)
        st["ema"] = theta + 0.002 * _normal(gen, *shape)
    else:
        c, m, n, k = case["count"], case["m"], case["n"], case["k"]
        st["a"] = _plain_pack(*_plain_codes(_activations(gen, c, m, k)))
        st["b"] = _plain_pack(*_plain_codes(0.02 * _normal(gen, c, n, k)))
        if case["add"]:
            st["add"] = _normal(gen, c, m, n).to(dt)
    if own:
        _prepare_own(st, dt)
    return st


def _prepare_own(st, dt):
    """The buffers and handles that a program of the package's keeps."""
    import muon_newton_schulz_05_b200 as mb
    case = st["case"]
    if case["op"] == "dropout":
        st["out"] = torch.empty_like(st["x"])
    elif case["op"] == "matmul":
        c, m, n, k = case["count"], case["m"], case["n"], case["k"]
        st["qa"] = mb.Mxfp4(*st["a"], shape=(c, m, k))
        st["qb"] = mb.Mxfp4(*st["b"], shape=(c, n, k))
        st["out"] = torch.empty(c, m, n, dtype=dt, device=DEV)
        st["workspace"] = mb.alloc_matmul_workspace((c, m, k), (c, n, k))
    else:
        c, r, k = case["count"], case["rows"], case["cols"]
        if case["op"] == "quantize":
            st["q"] = mb.alloc_mxfp4((c, r, k))
            st["values"] = torch.empty(c, r, k, dtype=torch.bfloat16, device=DEV)
        if case["op"] == "readout" or case["both"]:
            st["qt"] = mb.alloc_mxfp4((c, k, r))
            st["values_t"] = torch.empty(c, k, r, dtype=torch.bfloat16, device=DEV)


# ------------------------------------------------------------------ plain form
def _philox(seed, offset, site, domain, row0, rows, groups):
    """The four words of each counter (group, row) as int64 [rows, groups, 4]."""
    lo = 0xFFFFFFFF

    def mulhilo(a, b):  # 32 x 32 -> (high, low); a is a number below 2^32
        high = ((a >> 16) * b + (((a & 0xFFFF) * b) >> 16)) >> 16
        return high, (a * b) & lo

    n = offset + site
    c0 = torch.arange(groups, device=DEV).expand(rows, groups)
    c1 = torch.arange(row0, row0 + rows, device=DEV).unsqueeze(1).expand(rows, groups)
    c2 = (n & lo).expand(rows, groups)
    c3 = (((n >> 32) & 0x3FFFFFFF) | (domain << 30)).expand(rows, groups)
    k0, k1 = seed & lo, (seed >> 32) & lo
    for _ in range(10):
        h0, l0 = mulhilo(0xD2511F53, c0)
        h1, l1 = mulhilo(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & lo, (k1 + 0xBB67AE85) & lo
    return torch.stack([c0, c1, c2, c3], dim=-1)


def _uniform16(rng, domain, rows, cols, row0=0):
    """The 16-bit random numbers of a [rows, cols] matrix, as float32."""
    groups = -(-cols // 8)
    words = _philox(rng[0], rng[1], 0, domain, row0, rows, groups)
    halves = torch.stack([words & 0xFFFF, words >> 16], dim=-1)
    return halves.reshape(rows, groups * 8)[:, :cols].float()


def _in_rows(rows, cols, f):
    """f(first row, rows) over slabs of rows, joined (bounds the temporaries of the integer arithmetic)."""
    step = max(1, (1 << 25) // cols)
    return torch.cat([f(r, min(step, rows - r)) for r in range(0, rows, step)])


def _plain_dropout(x, p, rng):
    """[rows, cols] -> float32, zero where dropped."""
    t = round(p * 65536)
    scale = torch.tensor(65536.0 / (65536 - t), dtype=torch.float32, device=DEV)

    def slab(r, n):
        return torch.where(_uniform16(rng, 0, n, x.shape[1], r) >= t, x[r:r + n].float() * scale, 0.0)
    return _in_rows(x.shape[0], x.shape[1], slab)


def _plain_codes(x, rng=None, domain=1):
    """Codes (0..7, plus 8 for the sign) [count, rows, padded cols] and scale bytes [count, rows, blocks] of a
    float32 tensor; rng for stochastic rounding."""
    c, r, k = x.shape
    x = torch.nn.functional.pad(x, (0, _up(k, 32) - k)).reshape(c, r, -1, 32)
    amax = x.abs().amax(-1)
    bad = ~torch.isfinite(amax)
    mant, ex = torch.frexp(torch.where(bad, 1.0, amax))      # amax = mant 2^ex, mant in [.5, 1)
    ex = ex.int() - 3 + (mant > 0.75).int()
    ex = torch.where(amax == 0, -127, ex.clamp(min=-127))
    y = torch.ldexp(x.abs(), -ex.unsqueeze(-1))
    y = torch.where(bad.unsqueeze(-1), 0.0, y)
    if rng is None:
        code = ((y > 0.25).int() + (y >= 0.75).int() + (y > 1.25).int() + (y >= 1.75).int() + (y > 2.5).int() +
                (y >= 3.5).int() + (y > 5.0).int())
    else:
        u = _in_rows(c * r, _up(k, 32), lambda r0, n: _uniform16(rng, domain, n, _up(k, 32), r0)).reshape(y.shape)
        steps = torch.where(y < 2, 2 * y, torch.where(y < 4, y, 0.5 * y))
        base = torch.where(y < 2, 0, torch.where(y < 4, 2, 4))
        low = torch.floor(steps)
        code = (low + base + (u + 0.5 < (steps - low) * 65536)).int()
    code = code + 8 * (torch.signbit(x) & ~bad.unsqueeze(-1)).int()
    scales = torch.where(bad, 255, ex + 127)
    return code.reshape(c, r, -1).to(torch.uint8), scales.to(torch.uint8)


def _plain_pack(codes, scales):
    """(data, scales) as they are stored."""
    c, r, b = scales.shape
    data = codes[..., 0::2] | (codes[..., 1::2] << 4)
    tiles = torch.nn.functional.pad(scales, (0, _up(b, 4) - b, 0, _up(r, 128) - r))
    tiles = tiles.reshape(c, -1, 4, 32, tiles.shape[2] // 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(c, -1)
    return data.contiguous(), tiles.contiguous()


def _plain_unpack(stored, rows, cols):
    """The float32 values of a stored matrix."""
    data, tiles = stored
    c = data.shape[0]
    blocks = -(-cols // 32)
    s = tiles.reshape(c, -1, _up(blocks, 4) // 4, 32, 4, 4).permute(0, 1, 4, 3, 2, 5)
    s = s.reshape(c, _up(rows, 128), -1)[:, :rows, :blocks]
    codes = torch.stack([data & 15, data >> 4], dim=-1).reshape(c, rows, blocks, 32)
    return _plain_values(codes, s)[..., :cols]


def _plain_values(codes, scales):
    """float32 values [count, rows, padded cols] of codes and scale bytes."""
    c, r, b = scales.shape
    levels = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=DEV)
    v = levels[codes.reshape(c, r, b, 32).int()]
    v = torch.ldexp(v, scales.int().unsqueeze(-1) - 127)
    return torch.where(scales.unsqueeze(-1) == 255, float("nan"), v).reshape(c, r, -1)


def _plain_quantized(x, cols, rng=None, domain=1):
    """The values that the quantised x stands for, in bf16 (which holds them exactly)."""
    codes, scales = _plain_codes(x, rng, domain)
    return _plain_values(codes, scales)[..., :cols].to(torch.bfloat16)


def _run_plain(st):
    case = st["case"]
    if case["op"] == "dropout":
        y = _plain_dropout(st["x"], case["p"], st["rng"])
        return (y if not case["residual"] else y + st["residual"].float()).to(st["x"].dtype)
    if case["op"] == "quantize":
        x = st["x"].float()
        if case["p"] > 0:
            x = _plain_dropout(x.reshape(-1, case["cols"]), case["p"], st["rng"]).reshape(x.shape)
        rng = st["rng"] if case["stochastic"] else None
        out = [_plain_quantized(x, case["cols"], rng, 1)]
        if case["both"]:
            out.append(_plain_quantized(x.transpose(1, 2), case["rows"], rng, 2))
        return out
    if case["op"] == "readout":
        # in 64 bits: a value next to the border of two codes must not move
        w = torch.tensor(case["w_final"], dtype=torch.float32, device=DEV)
        kept = ((1 - w) * st["ema"]).double()
        x = (w.double() * st["theta"].double() + kept).float()
        return [_plain_quantized(x.transpose(1, 2), case["rows"])]
    a = _plain_unpack(st["a"], case["m"], case["k"])
    b = _plain_unpack(st["b"], case["n"], case["k"])
    y = torch.matmul(a, b.transpose(1, 2))
    if case["add"]:
        y = y + st["add"].float()
    return y.to(DTYPES[case["dtype"]])


# ------------------------------------------------------------ the package's calls
def _run_own(st):
    import muon_newton_schulz_05_b200 as mb
    case = st["case"]
    if case["op"] == "dropout":
        mb.dropout(st["x"], st["out"], case["p"], st["rng"], residual=st.get("residual"))
        return st["out"]
    if case["op"] == "matmul":
        mb.mxfp4_matmul(st["qa"], st["qb"], st["out"], st["workspace"], add=st.get("add"))
        return st["out"]
    if case["op"] == "readout":
        mb.mxfp4_readout(st["theta"], st["ema"], out_t=st["qt"], w_final=case["w_final"])
        mb.mxfp4_dequantize(st["qt"], st["values_t"])
        return [st["values_t"]]
    mb.mxfp4_quantize(st["x"], out=st["q"], out_t=st.get("qt"), dropout=case["p"],
                      stochastic=case["stochastic"], rng=st["rng"])
    mb.mxfp4_dequantize(st["q"], st["values"])
    if not case["both"]:
        return [st["values"]]
    mb.mxfp4_dequantize(st["qt"], st["values_t"])
    return [st["values"], st["values_t"]]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------- exact
def _exact_random(rng, domain, rows, cols):
    """16-bit numbers [rows, cols] from the generator's definition, on the host in unsigned 64-bit integers."""
    import numpy as np
    seed, offset = (int(v) % 2 ** 64 for v in rng.tolist())
    u, mask = np.uint64, np.uint64(0xFFFFFFFF)
    groups = (cols + 7) // 8
    out = np.empty((rows, groups, 8), dtype=np.uint16)
    for r in range(0, rows, max(1, (1 << 20) // groups)):
        stop = min(rows, r + max(1, (1 << 20) // groups))
        ctr = [np.broadcast_to(np.arange(groups, dtype=u), (stop - r, groups)),
               np.broadcast_to(np.arange(r, stop, dtype=u)[:, None], (stop - r, groups)),
               u(offset & 0xFFFFFFFF), u((offset >> 32) & 0x3FFFFFFF | domain << 30)]
        key = [seed & 0xFFFFFFFF, seed >> 32]
        for _ in range(10):
            p, q = u(0xD2511F53) * ctr[0], u(0xCD9E8D57) * ctr[2]
            ctr = [(q >> u(32)) ^ ctr[1] ^ u(key[0]), q & mask, (p >> u(32)) ^ ctr[3] ^ u(key[1]), p & mask]
            key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
        for i, w in enumerate(ctr):
            out[r:stop, :, 2 * i] = w & u(0xFFFF)
            out[r:stop, :, 2 * i + 1] = w >> u(16)
    return torch.from_numpy(out.reshape(rows, groups * 8)[:, :cols].astype(np.float64)).to(DEV)


def _exact_quantized(x, u=None):
    """Values of the quantised x ([count, rows, cols], float64), found level by level; u: random numbers."""
    c, r, k = x.shape
    pad = (-k) % 32
    x = torch.cat([x, x.new_zeros(c, r, pad)], -1).view(c, r, -1, 32)
    top = x.abs().max(-1, keepdim=True).values
    # the smallest power of two s with top <= 6 s, by stepping from a first guess
    e = torch.floor(torch.log2(top.clamp(min=2.0 ** -149) / 6)) - 1
    for _ in range(3):
        e = e + (top > 6 * torch.exp2(e)).double()
    s = torch.exp2(e.clamp(min=-127))
    y = x.abs() / s
    lv = [float(v) for v in LEVELS]
    out = torch.zeros_like(y)
    if u is not None:
        u = torch.cat([u.view(c, r, k), u.new_zeros(c, r, pad)], -1).view_as(y)
    for i in range(7):
        lo, hi = lv[i], lv[i + 1]
        frac = (y - lo) / (hi - lo)
        up = (frac > 0.5) | ((frac == 0.5) & (i % 2 == 1)) if u is None else u + 0.5 < frac * 65536
        out = torch.where((y >= lo) & (y < hi), torch.where(up, hi, lo), out)
    out = torch.where(y >= 6, 6.0, out) * s * torch.sign(x)
    return torch.where(torch.isfinite(top), out, float("nan")).view(c, r, -1)[..., :k]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "matmul":
        a = _exact_unpack(st["a"], case["m"], case["k"])
        b = _exact_unpack(st["b"], case["n"], case["k"])
        y = torch.einsum("cmk,cnk->cmn", a, b)
        return y + st["add"].double() if case["add"] else y
    if case["op"] == "readout":
        w = float(torch.tensor(case["w_final"], dtype=torch.float32))
        # the blend is defined in float32 with one rounding of (1 - w) ema and one of the sum
        kept = (st["ema"] * torch.tensor(1.0 - w, dtype=torch.float32, device=DEV)).double()
        x = (st["theta"].double() * w + kept).float().double()
        return [_exact_quantized(x.transpose(1, 2))]
    if case["op"] == "dropout":
        t = round(case["p"] * 65536)
        keep = _exact_random(st["rng"], 0, case["rows"], case["cols"]) >= t
        y = torch.where(keep, st["x"].double() * (65536.0 / (65536 - t)), 0.0)
        return y + st["residual"].double() if case["residual"] else y
    c, r, k = case["count"], case["rows"], case["cols"]
    x = st["x"].double()
    if case["p"] > 0:
        t = round(case["p"] * 65536)
        keep = _exact_random(st["rng"], 0, c * r, k).view(c, r, k) >= t
        # the scaled value is defined in float32, so that the code it gets does not depend on where it is formed
        scaled = (st["x"].float() * torch.tensor(65536.0 / (65536 - t), device=DEV)).double()
        x = torch.where(keep, scaled, 0.0)
    rows = _exact_random(st["rng"], 1, c * r, k) if case["stochastic"] else None
    out = [_exact_quantized(x, rows)]
    if case["both"]:
        cols = _exact_random(st["rng"], 2, c * k, r) if case["stochastic"] else None
        out.append(_exact_quantized(x.transpose(1, 2), cols))
    return out


def _exact_unpack(stored, rows, cols):
    """float64 values, looked up by the address of each code and scale."""
    data, tiles = stored
    c = data.shape[0]
    j = torch.arange(cols, device=DEV)
    i = torch.arange(rows, device=DEV).unsqueeze(1)
    code = (data[:, :, j // 2] >> (4 * (j % 2)).to(torch.uint8)) & 15
    nb = -(-(-(-cols // 32)) // 4)
    at = ((i // 128) * nb + j // 128) * 512 + (i % 32) * 16 + (i % 128 // 32) * 4 + (j // 32) % 4
    sc = tiles.view(c, -1)[:, at.reshape(-1)].view(c, rows, cols)
    mag = torch.tensor(LEVELS, dtype=torch.float64, device=DEV)[(code & 7).int()]
    val = mag * (1 - 2 * (code >> 3).double()) * torch.exp2(sc.double() - 127)
    return torch.where(sc == 255, float("nan"), val)
