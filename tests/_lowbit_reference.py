"""Plain float64 forms of dropout and of the 4-bit operators (test infrastructure;
numpy only, no code shared with the library)."""
import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
M32 = 0xFFFFFFFF


def philox(ctr, key):
    """Philox4x32-10 of one counter (four ints) and key (two ints), in Python integers."""
    c, k = list(ctr), list(key)
    for _ in range(10):
        p, q = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(q >> 32) ^ c[1] ^ k[0], q & M32, (p >> 32) ^ c[3] ^ k[1], p & M32]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    return c


def numbers16(seed, offset, site, domain, rows, cols):
    """The 16-bit numbers of a [rows, cols] matrix (seed, offset as unsigned 64-bit)."""
    n = (offset + site) % 2 ** 64
    g = (cols + 7) // 8
    c0 = np.broadcast_to(np.arange(g, dtype=np.uint64), (rows, g)).copy()
    c1 = np.broadcast_to(np.arange(rows, dtype=np.uint64)[:, None], (rows, g)).copy()
    c2 = np.full((rows, g), n & M32, dtype=np.uint64)
    c3 = np.full((rows, g), ((n >> 32) & 0x3FFFFFFF) | (domain << 30), dtype=np.uint64)
    k0, k1 = seed & M32, seed >> 32
    m, s = np.uint64(M32), np.uint64(32)
    for _ in range(10):
        p, q = np.uint64(0xD2511F53) * c0, np.uint64(0xCD9E8D57) * c2
        c0, c1, c2, c3 = (q >> s) ^ c1 ^ np.uint64(k0), q & m, (p >> s) ^ c3 ^ np.uint64(k1), p & m
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    out = np.empty((rows, g, 8), dtype=np.int64)
    for i, w in enumerate((c0, c1, c2, c3)):
        out[:, :, 2 * i] = (w & np.uint64(0xFFFF)).astype(np.int64)
        out[:, :, 2 * i + 1] = (w >> np.uint64(16)).astype(np.int64)
    return out.reshape(rows, g * 8)[:, :cols]


def dropout_terms(p):
    t = round(p * 65536)
    return t, 65536.0 / (65536 - t)


def dropped(x, p, rng, site=0):
    """dropout(x) in float64, x [rows, cols]."""
    t, scale = dropout_terms(p)
    keep = numbers16(rng[0], rng[1], site, 0, *x.shape) >= t
    return np.where(keep, x * scale, 0.0)


def dropped_f32(x, p, rng, site=0):
    """dropout(x) as the quantiser sees it: the scaled value rounded to float32."""
    t, scale = dropout_terms(p)
    keep = numbers16(rng[0], rng[1], site, 0, *x.shape) >= t
    with np.errstate(over="ignore"):
        return np.where(keep, (x.astype(np.float32) * np.float32(scale)).astype(np.float64), 0.0)


def block_scale_exponent(amax):
    """Exponent of the smallest power of two s >= 2^-127 with amax <= 6 s."""
    if amax == 0:
        return -127
    e = -127
    m, ex = np.frexp(amax)          # amax = m 2^ex, .5 <= m < 1
    e = max(e, int(ex) - 4)
    while amax > 6.0 * 2.0 ** e:
        e += 1
    return e


def quantize(x, numbers=None):
    """x [rows, cols] float64 -> (codes [rows, 32 blocks], scale bytes [rows, blocks]).
    numbers: 16-bit numbers of x's shape for stochastic rounding."""
    r, k = x.shape
    b = (k + 31) // 32
    xp = np.zeros((r, b * 32))
    xp[:, :k] = x
    codes = np.zeros((r, b * 32), dtype=np.uint8)
    scales = np.zeros((r, b), dtype=np.uint8)
    num = None
    if numbers is not None:
        num = np.zeros((r, b * 32), dtype=np.int64)
        num[:, :k] = numbers
    for i in range(r):
        for j in range(b):
            v = xp[i, 32 * j:32 * j + 32]
            if not np.all(np.isfinite(v)):
                scales[i, j] = 255
                continue
            e = block_scale_exponent(np.max(np.abs(v)))
            scales[i, j] = e + 127
            y = np.abs(v) / 2.0 ** e
            lo = np.clip(np.searchsorted(LEVELS, y, side="right") - 1, 0, 6)
            frac = (y - LEVELS[lo]) / (LEVELS[lo + 1] - LEVELS[lo])
            if num is None:
                up = (frac > 0.5) | ((frac == 0.5) & (lo % 2 == 1))
            else:
                up = num[i, 32 * j:32 * j + 32] + 0.5 < frac * 65536
            codes[i, 32 * j:32 * j + 32] = (lo + up) | (np.signbit(v).astype(np.uint8) << 3)
    return codes, scales


def values(codes, scales, cols):
    """float64 values of codes and scale bytes."""
    mag = LEVELS[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (mag * np.repeat(s, 32, axis=1))[:, :cols]


def pack(codes, scales):
    """The stored bytes of one matrix: (data [rows, blocks * 16], scales flat)."""
    r, b = scales.shape
    data = codes[:, 0::2] | (codes[:, 1::2] << 4)
    nb = (b + 3) // 4
    flat = np.zeros(((r + 127) // 128) * nb * 512, dtype=np.uint8)
    i, j = np.meshgrid(np.arange(r), np.arange(b), indexing="ij")
    at = ((i // 128) * nb + j // 4) * 512 + (i % 32) * 16 + (i % 128 // 32) * 4 + j % 4
    flat[at.reshape(-1)] = scales.reshape(-1)
    return data, flat
