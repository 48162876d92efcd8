"""The AdamW plan's stored state, bit for bit: NumPy in float32, every
operation rounded once (NumPy's +, *, / and sqrt are IEEE), in the order that
the kernels document.  Used for codes and scales; values are checked against
the float64 oracle as well."""

import numpy as np

F = np.float32
BLOCK = 256
TINY = F(2.0) ** F(-100)


def mix32(x):
    x = np.asarray(x, dtype=np.uint32)
    with np.errstate(over="ignore"):
        x = x ^ (x >> np.uint32(16))
        x = x * np.uint32(0x7FEB352D)
        x = x ^ (x >> np.uint32(15))
        x = x * np.uint32(0x846CA68B)
        return x ^ (x >> np.uint32(16))


def hashed(n, seed, step, tensor, first=0):
    """(h16 for codes, h16 for a bf16 parameter) of elements first .. first+n."""
    with np.errstate(over="ignore"):
        key = mix32(mix32(mix32(np.uint32(seed)) + np.uint32(step & 0xFFFFFFFF)) + np.uint32(tensor))
        i = np.arange(first, first + n, dtype=np.uint64)
        q = i >> np.uint64(1)
        lo, hi = (q & np.uint64(0xFFFFFFFF)).astype(np.uint32), (q >> np.uint64(32)).astype(np.uint32)
        w = mix32((lo ^ key) + hi * np.uint32(0x9E3779B9))
        wp = mix32(w ^ np.uint32(0x5BD1E995))
    sh = ((i & np.uint64(1)) * np.uint64(16)).astype(np.uint32)
    return (w >> sh) & np.uint32(0xFFFF), (wp >> sh) & np.uint32(0xFFFF)


def unit(h):
    return (h.astype(F) + F(0.5)) * F(1.0 / 65536.0)


def swap(h):
    return ((h >> np.uint32(8)) | (h << np.uint32(8))) & np.uint32(0xFFFF)


def encode(x, levels, low, u):
    """(codes as floats in low .. levels, scales) of magnitudes x (float32)."""
    x = x.astype(F)
    codes, scales = np.zeros(x.size, F), np.zeros(-(-x.size // BLOCK), F)
    for b in range(scales.size):
        s = slice(b * BLOCK, min(x.size, (b + 1) * BLOCK))
        big = x[s].max() if not np.isnan(x[s]).any() else F(np.nan)
        codes[s] = low
        if not np.isfinite(big):
            scales[b] = np.nan
        elif big >= TINY:
            scales[b] = big * F(1.0 / (levels * levels))
            inv = F(1.0) / scales[b]
            y = np.sqrt(x[s] * inv)
            codes[s] = np.clip(np.floor(y + (u if np.isscalar(u) else u[s])), F(low), F(levels))
    return codes, scales


def encode_m(m, u=F(0.5)):
    c, s = encode(np.abs(m), 127.0, 0.0, u)
    return (c * np.sign(np.where(np.isnan(m), 0, m))).astype(np.int8), s


def encode_v(v, u=F(0.5)):
    with np.errstate(invalid="ignore"):
        c, s = encode(np.sqrt(v.astype(F)), 256.0, 1.0, u)
    return (c - 1).astype(np.uint8), s


def spread(s, n):
    return np.repeat(s, BLOCK)[:n]


def decode_m(c, s):
    c = c.astype(F)
    return (c * np.abs(c)) * spread(s, c.size)


def decode_v(c, s):
    c = c.astype(F) + F(1.0)
    r = (c * c) * spread(s, c.size)
    return r * r


def moments(m, v, g, beta1, beta2, scale=None):
    g = g.astype(F)
    if scale is not None:
        g = g * F(scale)
    m = m * F(beta1) + g * F(1.0 - beta1)
    v = v * F(beta2) + (g * g) * F(1.0 - beta2)
    return m, v


def round_bf16(p, h16=None):
    """float32 -> bf16 values (as float32); stochastic with h16."""
    b = p.astype(F).view(np.uint32).astype(np.uint64)
    add = np.uint64(0x7FFF) + ((b >> np.uint64(16)) & np.uint64(1)) if h16 is None else h16.astype(np.uint64)
    return ((b + add) & np.uint64(0xFFFF0000)).astype(np.uint32).view(F)
