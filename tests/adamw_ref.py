"""Plain forms of the AdamW step and of its 8-bit states, for the tests."""
import numpy as np

U = 2.0 ** -24
BLOCK = 256


def step(p, g, m, v, t, lr, b1, b2, eps, decay, scale=1.0):
    """((p, m, v) after a step in 64 bits, the most that 32 bits may be off).

    With u = 2^-24.  g: one rounding.  m: its two products have a rounded
    factor each (b or 1 - b) and are rounded, then their sum: 3 u of each
    product, one more for g.  v: the same with g's rounding twice and the
    square's, so 3 u and 6 u.  p: 1 - lr decay and its product are 3 u of p
    (the factor has lr, decay, their product and the difference, all but the
    last scaled by lr decay <= 1), the sum one more.  The quotient: rate has
    the roundings of lr, of log b and its product with t (whose errors in 1 -
    b^t are at most their own relative size), 2 ulp of expm1 and the division,
    10 u; the root 8 u likewise, the square root and its product 2 u, the sum
    with eps and its rounding 2 u, rate * m and the division 2 u: 24 u together.
    What m and v are off comes on top."""
    f = np.float64
    x = g * f(scale)
    m1, v1 = b1 * m + (1 - b1) * x, b2 * v + (1 - b2) * x * x
    em = U * (3 * np.abs(b1 * m) + 4 * np.abs((1 - b1) * x)) + 2.0 ** -148
    ev = U * (3 * np.abs(b2 * v) + 6 * (1 - b2) * x * x) + 2.0 ** -148
    root = np.sqrt(v1 / (1 - b2 ** t))
    low = np.sqrt(np.maximum(v1 - ev, 0) / (1 - b2 ** t))
    rate = lr / (1 - b1 ** t)
    with np.errstate(divide="ignore", invalid="ignore"):
        change = np.where(m1 == 0, 0.0, rate * m1 / (root + eps))
        most = rate * (np.abs(m1) + em) / (low + eps)
    p1 = p * (1 - lr * decay) - change
    ep = U * (4 * np.abs(p) + np.abs(p1)) + np.abs(most) * 24 * U + np.abs(most - np.abs(change)) + 2.0 ** -148
    return (p1, m1, v1), (ep, em, ev)


def step32(m, v, g, b1, b2, scale=1.0):
    """The states in 32 bits, each product and sum rounded."""
    f = np.float32
    x = g.astype(f) * f(scale)
    return m * f(b1) + x * f(1 - b1), v * f(b2) + x * x * f(1 - b2)


def mix(x):
    x = np.asarray(x, np.uint32)
    with np.errstate(over="ignore"):
        x = x ^ (x >> np.uint32(16))
        x = x * np.uint32(0x6A09E667)
        x = x ^ (x >> np.uint32(15))
        x = x * np.uint32(0xBB67AE85)
    return x ^ (x >> np.uint32(16))


def dither(first, n, seed, step):
    """(16 bits for exp_avg, 16 for exp_avg_sq) of n elements from place `first` on."""
    at = np.arange(first, first + n, dtype=np.uint64)
    with np.errstate(over="ignore"):
        key = mix(mix(np.uint32(seed & 0xFFFFFFFF)) + np.uint32(step))
        r = mix(at.astype(np.uint32) ^ mix(key + (at >> np.uint64(32)).astype(np.uint32)))
    return r >> np.uint32(16), r & np.uint32(0xFFFF)


def value(codes, exponents, signed):
    """What codes stand for, in 64 bits, by the formula of their parts."""
    c = codes.astype(np.int64)
    size = c & 127 if signed else c
    e, f = size >> 3, size & 7
    top = 14 if signed else 30
    x = np.where(e > 0, np.ldexp(1 + f / 8, e - top), np.ldexp(f / 8, 1 - top))
    unit = np.ldexp(1.0, exponents.astype(np.int64) - 127)
    unit = np.where(exponents == 255, np.nan, np.where(exponents == 0, 0.0, unit)).repeat(BLOCK)[:c.size]
    x = x * unit
    return np.where(c > 127, -x, x) if signed else x


def encode(x, random, signed):
    """(codes, exponents) of float32 values in blocks; random: 16 bits each, or
    None for nearest (half a step up).  By shares of a step, in 64 bits."""
    n = x.size
    pad = -n % BLOCK
    a = np.concatenate([np.abs(x.astype(np.float64)), np.zeros(pad)]).reshape(-1, BLOCK)
    bits = np.concatenate([x.astype(np.float32).view(np.uint32), np.zeros(pad, np.uint32)]).reshape(-1, BLOCK)
    e = np.maximum((bits >> np.uint32(23) & np.uint32(255)).max(1).astype(np.int64), 1)
    bad = e >= 254
    top = 14 if signed else 30
    with np.errstate(invalid="ignore", over="ignore"):
        z = (a * np.ldexp(1.0, 127 - np.minimum(e, 253))[:, None]).ravel()[:n]
        z = np.where(np.isfinite(z), z, 0.0)
        field = np.maximum(np.floor(np.log2(np.maximum(z, 1e-300))), 1 - top)
        field = np.where(np.ldexp(1.0, field.astype(int)) > z, np.maximum(field - 1, 1 - top), field)
        shares = z / np.ldexp(1.0, field.astype(int) - 3)  # in steps of the code's last bit
        up = 0.5 if random is None else random / 65536.0
        q = np.floor(shares + up)
    base = np.where(field > 1 - top, (field + top - 1) * 8, 0)
    code = (base + q).astype(np.int64)
    if signed:
        code = code | np.where(x < 0, 128, 0)
    else:
        code = np.where((x > 0) & (code == 0), 1, code)
    code = np.where(bad.repeat(BLOCK)[:n], 0, code)
    return code.astype(np.uint8), np.where(bad, 255, e).astype(np.uint8)
