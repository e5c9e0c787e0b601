"""AdamW over one tensor and the 8-bit form of its states (TEST INFRASTRUCTURE
ONLY).

  m <- b1 m + (1 - b1) g,  v <- b2 v + (1 - b2) g^2
  w <- w - lr ((m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps) + wd w)
[KINGMA15] Kingma & Ba, ICLR 2015, Algorithm 1; [LOSHCHILOV19] Loshchilov &
Hutter, "Decoupled Weight Decay Regularization", ICLR 2019, Algorithm 2.

8-bit form: blocks of 32 entries share an exponent E in 16..254.  A magnitude
keeps `keep` mantissa bits (3 for m, 4 for sqrt(v)) over the 16 binades up to
2^(E - 127): with q the spacing at x, it is floor(x / q + u) q for the dither
u in [0, 1) of the entry and step.  Values below the least code are 0 (m) or
the least value (sqrt(v) > 0); a block of zeros has E = 16.  E = 255: the block holds a non-finite value.
All arithmetic is fp64 (written with frexp and ldexp, not with bit patterns).
"""
import numpy as np

BLOCK = 32
KEEP = {"m": 3, "v": 4}


def step(w, g, m, v, lr, b1, b2, eps, wd, t):
    """(w, m, v) after one step; v is the second moment itself."""
    m = b1 * m + (1.0 - b1) * g
    v = b2 * v + (1.0 - b2) * g * g
    upd = (m / (1.0 - b1 ** t)) / (np.sqrt(v / (1.0 - b2 ** t)) + eps)
    return w - lr * (upd + wd * w), m, v


def dither(n, t, which, first=0):
    """u in [0, 1) of entries first .. first + n - 1 at step t."""
    i = np.arange(first, first + n, dtype=np.uint64)
    h = i * np.uint64(0x6A09E667) + np.uint64(t) * np.uint64(0x9E3779B9)
    if which == "v":
        h = h + np.uint64(1 << 31)
    bits = 23 - KEEP[which]
    return ((h & np.uint64(0xFFFFFFFF)) >> np.uint64(32 - bits)).astype(np.float64) / 2.0 ** bits


def _blocks(x):
    pad = -len(x) % BLOCK
    return np.concatenate([x, np.zeros(pad)]).reshape(-1, BLOCK)


def encode(x, t, which, first=0):
    """(codes uint8, exponents uint8) of x = m, or sqrt(v) >= 0 (fp32 values)."""
    keep = KEEP[which]
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    u = dither(len(a), t, which, first)
    with np.errstate(invalid="ignore"):
        _, e = np.frexp(np.where(np.isfinite(a), a, 1.0))
        q = np.ldexp(1.0, np.maximum(e - 1, -126) - keep)
        y = np.floor(a / q + u) * q
    y = np.where(a == 0, 0.0, y)
    yb, ab = _blocks(y), _blocks(a)
    bad = ~np.isfinite(ab).all(axis=1) | (yb.max(axis=1) >= 2.0 ** 128)
    top = np.where(bad, 1.0, yb.max(axis=1))
    _, e = np.frexp(top)
    E = np.where(top == 0, 16, np.clip(e - 1 + 127, 16, 254))
    _, ey = np.frexp(np.where(yb > 0, yb, 1.0))
    yb = np.where(bad[:, None], 0.0, yb)
    mant = np.round(np.ldexp(yb, keep - (ey - 1))).astype(np.int64) - (1 << keep)
    c = (((ey - 1 + 127) - (E[:, None] - 15)) << keep) + mant
    c = np.where((yb > 0) & (c > 0), c, 0)
    if which == "v":
        c = np.where((ab > 0) & (c < 1), 1, c)
    c = c.reshape(-1)[:len(x)]
    if which == "m":
        c = c + np.where(np.signbit(x), 128, 0)
    return c.astype(np.uint8), np.where(bad, 255, E).astype(np.uint8)


def decode(codes, exps, which):
    """Values (fp64) of codes with their blocks' exponents."""
    keep = KEEP[which]
    codes = np.asarray(codes, np.int64)
    E = np.repeat(np.asarray(exps, np.int64), BLOCK)[:len(codes)]
    c = codes & 127 if which == "m" else codes
    x = np.ldexp(1.0 + (c % (1 << keep)) / 2.0 ** keep, (E - 15) + (c >> keep) - 127)
    x = np.where(c > 0, x, 0.0)
    x = np.where(E == 255, np.nan, x)
    return np.where((codes > 127) & (which == "m"), -x, x)
