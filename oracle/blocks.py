"""CPU oracle of the gated block, the norms and the AdamW step: numpy in
float64, from the definitions.  Shares nothing with the product library."""
import numpy as np

SILU, GELU = 0, 1
EPS32 = 2.0 ** -24  # half a step of fp32, relative


# ---- gated feed-forward ----

def act_parts(g, act):
    """(s, z, z') with act(g) = g s(z(g))."""
    g = np.asarray(g, np.float64)
    if act == SILU:
        z, dz = g, np.ones_like(g)
    else:
        a = 2.0 * np.sqrt(2.0 / np.pi)
        z, dz = a * (g + 0.044715 * g ** 3), a * (1.0 + 3 * 0.044715 * g * g)
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-z))
    return s, z, dz


def act_value(g, act):
    return g * act_parts(g, act)[0]


def act_slope(g, act):
    s, _, dz = act_parts(g, act)
    return s + g * s * (1.0 - s) * dz


def gated(G, U, act):
    return act_value(G, act) * U


def gated_grad(D, G, U, act):
    """(dG, dU) for the gradient D of act(G) * U."""
    return D * U * act_slope(G, act), D * act_value(G, act)


# ---- norms ----

def norm_stats(x, eps, rms):
    x = np.asarray(x, np.float64)
    mean = np.zeros(x.shape[0]) if rms else x.mean(1)
    d = x - mean[:, None]
    return mean, 1.0 / np.sqrt((d * d).mean(1) + eps)


def norm(x, w, b, eps, rms):
    mean, rstd = norm_stats(x, eps, rms)
    y = (x - mean[:, None]) * rstd[:, None]
    y = y * (1.0 if w is None else w)
    return y + (0.0 if b is None else b), mean, rstd


def norm_grad(dy, x, w, mean, rstd, rms):
    """(dx, dw, db) of rows with the given statistics."""
    xh = (x - (0.0 if rms else mean[:, None])) * rstd[:, None]
    t = dy * (1.0 if w is None else w)
    dx = t - xh * (t * xh).mean(1, keepdims=True)
    if not rms:
        dx = dx - t.mean(1, keepdims=True)
    return dx * rstd[:, None], (dy * xh).sum(0), dy.sum(0)


# ---- AdamW with 32-bit or 8-bit moments ----

def e4m3_table():
    """Values of the 256 E4M3 codes, from the layout: sign, 4 exponent bits
    (bias 7), 3 mantissa bits; all ones below the sign is NaN, no infinities."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        mag = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if (c & 127) == 127:
            mag = np.nan
        v[c] = -mag if c & 128 else mag
    return v


def e4m3_scale_byte(amax):
    """E8M0 byte of a block: floor(log2 amax) - 7, clamped below at -127."""
    amax = np.asarray(amax, np.float64)
    e = np.frexp(np.where(amax > 0, amax, 1.0))[1] - 1 - 7
    return np.where(amax > 0, np.clip(e, -127, 127) + 127, 0).astype(np.int64)


def sr_e4m3(y, u):
    """Code of the magnitude y (0 <= y <= 256) rounded with 16 random bits:
    up iff u + floor(frac 2^16) >= 2^16."""
    y = np.asarray(y, np.float64)
    mags = e4m3_table()[:127]
    lo = np.clip(np.searchsorted(mags, y, side="right") - 1, 0, 125)
    frac = (y - mags[lo]) / (mags[lo + 1] - mags[lo])
    return lo + (np.floor(frac * 65536.0) + u >= 65536.0)


def philox_words(pos, step, seed):
    """32-bit word of each position: Philox4x32-10 with counter (position / 4,
    step, 0) and the seed as key; word position % 4."""
    pos = np.asarray(pos, np.uint64)
    low = np.uint64(0xFFFFFFFF)
    n = pos >> np.uint64(2)
    c = [n & low, n >> np.uint64(32), np.full_like(n, step), np.zeros_like(n)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        p0 = np.uint64(0xD2511F53) * c[0]
        p1 = np.uint64(0xCD9E8D57) * c[2]
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), p1 & low,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), p0 & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    c = np.stack(c, -1)
    return np.take_along_axis(c, (pos & np.uint64(3)).astype(np.int64)[..., None], -1)[..., 0]


def decode8(codes, scales):
    """Values of E4M3 codes [n] with a scale byte per 32 (0xFF: NaN)."""
    n = len(codes)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return e4m3_table()[codes] * np.repeat(s, 32)[:n]


def adamw(p, g, m, v, lr, beta1, beta2, eps, step, wd, grad_scale=1.0):
    """New (p, m, v) and the update's magnitude parts (|b1 m| + |a1 g|, denominator)."""
    g = g * grad_scale
    parts = np.abs(beta1 * m) + np.abs((1 - beta1) * g)
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    den = np.sqrt(v / (1 - beta2 ** step)) + eps
    up = lr * (m / (1 - beta1 ** step)) / den
    return p * (1 - lr * wd) - up, m, v, parts, den
