"""Plain 64-bit implementations of the attention operators (numpy, CPU),
written from the definitions in include/qoq_attn.h, for the tests."""
import numpy as np

HALF_STEP = 2.0 ** -11        # a rounding to FP16, relative


def positions(cu, kv_len):
    """(sequence, position) of every row, -1 where a row has no sequence."""
    T = int(cu[-1])
    seq, pos = np.full(T, -1), np.zeros(T, dtype=np.int64)
    for b in range(len(cu) - 1):
        n = int(cu[b + 1] - cu[b])
        seq[cu[b]:cu[b + 1]] = b
        pos[cu[b]:cu[b + 1]] = int(kv_len[b]) - n + np.arange(n)
    return seq, pos


def place(table, pages, page_size, b, pos):
    """(page, offset) or None where the page is absent."""
    if pos < 0 or pos // page_size >= table.shape[1]:
        return None
    p = int(table[b, pos // page_size])
    return (p, pos % page_size) if 0 <= p < pages else None


def rotate64(x, pos, freq, interleaved, amplitude=1.0):
    """x FP16 [T, H, d] -> FP64, the first 2 * len(freq) channels turned."""
    y = x.astype(np.float64).copy()
    n = len(freq)
    a = np.asarray(pos, dtype=np.float64)[:, None, None] * np.asarray(freq, dtype=np.float64)
    c, s = amplitude * np.cos(a), amplitude * np.sin(a)
    one, two = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    x1, x2 = y[..., one].copy(), y[..., two].copy()
    y[..., one], y[..., two] = x1 * c - x2 * s, x1 * s + x2 * c
    return y


def quantise(x, bits):
    """x FP16 [..., d] -> (codes uint8 [..., d], scale FP16 [...], minimum FP16 [...])."""
    f = x.astype(np.float32)
    m = f.min(-1)
    r = (f.max(-1) - m) / np.float32(2 ** bits - 1)
    s = r.astype(np.float16)
    s = np.where(s.astype(np.float32) > r, (s.view(np.uint16) - 1).view(np.float16), s)
    sf = s.astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(sf == 0, np.float32(0), np.minimum(np.rint((f - m[..., None]) / sf), np.float32(2 ** bits - 1)))
    return c.astype(np.uint8), s, m.astype(np.float16)


def unpack(rows, bits):
    return np.stack([rows & 15, rows >> 4], -1).reshape(*rows.shape[:-1], 2 * rows.shape[-1]) if bits == 4 else rows


def values64(rows, par, bits):
    """Packed rows and (scale, minimum) FP16 -> the values they stand for, FP64."""
    return unpack(rows, bits) * par[..., :1].astype(np.float64) + par[..., 1:].astype(np.float64)


def attend(q, k, v, seen, scale):
    """q [n, d], k, v [L, d] (FP64), seen [n, L] -> (out, spread): spread bounds the output's error by the operands'
    roundings (see `tolerance`)."""
    s = scale * (q @ k.T)
    size = abs(scale) * (np.abs(q) @ np.abs(k).T)
    s = np.where(seen, s, -np.inf)
    top = s.max(-1, keepdims=True, initial=-np.inf)
    p = np.where(seen, np.exp(s - np.where(np.isfinite(top), top, 0)), 0.0)
    l = p.sum(-1, keepdims=True)
    w = np.divide(p, l, out=np.zeros_like(p), where=l > 0)
    out = w @ v
    worst = np.where(seen, size, 0).max(-1, keepdims=True, initial=0.0)
    return out, tolerance(out, w @ np.abs(v), worst)


def tolerance(out, mass, worst):
    """A bound of |error|. The output is rounded to FP16 once (half a step, at least half the smallest subnormal).  The
    product's weights and the cached values are rounded to FP16: half a step of `mass` = sum w |v| each.  Keys
    rounded to FP16 move a score by at most half a step of `worst` = scale * max sum |q k|, which changes a weight
    by that factor up and its normaliser by the same down.  FP32 sums of up to 2^17 terms and the exponential add
    at most 2^-16 of the mass and of a score of that size."""
    eps = HALF_STEP
    return (eps * np.abs(out) + 2.0 ** -25 + 2 * eps * mass + 2 * (eps + 2.0 ** -19) * worst * mass * 1.01 +
            2.0 ** -16 * mass)
