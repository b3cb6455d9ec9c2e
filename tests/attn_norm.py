"""Errors of attention in the norm, for the tests: the bound of attn_ref.tolerance is a worst case over every element, which
a lost token of a long context stays below; the error in the norm is not."""
import numpy as np

HALF_STEP = 2.0 ** -11        # a rounding to FP16, relative, at most


def norm_tolerance(q, k, v, seen, scale, keys=False, values=False):
    """(out [n, d], tol [n]) for q [n, d], k, v [L, d] in FP64 and seen [n, L]: tol bounds the norm of each row's error by the
    roundings that are taken for independent, each within HALF_STEP of what it rounds: the output; the weights P (sums of
    weights are not rounded); the values and the keys, where `values` and `keys` say that they are rounded to FP16.  A
    rounding moves
      the output by           out,
      weight j by             w_j,            and with it the output by  w_j v_j,
      value j by              v_j,                                       w_j v_j,
      key j in channel c by   k_jc, score j by scale q_c k_jc, and       w_j (v_j - out) times that.
    Their squares are added.  Uniform roundings have 1 / sqrt(3) of their bound as deviation; where one or two tokens hold
    the weight, the sum can reach the bounds of both, sqrt(3) * sqrt(2) = 2.45 deviations: 2.5 are allowed.  FP32 sums,
    exponentials and scores: 2^-19 of a score as large as the largest sum |q k|, and 2^-14 of a weight (prompts: the
    polynomial's 7.5e-5 = 2^-13.7 goes with P's rounding), once each, times w_j (v_j - out)."""
    s = np.where(seen, scale * (q @ k.T), -np.inf)
    top = s.max(-1, keepdims=True, initial=-np.inf)
    p = np.where(seen, np.exp(s - np.where(np.isfinite(top), top, 0)), 0.0)
    l = p.sum(-1, keepdims=True)
    w = np.divide(p, l, out=np.zeros_like(p), where=l > 0)
    out = w @ v
    w2 = w * w
    each = (v * v).sum(-1)                                                        # |v_j|^2
    apart = each[None] - 2 * out @ v.T + (out * out).sum(-1, keepdims=True)       # |v_j - out|^2
    var = (out * out).sum(-1) + (w2 @ each) * (2.0 if values else 1.0)
    if keys:
        var = var + (w2 * apart * scale ** 2 * ((q * q) @ (k * k).T)).sum(-1)
    size = abs(scale) * (np.abs(q) @ np.abs(k).T)
    worst = np.where(seen, size, 0).max(-1, initial=0.0)
    fp32 = (2.0 ** -14 + 2.0 ** -19 * worst) * np.sqrt((w2 * np.maximum(apart, 0)).sum(-1))
    tiny = 2.0 ** -25 * np.sqrt(v.shape[-1])                                      # half the smallest step of FP16
    return out, 2.5 * HALF_STEP / np.sqrt(3) * np.sqrt(var) + fp32 + tiny
