"""The bound of attention's error in the norm (attn_norm.py) sees what the elementwise one does not (no GPU)."""
import numpy as np
import pytest

from attn_norm import norm_tolerance


def _data(L, d, seed):
    r = np.random.default_rng(seed)
    k = r.standard_normal((L, d)).astype(np.float16).astype(np.float64)
    k[:, :2] *= 25
    return r.standard_normal((4, d)), k / 4, r.standard_normal((L, d)).astype(np.float16).astype(np.float64)


@pytest.mark.parametrize("L,lost", [(20000, 16), (20000, 64), (7777, 16), (2000, 4)])
def test_lost_tokens_are_beyond_the_bound(L, lost):
    """At least one query in four sees its error beyond the bound, and most do, when neighbouring tokens are left out."""
    d = 128
    q, k, v = _data(L, d, lost)
    seen = np.ones((4, L), dtype=bool)
    out, tol = norm_tolerance(q, k, v, seen, d ** -0.5, keys=True, values=True)
    beyond = 0
    for at in range(0, L - lost, L // 10):
        less = seen.copy()
        less[:, at:at + lost] = False
        wrong, _ = norm_tolerance(q, k, v, less, d ** -0.5)
        beyond += int((np.linalg.norm(wrong - out, axis=-1) > tol).sum())
    assert beyond >= 20                                       # of 40 and more


def test_rounded_operands_stay_within_it():
    """The roundings it allows for, made: weights, values, keys and the output in FP16."""
    d, L = 128, 1500
    half = lambda x: x.astype(np.float16).astype(np.float64)  # noqa: E731
    for seed in range(6):
        q, k, v = _data(L, d, seed)
        q, k, v = half(q), k * 1.003, v * 1.001
        out, tol = norm_tolerance(q, k, v, np.ones((4, L), dtype=bool), d ** -0.5, keys=True, values=True)
        s = d ** -0.5 * (q @ half(k).T)
        p = np.exp(s - s.max(-1, keepdims=True))
        got = half(half(p) @ half(v) / p.sum(-1, keepdims=True))
        err = np.linalg.norm(got - out, axis=-1) / tol
        assert err.max() < 1 and err.max() > 0.05
