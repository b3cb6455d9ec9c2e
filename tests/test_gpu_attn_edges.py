"""The attention operators where their inputs are unusual: copied cache handles, row tiles without
keys between others, queries with a few large channels,
mass in the tail of the weights.  (The operators themselves:
test_gpu_attn.py, whose helpers are used here.)"""
import copy
import pickle

import numpy as np
import pytest
import torch

import attn_ref as ref
import w4a8_integer_gemm_b200 as q
from attn_norm import norm_tolerance
from test_gpu_attn import Batch, _check_paged, _check_prompt, _dev, _filled_pool, _half, _poisoned_pool, _rng

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from w4a8_integer_gemm_b200 import build_lib
    build_lib.build()
    q.lib()
    yield
    torch.cuda.synchronize()
    assert q.qoq_device_error() == q.QOQ_OK


def _arrays(c):
    return c.k_codes, c.v_codes, c.k_par.view(torch.int16), c.v_par.view(torch.int16)


@pytest.mark.parametrize("way", [copy.deepcopy, lambda c: pickle.loads(pickle.dumps(c))])
def test_append_to_a_copied_handle(way):
    """A snapshot of a cache is written and read; the original keeps every byte."""
    d, Hkv, bits = 64, 2, 4
    b = Batch([3, 1], [40, 17], 16, seed=4)
    c = _filled_pool(b, Hkv, d, bits, seed=4)
    kept = [t.clone() for t in _arrays(c)]
    snap = way(c)
    x = _dev(_half(_rng(6), b.T, 2 * Hkv, d))
    q.qattn_cache_append(x[:, :Hkv], x[:, Hkv:], snap, *b.dev)
    q.qattn_cache_append(x[:, :Hkv], x[:, Hkv:], c2 := copy.deepcopy(c), *b.dev)
    assert all(torch.equal(t, k) for t, k in zip(_arrays(c), kept))
    q.qattn_cache_append(x[:, :Hkv], x[:, Hkv:], c, *b.dev)
    for y in (snap, c2):
        assert all(torch.equal(t, k) for t, k in zip(_arrays(y), _arrays(c)))
    assert not all(torch.equal(t, k) for t, k in zip(_arrays(c), kept))


@pytest.mark.parametrize("d", [64, 128])
def test_row_tiles_without_keys(d):
    """Items of one and of two row tiles in turn, several to a CTA: the second row tile has keys in one item and none in
    the next.  The values are right, and the same every time."""
    Hkv, Hq, bits, new = 8, 8, 8, [200, 64, 129, 128] * 20
    X = _half(_rng(d), sum(new), Hq + 2 * Hkv, d)
    qd, kd, vd = _dev(X).split([Hq, Hkv, Hkv], 1)
    cu = _dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))
    o = q.qattn_prompt_attention(qd, kd, vd, cu)
    _check_prompt(X, new, Hq, Hkv, o.cpu().numpy(), d ** -0.5)
    # over a cache; every fifth sequence has no positions for its rows (they see nothing)
    kv = [0 if i % 5 == 4 else n + 40 * (i % 7) for i, n in enumerate(new)]
    b = Batch(new, kv, 16, seed=3)
    c = _filled_pool(b, Hkv, d, bits, seed=5)
    at = np.arange(0, b.T, 7)
    p = q.qattn_paged_attention(qd, c, *b.dev, max_new=200)
    _check_paged(b, c, X[:, :Hq], Hkv, bits, d ** -0.5, p.cpu().numpy(), rows=at)
    for _ in range(20):
        assert torch.equal(q.qattn_prompt_attention(qd, kd, vd, cu).view(torch.int16), o.view(torch.int16))
        assert torch.equal(q.qattn_paged_attention(qd, c, *b.dev, max_new=200).view(torch.int16), p.view(torch.int16))


def _cached(b, c, s, h, bits):
    """Keys, values (FP64) of sequence s and KV head h, and which tokens are there."""
    kc, vc, kp, vp = (t.cpu().numpy() for t in (c.k_codes, c.v_codes, c.k_par, c.v_par))
    at = [b.place(s, p) for p in range(max(b.kv[s], 0))]
    there = np.array([p is not None for p in at], dtype=bool)
    pg, off = (np.array([p[i] if p else 0 for p in at], dtype=int) for i in (0, 1))
    k, v = (np.where(there[:, None], ref.values64(x[pg, h, off], y[pg, h, off], bits), 0) for x, y in ((kc, kp), (vc, vp)))
    return k, v, there


def _norm_errors(b, c, Q, Hkv, bits, scale, got, **rounded):
    """The largest error in the norm of a row of `got`, in units of its tolerance."""
    G, most = Q.shape[1] // Hkv, 0.0
    for s in range(len(b.new)):
        t = np.arange(b.cu[s], b.cu[s + 1])
        for h in range(Hkv if len(t) else 0):
            k, v, there = _cached(b, c, s, h, bits)
            seen = there[None] & (np.arange(len(there))[None] <= b.pos[t][:, None])
            for g in range(G):
                o, tol = norm_tolerance(Q[t, h * G + g].astype(np.float64), k, v, seen, scale, **rounded)
                err = np.linalg.norm(got[t, h * G + g].astype(np.float64) - o, axis=-1)
                most = max(most, float((err / tol).max()))
    return most


@pytest.mark.parametrize("times", [1, 30, 100, 300])
@pytest.mark.parametrize("new,kv,Hq,d,bits", [([1, 1], [2000, 515], 8, 128, 4), ([1], [3000], 4, 64, 8), ([1], [1200], 32, 128, 8),
                                              ([2, 5], [900, 400], 6, 64, 4)])
def test_queries_with_large_channels(new, kv, Hq, d, bits, times):
    """Few rows, a channel of q as many times the rest as is said and small in the keys: the other channels, which decide
    the scores, keep their bits."""
    Hkv = 2
    b = Batch(new, kv, 16, seed=times)
    c = _filled_pool(b, Hkv, d, bits, seed=7)
    Q = _half(_rng(8), b.T, Hq, d)
    quiet = int(np.abs(_cached(b, c, 0, 0, bits)[0]).mean(0).argmin())
    Q[..., quiet] = (Q[..., quiet].astype(np.float32) * times).astype(np.float16)
    o = q.qattn_paged_attention(_dev(Q), c, *b.dev, max_new=max(new))
    worst = _norm_errors(b, c, Q, Hkv, bits, d ** -0.5, o.cpu().numpy())
    assert worst < 1, worst


def _tail_case(n, d, first):
    """Keys and values [n, d]: one token (the first, or one in the middle) that outweighs each other by 2^27 to 2^31 for a
    query of ones, with values of zero; the others have no scores and large values, the same in every channel, so
    that a 4- or 8-bit row holds them exactly."""
    k, v = np.zeros((n, d), np.float16), np.zeros((n, d), np.float16)
    v[:] = (40000 + 64 * (np.arange(n) % 300))[:, None].astype(np.float16)
    at = 0 if first else n // 2
    k[at] = np.float16(29 * np.log(2) / d ** 0.5)
    v[at] = 0
    return k, v


def _check_tail(q_rows, k, v, pos, got, scale):
    """Within attn_ref's bound and what rounding the weights costs below FP16's normal numbers: half a step, 2^-25, of
    a weight of one, 2^-8 of the largest: 2^-33 of it each, times the values."""
    k, v = k.astype(np.float64), v.astype(np.float64)
    for i, p in enumerate(pos):
        seen = (np.arange(len(k)) <= p)[None]
        o, tol = ref.attend(q_rows[i:i + 1].astype(np.float64), k, v, seen, scale)
        largest = 1.0                                         # the weights' sum is the largest one's within 2^-10
        err = np.abs(got[i].astype(np.float64) - o[0])
        assert np.all(err <= tol[0] + 2.0 ** -33 * largest * (np.abs(v) * seen[0][:, None]).sum(0)), (i, float(err.max()))
        assert o.min() > 0.05                                 # (the tail is what the output consists of)


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_mass_in_the_tail_of_a_prompt(d, first):
    n, scale = 4000, d ** -0.5
    k, v = _tail_case(n, d, first)
    X = np.zeros((n, 3, d), np.float16)
    X[:, 0] = (0.95 + 0.1 * _rng(1).random(n))[:, None]
    X[:, 1], X[:, 2] = k, v
    o = q.qattn_prompt_attention(*_dev(X).split([1, 1, 1], 1), _dev(np.array([0, n], np.int32))).cpu().numpy()
    at = np.array([2900, 3071, 3500, 3999])
    _check_tail(X[at, 0], k, v, at, o[at, 0], scale)


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("d,bits", [(64, 4), (128, 4), (128, 8)])
def test_mass_in_the_tail_of_a_cache(d, bits, first):
    n, new, scale = 9000, 64, d ** -0.5
    k, v = _tail_case(n, d, first)
    b = Batch([n], [n], 64, seed=2)
    c = _poisoned_pool(b, 1, d, bits)
    q.qattn_cache_append(_dev(k[:, None]), _dev(v[:, None]), c, *b.dev)
    Q = np.repeat((0.95 + 0.1 * _rng(2).random(new))[:, None, None], d, 2).astype(np.float16)
    cu = _dev(np.array([0, new], np.int32))
    o = q.qattn_paged_attention(_dev(Q), c, b.dev[0], cu, b.dev[2]).cpu().numpy()
    at = np.array([0, 31, 63])
    _check_tail(Q[at, 0], k, v, n - new + at, o[at, 0], scale)
