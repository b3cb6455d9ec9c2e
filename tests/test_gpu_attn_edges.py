"""The attention operators where their inputs are unusual: copied cache handles, row tiles without
keys between others, queries with a few large channels,
mass in the tail of the weights; and whether every token
of a long context counts, once; NaN and infinities.  (The operators themselves:
test_gpu_attn.py, whose helpers are used here.)"""
import copy
import pickle

import numpy as np
import pytest
import torch

import attn_ref as ref
import w4a8_integer_gemm_b200 as q
from attn_norm import norm_tolerance
from test_gpu_attn import DEV, Batch, _check_paged, _check_prompt, _dev, _filled_pool, _freq, _half, _poisoned_pool, _rng

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


# ------------------------------------------------------ every token counted ----
def _marked_cache(b, Hkv, d, bits):
    """A cache whose values mark their 16-token granule: granule n of a sequence has ones in channel 5 n mod d."""
    c = _poisoned_pool(b, Hkv, d, bits)
    V = np.zeros((sum(b.kv), 1, d), np.float16)
    at = 0
    for n in b.kv:
        V[at + np.arange(n), 0, 5 * (np.arange(n) // 16) % d] = 1
        at += n
    r = _rng(1)
    K = _half(r, sum(b.kv), 1, d)
    cu = _dev(np.concatenate([[0], np.cumsum(b.kv)]).astype(np.int32))
    K, V = (_dev(np.repeat(x, Hkv, 1)) for x in (K, V))
    q.qattn_cache_append(K, V, c, b.dev[0], cu, b.dev[2])
    return c


@pytest.mark.parametrize("G,new,kv,d,bits", [
    (4, [1], [20000], 128, 4), (4, [1], [7777], 128, 8), (1, [1, 1, 1], [131, 20011, 4999], 64, 4), (16, [1, 1], [30000, 16], 128, 4),
    (32, [1], [9001], 64, 8), (8, [1] * 40, [300 + 211 * i for i in range(40)], 128, 4), (4, [3, 8], [5000, 7000], 64, 4),
    (8, [64], [20000], 128, 4), (4, [300, 70], [7777, 15001], 64, 8), (1, [513, 1, 40], [6000, 9000, 3000], 128, 8), (64, [1], [12000], 128, 4)])
def test_every_token_counts_once(G, new, kv, d, bits):
    """Queries of zeros weigh all tokens alike, so a channel of the output is the share of its granules' tokens: a granule
    that is left out or counted twice at a cut moves it by 6% or more here, a single token by 2^-8 or more."""
    Hkv = 2
    b = Batch(new, kv, 16, seed=G)
    c = _marked_cache(b, Hkv, d, bits)
    Q = torch.zeros(b.T, G * Hkv, d, dtype=torch.float16, device=DEV)
    for hint in (max(new), None, 1):
        o = q.qattn_paged_attention(Q, c, *b.dev, max_new=hint).cpu().numpy().astype(np.float64)
        for t in range(b.T):
            n = b.pos[t] + 1
            count = np.bincount(5 * (np.arange(n) // 16) % d, minlength=d)
            one = _one(bits)                                  # what the cache makes of a one among zeros
            want = one * count / n
            # weights of 1 and codes are exact operands; the cached one in FP16 (tiles) and the output are rounded.  FP32:
            # centred, every token adds half a one to every channel, and its half comes off again; up to 2^7 additions
            # in a share round by 2^-25 of what they have got to
            tol = (2 * ref.HALF_STEP + 2.0 ** -20) * want + 2.0 ** -18 * one / 2 + 2.0 ** -25
            assert np.all(np.abs(o[t] - want[None]) <= tol[None]), (hint, t, float((np.abs(o[t] - want) / tol).max()))


def _one(bits):
    code, s, m = ref.quantise(np.array([0.0, 1.0], np.float16), bits)
    return float(code[1]) * float(s) + float(m)


@pytest.mark.parametrize("new,kv,page,Hkv,Hq,d,bits,absent", [
    ([1, 1], [20000, 7777], 128, 2, 14, 128, 4, [(0, 7)]), ([1, 1], [9000, 300], 32, 1, 32, 64, 8, []),
    ([3, 5], [15000, 2000], 64, 2, 8, 128, 8, []), ([70, 1], [20000, 4000], 64, 1, 8, 128, 4, []),
    ([40, 64], [9000, 1200], 16, 1, 7, 64, 8, [(0, 3)]), ([130, 3], [6000, 800], 32, 2, 4, 128, 8, [])])
def test_errors_in_the_norm(new, kv, page, Hkv, Hq, d, bits, absent):
    """Long contexts, where a token lost at a cut is beyond the bound (test_attn_norm.py)."""
    b = Batch(new, kv, page, seed=d, absent=absent)
    c = _filled_pool(b, Hkv, d, bits, seed=bits)
    Q = _half(_rng(11), b.T, Hq, d)
    for hint in (max(new), 1):
        o = q.qattn_paged_attention(_dev(Q), c, *b.dev, max_new=hint)
        tiles = hint > 1 and max(new) * Hq // Hkv > 32        # (tiles round the cached keys and values to FP16)
        worst = _norm_errors(b, c, Q, Hkv, bits, d ** -0.5, o.cpu().numpy(), keys=tiles, values=tiles)
        assert worst < 1, (hint, worst)


# ------------------------------------------------------------ not finite ----
BAD = {"nan": float("nan"), "inf": float("inf"), "-inf": float("-inf")}


@pytest.mark.parametrize("what", list(BAD))
@pytest.mark.parametrize("d,bits,rot", [(64, 4, 0), (128, 4, 128), (128, 8, 32), (64, 8, 64)])
def test_append_keeps_what_is_not_finite(d, bits, rot, what):
    """Every value of a cached row with a NaN or an infinity reads back as one; the other rows are as without it."""
    Hkv, n = 3, 70
    b = Batch([n], [n + 5], 16, seed=d)
    x = _half(_rng(d + bits), n, 2 * Hkv, d)
    y = x.copy()
    bad = np.zeros((n, 2 * Hkv), dtype=bool)
    for t, h, ch in ((0, 0, [0]), (3, 4, [d - 1]), (n - 1, 5, [d // 2]), (17, 2, range(0, d, 5)), (30, 1, range(d)), (31, 3, range(d))):
        y[t, h, list(ch)] = BAD[what]
        bad[t, h] = True
    y[40, 1, :2], bad[40, 1] = [float("inf"), float("-inf")], True
    got = []
    for rows in (x, y):
        c = _poisoned_pool(b, Hkv, d, bits)
        rotary = q.Rotary(_dev(_freq(rot))) if rot else None
        xd = _dev(rows)
        q.qattn_cache_append(xd[:, :Hkv], xd[:, Hkv:], c, *b.dev, rotary=rotary)
        got.append(np.concatenate([t.cpu().numpy() for t in q.qattn_cache_read(c, *b.dev, n)], 1))
    assert np.array_equal(got[0][~bad], got[1][~bad]) and np.isfinite(got[0]).all()
    assert np.isnan(got[1][bad]).all()


PLACES = [  # new, kv, Hq, Hkv, d, bits, hint: a run in one warp, runs over warps and CTAs, 16 rows, tiles of one CTA and of several
    ([1], [40], 4, 1, 64, 4, 1), ([1, 1], [9000, 40], 8, 2, 128, 4, 1), ([1] * 30, [2000] * 30, 8, 2, 128, 8, 1), ([2, 1], [3000, 90], 32, 2, 64, 8, 2),
    ([60, 1], [9000, 300], 8, 2, 128, 4, None), ([300, 40], [500, 40], 4, 2, 64, 8, 300), ([50], [70], 2, 1, 128, 8, 50)]


@pytest.mark.parametrize("new,kv,Hq,Hkv,d,bits,hint", PLACES)
def test_paged_attention_keeps_what_is_not_finite(new, kv, Hq, Hkv, d, bits, hint):
    """A row of q with a NaN or an infinity, and the rows that see a cached key or value row with one, come out as NaN or
    infinities throughout.  Other sequences and KV heads have the bits that they have without it.  Rows of the same work
    item may have their maximum taken at other times, so that the weights' and the output's roundings differ: by 2^-11 of
    the largest value each, in either call."""
    b = Batch(new, kv, 16, seed=d)
    c = _filled_pool(b, Hkv, d, bits, seed=3)
    Q = _half(_rng(4), b.T, Hq, d)
    G = Hq // Hkv

    def run(Q):
        return q.qattn_paged_attention(_dev(Q), c, *b.dev, max_new=hint).cpu().numpy()

    clean = run(Q)
    assert np.isfinite(clean).all()
    near = 2.0 ** -8 * max(float(np.abs(_cached(b, c, s, h, bits)[1]).max()) for s in range(len(new)) for h in range(Hkv))
    for value in BAD.values():
        for row, head, ch in ((0, 0, 0), (b.T - 1, Hq - 1, d - 1), (b.T // 2, Hq // 2, d // 2)):
            Z = Q.copy()
            Z[row, head, ch] = value
            o = run(Z)
            hit = np.zeros((b.T, Hq), dtype=bool)
            hit[row, head] = True
            assert not np.isfinite(o[hit]).any()
            assert np.abs(o[~hit].astype(np.float64) - clean[~hit].astype(np.float64)).max() <= near
            hit[b.seq == b.seq[row], head // G * G:head // G * G + G] = True     # what shares work items with it
            assert np.array_equal(o[~hit], clean[~hit])
    old = min(b.kv[0] - b.new[0], 37)                         # a token that every row of the sequence sees
    for token in sorted({0, old, max(0, b.kv[0] - b.new[0] - 1)}):
        page, off = b.place(0, token)
        for par in (c.k_par, c.v_par):
            kept = par[page, Hkv - 1, off].clone()
            par[page, Hkv - 1, off] = float("nan")
            o = run(Q)
            hit = np.zeros((b.T, Hq), dtype=bool)
            hit[:b.new[0], (Hkv - 1) * G:] = True
            assert np.array_equal(o[~hit], clean[~hit])
            assert not np.isfinite(o[hit]).any(), token
            par[page, Hkv - 1, off] = kept
    assert np.array_equal(run(Q), clean)


@pytest.mark.parametrize("d,Hq,Hkv", [(64, 2, 1), (128, 3, 3)])
def test_prompt_attention_keeps_nan(d, Hq, Hkv):
    """A NaN key (each column of a key tile in turn) makes the rows that see it NaN, a NaN or infinite value its channel, a
    row of q with one itself; other prompts and KV heads keep their bits, other rows their values up to the roundings of
    weights and outputs (2^-11 of the largest value each, in either call)."""
    lens = [300, 270]
    T, G = sum(lens), Hq // Hkv
    X = _half(_rng(d), T, Hq + 2 * Hkv, d)
    cu = _dev(np.array([0, 300, T], np.int32))

    def run(X):
        return q.qattn_prompt_attention(*_dev(X).split([Hq, Hkv, Hkv], 1), cu).cpu().numpy()

    clean = run(X)
    near = 2.0 ** -8 * float(np.abs(X[:, Hq + Hkv:]).max())
    first = np.arange(T) < 300
    for j in list(range(0, 16)) + [63, 64, 127, 128, 140, 299]:
        Z = X.copy()
        Z[j, Hq + Hkv - 1, j % d] = np.nan
        o = run(Z)
        sees = first & (np.arange(T) >= j)
        assert not np.isfinite(o[sees, (Hkv - 1) * G:]).any(), j
        assert np.array_equal(o[~first], clean[~first]) and np.array_equal(o[:, :(Hkv - 1) * G], clean[:, :(Hkv - 1) * G])
        # (a masked key only makes masked scores)
        assert not j or np.abs(o[:j].astype(np.float64) - clean[:j].astype(np.float64)).max() <= near
    for value in (np.nan, np.inf):
        Z = X.copy()
        Z[20, Hq + 2 * Hkv - 1, 5] = value
        o = run(Z)
        assert not np.isfinite(o[20:300, (Hkv - 1) * G:, 5]).any() and np.array_equal(o[300:], clean[300:])
        other = np.arange(d) != 5
        assert np.array_equal(o[..., other], clean[..., other])
        Z = X.copy()
        Z[33, 0, 7] = value
        o = run(Z)
        hit = np.zeros((T, Hq), dtype=bool)
        hit[33, 0] = True
        assert not np.isfinite(o[hit]).any()
        assert np.abs(o[~hit].astype(np.float64) - clean[~hit].astype(np.float64)).max() <= near
        assert np.array_equal(o[300:], clean[300:]) and np.array_equal(o[:, G:], clean[:, G:])
