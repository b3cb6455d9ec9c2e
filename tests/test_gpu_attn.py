"""The attention operators against plain 64-bit implementations (attn_ref.py), through the Python calls.

Codes, scales and read-back values are equal bit for bit.  A rotation is within half an FP16 step of the 64-bit value
(its own 64-bit error, far below 2^-30 of a step at these positions, aside).  Attention is within the bound that
attn_ref.tolerance derives from the roundings of its operands."""
import numpy as np
import pytest
import torch

import attn_ref as ref
import w4a8_integer_gemm_b200 as q

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from w4a8_integer_gemm_b200 import build_lib
    build_lib.build()
    q.lib()
    yield
    torch.cuda.synchronize()
    assert q.qoq_device_error() == q.QOQ_OK


def _rng(seed):
    return np.random.default_rng(seed)


def _half(r, *shape, outliers=False):
    x = r.standard_normal(shape)
    if outliers:
        x[..., r.integers(0, shape[-1], 2)] *= 25
    return x.astype(np.float16)


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _freq(rot, base=10000.0):
    return base ** (-2.0 * np.arange(rot // 2) / rot)


class Batch:
    """A batch with its pages in a shuffled pool; `absent`: (sequence, page of the sequence) that are dropped."""

    def __init__(self, new, kv, page=64, seed=0, absent=(), spare=2, extra_table=1):
        r = _rng(seed)
        self.new, self.kv, self.page = new, kv, page
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.kv_len = np.array(kv, dtype=np.int32)
        per = [max(0, -(-n // page)) for n in kv]
        self.pages = sum(per) + spare
        ids = list(r.permutation(self.pages))
        self.table = np.full((len(kv), max(per + [0]) + extra_table), -1, dtype=np.int32)
        for b, p in enumerate(per):
            for j in range(p):
                self.table[b, j] = ids.pop()
        for b, j in absent:
            self.table[b, j] = [-1, self.pages, 1 << 30][(b + j) % 3]
        self.T = int(self.cu[-1])
        self.seq, self.pos = ref.positions(self.cu, kv)
        self.dev = (_dev(self.table), _dev(self.cu), _dev(self.kv_len))

    def place(self, b, pos):
        return ref.place(self.table, self.pages, self.page, b, pos)


def _poisoned_pool(b, Hkv, d, bits):
    """A pool whose every byte is a pattern: codes 0xA5, parameters NaN."""
    c = q.paged_kv_cache(b.pages, Hkv, d, bits, b.page)
    for t in (c.k_codes, c.v_codes):
        t.fill_(0xA5)
    for t in (c.k_par, c.v_par):
        t.view(torch.int16).fill_(0x7E01)
    return c


def _filled_pool(b, Hkv, d, bits, seed):
    """A pool with quantised random tokens wherever the batch has some, the pattern elsewhere."""
    r = _rng(seed)
    c = _poisoned_pool(b, Hkv, d, bits)
    for codes, par, out in ((c.k_codes, c.k_par, True), (c.v_codes, c.v_par, False)):
        cn, pn = codes.cpu().numpy(), par.cpu().numpy()
        for s, L in enumerate(b.kv):
            for p0 in range(0, L, b.page):
                at, n = b.place(s, p0), min(b.page, L - p0)
                if at is None:
                    continue
                x = _half(r, Hkv, n, d, outliers=out) / np.float16(4 if out else 1)
                k, sc, m = ref.quantise(x, bits)
                cn[at[0], :, :n] = k[..., 0::2] | (k[..., 1::2] << 4) if bits == 4 else k
                pn[at[0], :, :n, 0], pn[at[0], :, :n, 1] = sc, m
        codes.copy_(torch.from_numpy(cn)), par.copy_(torch.from_numpy(pn))
    return c


# ---------------------------------------------------------------- rotary ----
@pytest.mark.parametrize("T,H,d,rot,inter,amp", [(1, 1, 64, 64, False, 1.0), (3, 5, 128, 128, True, 1.0), (37, 12, 128, 32, False, 1.2),
                                                 (2500, 3, 64, 16, True, 0.7), (9, 2, 80, 48, False, 1.0), (5, 7, 512, 512, True, 1.0),
                                                 (4, 2, 128, 0, False, 1.0)])
def test_rotary(T, H, d, rot, inter, amp):
    r = _rng(T + H)
    x = _half(r, T, H + 2, d)
    pos = r.integers(0, 1 << 21, T).astype(np.int32)
    pos[0] = -7 if T > 1 else 0
    f = _freq(rot, 5e5) if rot else np.zeros(0)
    rot_ = q.Rotary(_dev(f), inter, amp)
    wide = _dev(x)
    y = q.qattn_rotary(wide[:, 1:H + 1], _dev(pos), rot_)
    want = ref.rotate64(x[:, 1:H + 1], pos, f, inter, amp)
    got = y.cpu().numpy().astype(np.float64)
    if amp == 1.0:
        step = np.spacing(np.abs(want).astype(np.float16)).astype(np.float64)
        assert np.all(np.abs(got - want) <= 0.5 * step * (1 + 1e-6))
    else:                                                     # the factor is a float32: relative 2^-24 before the rounding
        assert np.all(np.abs(got - want) <= (ref.HALF_STEP + 2.0 ** -23) * np.abs(want) + np.abs(x[:, 1:H + 1]).max() * 2.0 ** -23 + 2.0 ** -25)
    same = q.qattn_rotary(wide[:, 1:H + 1], _dev(pos), rot_, out=wide[:, 1:H + 1])    # in place, strided
    assert torch.equal(same.view(torch.int16), y.view(torch.int16))
    assert np.array_equal(wide[:, 0].cpu().numpy(), x[:, 0]) and np.array_equal(wide[:, -1].cpu().numpy(), x[:, -1])


# ----------------------------------------------------------------- cache ----
CACHE = [  # new, kv_len, page, Hkv, Hq, d, bits, rot, interleaved, absent pages
    ([1], [1], 16, 1, 1, 64, 4, 64, False, []),
    ([1, 1, 1], [5, 64, 65], 64, 2, 8, 128, 4, 128, False, []),
    ([0, 7, 40, 0, 1], [0, 7, 100, 30, 17], 16, 3, 21, 128, 8, 32, True, [(2, 5)]),
    ([130, 3], [130, 400], 32, 8, 8, 64, 8, 64, True, [(1, 12)]),
    ([2500], [2600], 128, 4, 16, 128, 4, 64, False, [(0, 3)]),
    ([5], [3], 16, 2, 2, 64, 4, 0, False, []),                # more new tokens than cached: two have no position
]


@pytest.mark.parametrize("new,kv,page,Hkv,Hq,d,bits,rot,inter,absent", CACHE)
def test_append_and_read(new, kv, page, Hkv, Hq, d, bits, rot, inter, absent):
    r = _rng(sum(new) + d)
    b = Batch(new, kv, page, seed=len(new), absent=absent)
    pad = 3                                                   # rows behind the last sequence
    x = _half(r, b.T + pad, Hq + 2 * Hkv, d, outliers=True)
    x[0, Hq] = 0.5                                            # a constant row: scale 0
    x[0, Hq + Hkv, :2] = [65504, -65504]                      # the widest range
    x[-1 - pad, Hq + Hkv] = np.float16(2.0 ** -24) * (np.arange(d) % 3)   # subnormals
    c = _poisoned_pool(b, Hkv, d, bits)
    before = [t.clone() for t in (c.k_codes, c.v_codes, c.k_par.view(torch.int16), c.v_par.view(torch.int16))]
    xd = _dev(x)
    qd, kd, vd = xd.split([Hq, Hkv, Hkv], 1)
    f = _freq(rot)
    keys = x[:b.T, Hq:Hq + Hkv]
    if rot:
        rotary = q.Rotary(_dev(f), inter)
        q_out = torch.full((b.T + pad, Hq, d), 7.0, dtype=torch.float16, device=DEV)
        got_q = q.qattn_cache_append(kd, vd, c, *b.dev, rotary=rotary, q=qd, q_out=q_out)
        assert got_q is q_out and bool((q_out[b.T:] == 7).all())
        pos = _dev(b.pos.astype(np.int32))
        assert torch.equal(q_out[:b.T].view(torch.int16), q.qattn_rotary(qd[:b.T], pos, rotary).view(torch.int16))
        keys = q.qattn_rotary(kd[:b.T], pos, rotary).cpu().numpy()
    else:
        assert q.qattn_cache_append(kd, vd, c, *b.dev) is None
    want = [t.cpu().numpy() for t in before]
    wantK, wantV = np.zeros((b.T, Hkv, d), np.float16), np.zeros((b.T, Hkv, d), np.float16)
    for n, (rows, w) in enumerate(((keys, wantK), (x[:b.T, Hq + Hkv:], wantV))):
        for t in range(b.T):
            at = b.place(b.seq[t], b.pos[t])
            if at is None:
                continue
            code, s, m = ref.quantise(rows[t], bits)
            packed = code[..., 0::2] | (code[..., 1::2] << 4) if bits == 4 else code
            want[n][at[0], :, at[1]] = packed
            want[2 + n][at[0], :, at[1], 0], want[2 + n][at[0], :, at[1], 1] = s.view(np.int16), m.view(np.int16)
            w[t] = ref.values64(packed, np.stack([s, m], -1), bits).astype(np.float16)
    for t, w, name in zip((c.k_codes, c.v_codes, c.k_par.view(torch.int16), c.v_par.view(torch.int16)), want, "kvkv"):
        got = t.cpu().numpy()
        if got.dtype == np.int16:                             # the sign of a zero minimum is not part of the format
            got, w = np.where(got == -32768, 0, got), np.where(w == -32768, 0, w)
        assert np.array_equal(got, w), name
    K, V = (torch.full((b.T + pad, Hkv, d), 7.0, dtype=torch.float16, device=DEV) for _ in range(2))
    q.qattn_cache_read(c, *b.dev, b.T + pad, K=K, V=V)
    assert np.array_equal(K[:b.T].cpu().numpy(), wantK) and np.array_equal(V[:b.T].cpu().numpy(), wantV)
    assert bool((K[b.T:] == 7).all()) and bool((V[b.T:] == 7).all())


# ------------------------------------------------------ attention, paged ----
def _check_paged(b, c, Q, Hkv, bits, scale, got, rows=None):
    kc, vc, kp, vp = (t.cpu().numpy() for t in (c.k_codes, c.v_codes, c.k_par, c.v_par))
    Hq, d = Q.shape[1:]
    G = Hq // Hkv
    for s, L in enumerate(b.kv):
        n = b.new[s]
        t = np.arange(b.cu[s], b.cu[s] + n)
        if rows is not None:
            t = t[np.isin(t, rows)]
        if not len(t):
            continue
        places = [b.place(s, p) for p in range(max(L, 0))]
        there = np.array([p is not None for p in places], dtype=bool)
        pg = np.array([p[0] if p else 0 for p in places], dtype=int)
        off = np.array([p[1] if p else 0 for p in places], dtype=int)
        seen = there[None] & (np.arange(max(L, 0))[None] <= b.pos[t][:, None])
        for h in range(Hkv):
            k = np.where(there[:, None], ref.values64(kc[pg, h, off], kp[pg, h, off], bits), 0)
            v = np.where(there[:, None], ref.values64(vc[pg, h, off], vp[pg, h, off], bits), 0)
            for g in range(G):
                o, tol = ref.attend(Q[t, h * G + g].astype(np.float64), k, v, seen, scale)
                err = np.abs(got[t, h * G + g].astype(np.float64) - o)
                assert np.all(err <= tol), (s, h, g, float((err / tol).max()))
                assert not got[t, h * G + g][~seen.any(-1)].any()


PAGED = [  # new, kv_len, page, Hkv, Hq, d, bits, absent pages
    ([1], [1], 16, 1, 1, 64, 4, []),
    ([1, 1, 1, 1], [1, 63, 64, 65], 64, 2, 8, 128, 4, []),
    ([1, 1, 1], [1000, 0, 129], 16, 8, 32, 128, 8, [(0, 3), (0, 62), (2, 0)]),
    ([1, 1], [20000, 7777], 128, 2, 14, 128, 4, [(0, 7)]),
    ([1, 1], [9000, 300], 32, 1, 64, 64, 8, []),
    ([2, 1, 0, 4], [70, 700, 50, 4], 32, 4, 4, 64, 4, [(1, 20)]),
    ([17, 33, 1], [17, 400, 900], 64, 2, 6, 128, 4, []),
    ([300, 1, 129], [300, 2000, 1000], 64, 2, 8, 128, 4, [(2, 2), (2, 15)]),
    ([257, 64], [1300, 64], 16, 1, 7, 64, 8, [(0, k) for k in range(70)]),
    ([40], [30], 16, 2, 10, 128, 8, []),                      # ten rows have no position and see nothing
    ([5, 3], [5, 3], 16, 2, 128, 128, 4, []),
    ([1] * 70, list(range(0, 1400, 20)), 16, 2, 2, 128, 4, []),
]


@pytest.mark.parametrize("hint", [False, True])
@pytest.mark.parametrize("new,kv,page,Hkv,Hq,d,bits,absent", PAGED)
def test_paged_attention(new, kv, page, Hkv, Hq, d, bits, absent, hint):
    b = Batch(new, kv, page, seed=len(new), absent=absent)
    c = _filled_pool(b, Hkv, d, bits, seed=d + bits)
    pad = 2
    Q = _half(_rng(5), b.T + pad, Hq + 1, d)
    Qd = _dev(Q)[:, :Hq]
    out = torch.full((b.T + pad, Hq + 1, d), 7.0, dtype=torch.float16, device=DEV)
    o = q.qattn_paged_attention(Qd, c, *b.dev, max_new=max(new) if hint else None, out=out[:, 1:])
    torch.cuda.synchronize()
    assert q.qoq_device_error() == q.QOQ_OK
    assert bool((out[:, 0] == 7).all()) and bool((out[b.T:] == 7).all())
    _check_paged(b, c, Q[:, :Hq], Hkv, bits, d ** -0.5, o.cpu().numpy())
    if hint:                                                  # a bound that is too small is slower, not wrong
        o1 = q.qattn_paged_attention(Qd, c, *b.dev, max_new=1)
        _check_paged(b, c, Q[:, :Hq], Hkv, bits, d ** -0.5, o1.cpu().numpy())
        assert torch.equal(q.qattn_paged_attention(Qd, c, *b.dev, max_new=1)[:b.T].view(torch.int16), o1[:b.T].view(torch.int16))


@pytest.mark.parametrize("n", [1, 40, 300])
def test_paged_attention_scores_far_apart(n):
    """Scores of hundreds, rising and falling along the context: the running maximum moves, weights vanish, nothing
    overflows."""
    d, Hkv, Hq, bits = 128, 2, 8, 8
    b = Batch([n], [1500], 64, seed=1)
    c = _filled_pool(b, Hkv, d, bits, seed=9)
    for L in (c.k_par, c.v_par):
        x = L.float()
        x = x * torch.where(torch.arange(x.shape[0], device=DEV) % 3 == 0, 20.0, 0.01)[:, None, None, None]
        L.copy_(x.half())
    Q = _half(_rng(5), n, Hq, d) * np.float16(6)
    o = q.qattn_paged_attention(_dev(Q), c, *b.dev, scale=0.5)
    _check_paged(b, c, Q, Hkv, bits, 0.5, o.cpu().numpy())
    o = q.qattn_paged_attention(_dev(Q), c, *b.dev, scale=-0.5)
    _check_paged(b, c, Q, Hkv, bits, -0.5, o.cpu().numpy())


# ----------------------------------------------------- attention, prompts ----
PROMPTS = [  # lengths, Hkv, Hq, d
    ([1], 1, 1, 64), ([1, 2, 3], 2, 6, 128), ([128], 1, 4, 128), ([127, 129, 0, 1], 2, 8, 64), ([600, 31], 1, 7, 128),
    ([257, 513], 2, 2, 128), ([1025], 1, 1, 64), ([65, 64, 63], 1, 16, 128), ([300], 1, 64, 64),
]


def _check_prompt(X, lens, Hq, Hkv, got, scale, rows=None):
    """X [T, Hq + 2 Hkv, d]."""
    cu = np.concatenate([[0], np.cumsum(lens)])
    G = Hq // Hkv
    for s, n in enumerate(lens):
        e = slice(cu[s], cu[s + 1])
        at = np.arange(n) if rows is None else np.unique(np.clip(rows, 0, n - 1)) if n else np.arange(0)
        if not len(at):
            continue
        seen = np.arange(n)[None] <= at[:, None]
        for h in range(Hq):
            x = X[e].astype(np.float64)
            o, tol = ref.attend(x[at, h], x[:, Hq + h // G], x[:, Hq + Hkv + h // G], seen, scale)
            err = np.abs(got[e][at, h].astype(np.float64) - o)
            assert np.all(err <= tol), (s, h, float((err / tol).max()))


@pytest.mark.parametrize("lens,Hkv,Hq,d", PROMPTS)
def test_prompt_attention(lens, Hkv, Hq, d):
    T, pad = sum(lens), 4
    X = _half(_rng(T), T + pad, Hq + 2 * Hkv, d)
    Xd = _dev(X)
    Xd[T:] = float("nan")                                     # rows of no sequence: neither read into others nor written
    qd, kd, vd = Xd.split([Hq, Hkv, Hkv], 1)
    cu = _dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
    out = torch.full((T + pad, Hq, d), 7.0, dtype=torch.float16, device=DEV)
    o = q.qattn_prompt_attention(qd, kd, vd, cu, out=out)
    torch.cuda.synchronize()
    assert q.qoq_device_error() == q.QOQ_OK
    assert bool((out[T:] == 7).all())
    _check_prompt(X, lens, Hq, Hkv, o.cpu().numpy(), d ** -0.5)


def test_prompt_attention_isolates_sequences():
    """Infinities and NaN in one prompt reach no other, whichever comes first."""
    d, Hq, Hkv, lens = 128, 4, 2, [200, 90, 333]
    T = sum(lens)
    X = _half(_rng(3), T, Hq + 2 * Hkv, d)
    Xd = _dev(X)
    Xd[200:290, Hq:] = float("nan")
    Xd[205:215, Hq:] = float("inf")
    qd, kd, vd = Xd.split([Hq, Hkv, Hkv], 1)
    cu = _dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
    o = q.qattn_prompt_attention(qd, kd, vd, cu).cpu().numpy()
    X[200:290] = 0
    o[200:290] = 0
    _check_prompt(X, lens, Hq, Hkv, o, d ** -0.5)


def test_prompt_attention_scores_far_apart():
    d, Hq, Hkv, lens = 64, 2, 1, [700]
    X = _half(_rng(8), 700, Hq + 2 * Hkv, d)
    X[:, :Hq] *= np.float16(8)
    X[::5, Hq] *= np.float16(10)
    qd, kd, vd = _dev(X).split([Hq, Hkv, Hkv], 1)
    cu = _dev(np.array([0, 700], dtype=np.int32))
    for scale in (1.0, -1.0):
        _check_prompt(X, lens, Hq, Hkv, q.qattn_prompt_attention(qd, kd, vd, cu, scale=scale).cpu().numpy(), scale)
