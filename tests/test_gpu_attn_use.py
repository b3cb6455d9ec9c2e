"""The attention operators as a program uses them: together with the W4A8 layers through a prompt and its decode steps,
captured and replayed, on other streams, with workspaces of its own, over pools beyond 4 GB and batches of thousands; and
what the Python calls refuse.  (Each operator alone: test_gpu_attn.py, whose helpers are used here.)"""
import numpy as np
import pytest
import torch

import w4a8_integer_gemm_b200 as q
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


def _bits(x):
    return x.view(torch.int16)


def _set(b, new, kv):
    """b with other lengths over the same pages."""
    import attn_ref as ref
    b.new, b.kv = list(new), list(kv)
    b.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    b.kv_len = np.array(kv, dtype=np.int32)
    b.T = int(b.cu[-1])
    b.seq, b.pos = ref.positions(b.cu, kv)
    b.dev = (b.dev[0], _dev(b.cu), _dev(b.kv_len))
    return b


@pytest.mark.parametrize("bits,d,Hq,Hkv,page", [(4, 64, 4, 2, 16), (8, 128, 6, 2, 32)])
def test_prompt_then_decode(bits, d, Hq, Hkv, page):
    """Two prompts through a projection, positions, prompt attention and the output projection; then a chunk for one and
    steps for both over the cache.  Every attention is checked against the 64-bit one of what it was given."""
    r = _rng(bits)
    width, hidden = (Hq + 2 * Hkv) * d, Hq * d
    qkv_layer = q.W4A8Linear(torch.from_numpy(r.standard_normal((width, hidden)).astype(np.float32) / hidden ** 0.5))
    o_layer = q.W4A8Linear(torch.from_numpy(r.standard_normal((hidden, hidden)).astype(np.float32) / hidden ** 0.5))
    rotary = q.Rotary(_dev(_freq(d)))
    b = Batch([0, 0], [190, 90], page, seed=bits)
    c = _poisoned_pool(b, Hkv, d, bits)
    kv, scale = [0, 0], d ** -0.5
    for new in ([37, 70], [100, 1], [1, 1], [0, 1], [1, 1]):
        kv = [k + n for k, n in zip(kv, new)]
        _set(b, new, kv)
        x = _dev(_half(r, b.T, hidden))
        heads = qkv_layer(x).view(b.T, Hq + 2 * Hkv, d)
        qh, kh, vh = heads.split([Hq, Hkv, Hkv], 1)
        if kv == new:                                         # whole prompts
            turned = heads.clone()
            q.qattn_rotary(turned[:, :Hq + Hkv], _dev(b.pos.astype(np.int32)), rotary, out=turned[:, :Hq + Hkv])
            q.qattn_cache_append(kh, vh, c, *b.dev, rotary=rotary)
            o = q.qattn_prompt_attention(*turned.split([Hq, Hkv, Hkv], 1), b.dev[1])
            _check_prompt(turned.cpu().numpy(), new, Hq, Hkv, o.cpu().numpy(), scale)
            qh = turned[:, :Hq]
        else:
            qh = q.qattn_cache_append(kh, vh, c, *b.dev, rotary=rotary, q=qh)
            o = q.qattn_paged_attention(qh, c, *b.dev, max_new=max(new))
        over = q.qattn_paged_attention(qh, c, *b.dev)         # (a prompt's rows may be had from the cache as well)
        _check_paged(b, c, qh.cpu().numpy(), Hkv, bits, scale, over.cpu().numpy())
        if kv != new:
            _check_paged(b, c, qh.cpu().numpy(), Hkv, bits, scale, o.cpu().numpy())
        y = o_layer(o.reshape(b.T, hidden))
        assert y.shape == (b.T, hidden) and bool(torch.isfinite(y).all())


@pytest.mark.parametrize("n,Hq,Hkv,d,bits", [(1, 8, 2, 128, 4), (60, 8, 2, 64, 8), (3, 16, 1, 128, 8)])
def test_captured_steps(n, Hq, Hkv, d, bits):
    """Appends and attentions captured once and replayed with other rows and lengths, from two graphs at the same time on
    two streams, each with its own workspace: the bits of the same calls made one after another."""
    steps, B = 3, 3
    rotary = q.Rotary(_dev(_freq(d)), True)

    def sides():
        b = Batch([n] * B, [500 + steps * n, steps * n, 900 + steps * n], 32, seed=n)
        c = _filled_pool(b, Hkv, d, bits, seed=3)
        rows = [_dev(_half(_rng(50 + i), b.T, Hq + 2 * Hkv, d)) for i in range(steps)]
        lens = [_dev(np.array([500, 0, 900], dtype=np.int32) + (i + 1) * n) for i in range(steps)]
        return b, c, rows, lens

    def step(b, c, x, kl, out, ws=None):
        qh, kh, vh = x.split([Hq, Hkv, Hkv], 1)
        t = q.qattn_cache_append(kh, vh, c, b.dev[0], b.dev[1], kl, rotary=rotary, q=qh)
        return q.qattn_paged_attention(t, c, b.dev[0], b.dev[1], kl, max_new=n, out=out, workspace=ws)

    b, c, rows, lens = sides()
    want = [step(b, c, rows[i], lens[i], None).clone() for i in range(steps)]
    graphs, kept_alive = [], []
    for _ in range(2):
        b, c, rows, lens = sides()
        x, kl, out = rows[0].clone(), lens[0].clone(), torch.empty(b.T, Hq, d, dtype=torch.float16, device=DEV)
        need = q.qattn_paged_attention_workspace_bytes(b.T, B, Hq, Hkv, d, b.table.shape[1], 32, n)
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
        kept = [t.clone() for t in (c.k_codes, c.v_codes, c.k_par, c.v_par)]
        step(b, c, x, kl, out, ws)                            # (what is set up on a first call)
        for t, s in zip((c.k_codes, c.v_codes, c.k_par, c.v_par), kept):
            t.copy_(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(b, c, x, kl, out, ws)
        graphs.append((g, torch.cuda.Stream(), x, kl, out, rows, lens))
        kept_alive.append((b, c, ws))                         # (a graph does not hold what it works on)
    torch.cuda.synchronize()
    for i in range(steps):
        for g, s, x, kl, out, rows, lens in graphs:
            with torch.cuda.stream(s):
                x.copy_(rows[i])
                kl.copy_(lens[i])
                g.replay()
        torch.cuda.synchronize()
        for *_, out, _, _ in graphs:
            assert torch.equal(_bits(out), _bits(want[i])), i


@pytest.mark.parametrize("raw", [False, True])
def test_stream_argument(raw):
    """Calls on a stream that is not the current one, by object or handle, behind work queued there."""
    d, Hq, Hkv, bits = 128, 4, 2, 4
    b = Batch([40, 1], [300, 77], 64, seed=2)
    x = _dev(_half(_rng(1), b.T, Hq + 2 * Hkv, d))
    rotary = q.Rotary(_dev(_freq(d)))

    def run(x, c, **kw):
        qh, kh, vh = x.split([Hq, Hkv, Hkv], 1)
        t = q.qattn_cache_append(kh, vh, c, *b.dev, rotary=rotary, q=qh, **kw)
        K, V = q.qattn_cache_read(c, *b.dev, b.T, **kw)
        p = q.qattn_prompt_attention(t, kh, vh, b.dev[1], **kw)
        z = q.qattn_rotary(t, torch.arange(b.T, device=DEV, dtype=torch.int32) if not kw else at, rotary, **kw)
        return t, K, V, p, z, q.qattn_paged_attention(t, c, *b.dev, **kw), q.qattn_paged_attention(t, c, *b.dev, max_new=1, **kw)

    at = torch.arange(b.T, device=DEV, dtype=torch.int32)
    want = [t.clone() for t in run(x, _filled_pool(b, Hkv, d, bits, 4))]
    c = _filled_pool(b, Hkv, d, bits, 4)
    late = torch.zeros_like(x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)                         # about 10 ms
        late.copy_(x)
    got = run(late, c, stream=s.cuda_stream if raw else s)
    s.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(_bits(g), _bits(w))


@pytest.mark.parametrize("new,kv,Hq,Hkv,d", [([1, 1], [5000, 9], 8, 2, 128), ([200, 3], [900, 3], 4, 4, 64),
                                             ([300, 1, 20], [3000, 64, 400], 7, 1, 128)])
def test_workspace(new, kv, Hq, Hkv, d):
    """Any contents will do, nothing behind it is touched, one that is too small is refused; the same bits each time."""
    b = Batch(new, kv, 64, seed=1)
    c = _filled_pool(b, Hkv, d, 4, seed=2)
    Q = _dev(_half(_rng(1), b.T, Hq, d))
    for most in (b.T, max(new)):
        need = q.qattn_paged_attention_workspace_bytes(b.T, len(new), Hq, Hkv, d, b.table.shape[1], 64, most)
        want = None
        for fill in (0xFF, 0x00, 0x7B):
            ws = torch.full((need + 4096,), fill, dtype=torch.uint8, device=DEV)
            o = q.qattn_paged_attention(Q, c, *b.dev, max_new=most, workspace=ws[:need])
            assert bool((ws[need:] == fill).all())
            want = o if want is None else want
            assert torch.equal(_bits(o), _bits(want))
        with pytest.raises(q.QoQError):
            q.qattn_paged_attention(Q, c, *b.dev, max_new=most, workspace=ws[:need - 16])
        for _ in range(3):
            assert torch.equal(_bits(q.qattn_paged_attention(Q, c, *b.dev, max_new=most, workspace=ws)), _bits(want))


def test_shared_pages():
    """Sequences that share the pages of a common beginning read the same tokens."""
    d, Hq, Hkv, bits = 128, 8, 2, 4
    b = Batch([1, 70, 1], [700, 800, 700], 64, seed=1)
    c = _filled_pool(b, Hkv, d, bits, seed=2)
    b.table[1, :6] = b.table[0, :6]
    b.table[2] = b.table[0]
    b.dev = (_dev(b.table), *b.dev[1:])
    Q = _half(_rng(1), b.T, Hq, d)
    Q[-1] = Q[0]
    o = q.qattn_paged_attention(_dev(Q), c, *b.dev).cpu().numpy()
    _check_paged(b, c, Q, Hkv, bits, d ** -0.5, o)
    assert np.array_equal(o[0], o[-1])


@pytest.mark.parametrize("bits", [4, 8])
def test_pool_beyond_32_bits(bits):
    """Pages whose offsets pass 2^32 bytes: the bits of the same tokens in a small pool."""
    d, Hq, Hkv, page = 128, 8, 8, 128
    b = Batch([1, 90], [1000, 700], page, seed=3)
    small = _filled_pool(b, Hkv, d, bits, seed=4)
    pages = (1 << 32) // (Hkv * page * d * bits // 8) + b.pages + 5
    big = q.paged_kv_cache(pages, Hkv, d, bits, page)
    assert big.k_codes.numel() > 1 << 32
    far = pages - b.pages
    for x, y in ((big.k_codes, small.k_codes), (big.v_codes, small.v_codes), (big.k_par, small.k_par), (big.v_par, small.v_par)):
        x[far:] = y
    table = _dev(np.where(b.table >= 0, b.table + far, -1).astype(np.int32))
    X = _dev(_half(_rng(2), b.T, Hq + 2 * Hkv, d))
    qh, kh, vh = X.split([Hq, Hkv, Hkv], 1)
    rotary = q.Rotary(_dev(_freq(d)))
    out = []
    for c, t in ((small, b.dev[0]), (big, table)):
        turned = q.qattn_cache_append(kh, vh, c, t, *b.dev[1:], rotary=rotary, q=qh)
        out.append((turned, q.qattn_paged_attention(turned, c, t, *b.dev[1:]), *q.qattn_cache_read(c, t, *b.dev[1:], b.T)))
    for x, y in zip(*out):
        assert torch.equal(_bits(x), _bits(y))
    assert torch.equal(big.k_codes[far:], small.k_codes) and torch.equal(big.v_codes[far:], small.v_codes)


def test_many_sequences():
    """Thousands of sequences, most of them with no new token, lengths 0 to 40."""
    d, Hq, Hkv, bits, page, B = 64, 4, 2, 8, 16, 6000
    r = _rng(7)
    new = np.where(r.random(B) < 0.7, 0, r.integers(1, 4, B)).tolist()
    new[17], new[-1] = 150, 30
    kv = [n + int(r.integers(0, 40)) for n in new]
    b = Batch(new, kv, page, seed=5)
    x = _half(r, b.T, Hq + 2 * Hkv, d)
    qh, kh, vh = _dev(x).split([Hq, Hkv, Hkv], 1)
    c = _poisoned_pool(b, Hkv, d, bits)
    old = Batch(kv, kv, page, seed=5)                         # the same pages, every token new
    everything = _half(r, old.T, 2 * Hkv, d)
    q.qattn_cache_append(*_dev(everything).split([Hkv, Hkv], 1), c, b.dev[0], old.dev[1], b.dev[2])
    q.qattn_cache_append(kh, vh, c, *b.dev)
    o = q.qattn_paged_attention(qh, c, *b.dev, max_new=150).cpu().numpy()
    pick = np.concatenate([np.arange(0, b.T, 61), np.arange(b.cu[17], b.cu[18]), np.arange(b.cu[-2], b.T)])
    _check_paged(b, c, x[:, :Hq], Hkv, bits, d ** -0.5, o, rows=pick)
    lens = [n for n in new]
    p = q.qattn_prompt_attention(qh, kh, vh, b.dev[1]).cpu().numpy()
    some = [s for s in range(B) if new[s]][::97] + [17, B - 1]
    for s in some:
        e = slice(b.cu[s], b.cu[s + 1])
        _check_prompt(x[e], [lens[s]], Hq, Hkv, p[e], d ** -0.5)


@pytest.mark.parametrize("G,d,bits", [(4, 128, 4), (3, 128, 8), (1, 64, 8), (16, 64, 4)])
def test_many_work_items(G, d, bits):
    """Hundreds of short chunks and prompts: every SM gets many row tiles one after another."""
    Hkv, B = 8, 170
    r = _rng(G)
    new = [int(n) for n in r.integers(1, 2 + 200 // G, B)]
    kv = [n + int(k) for n, k in zip(new, r.integers(0, 150, B))]
    b = Batch(new, kv, 32, seed=2)
    c = _filled_pool(b, Hkv, d, bits, seed=3)
    x = _half(r, b.T, (G + 2) * Hkv, d)
    qh, kh, vh = _dev(x).split([G * Hkv, Hkv, Hkv], 1)
    o = q.qattn_paged_attention(qh, c, *b.dev)
    p = q.qattn_prompt_attention(qh, kh, vh, b.dev[1]).cpu().numpy()
    torch.cuda.synchronize()
    assert q.qoq_device_error() == q.QOQ_OK
    some = list(range(0, B, 23))
    rows = np.concatenate([np.arange(b.cu[s], b.cu[s + 1]) for s in some])
    _check_paged(b, c, x[:, :G * Hkv], Hkv, bits, d ** -0.5, o.cpu().numpy(), rows=rows)
    for s in some:
        e = slice(b.cu[s], b.cu[s + 1])
        _check_prompt(x[e], [new[s]], G * Hkv, Hkv, p[e], d ** -0.5)
    # the others against themselves: a sequence's outputs do not depend on its place in the batch
    turn = np.arange(B)[::-1]
    back = Batch([new[i] for i in turn], [kv[i] for i in turn], 32, seed=2)
    order = np.concatenate([np.arange(b.cu[i], b.cu[i + 1]) for i in turn])
    again = q.qattn_prompt_attention(*(y[_dev(order)] for y in (qh, kh, vh)), back.dev[1]).cpu().numpy()
    assert np.array_equal(again.view(np.int16), p[order].view(np.int16))


@pytest.mark.parametrize("extra", [8, 24])
def test_strides_of_eight(extra):
    """Rows whose distance is a multiple of 16 bytes and no more, in every argument."""
    d, Hq, Hkv, lens = 64, 3, 1, [150, 9]
    T = sum(lens)
    r = _rng(extra)
    X = _half(r, T, Hq + 2 * Hkv, d)

    def wide(x):
        w = torch.full((T, x.shape[1] * d + extra), 7.0, dtype=torch.float16, device=DEV)
        return w, w.as_strided((T, x.shape[1], d), (w.shape[1], d, 1), 8)

    parts = []
    for a, e in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)):
        y = wide(X[:, a:e])[1]
        y.copy_(_dev(X[:, a:e]))
        parts.append(y)
    w, out = wide(X[:, :Hq])
    cu = _dev(np.array([0, lens[0], T], dtype=np.int32))
    q.qattn_prompt_attention(*parts, cu, out=out)
    _check_prompt(X, lens, Hq, Hkv, out.cpu().numpy(), d ** -0.5)
    assert bool((w[:, :8] == 7).all()) and bool((w[:, 8 + Hq * d:] == 7).all())
    b = Batch(lens, lens, 16, seed=1)
    c = _poisoned_pool(b, Hkv, d, 8)
    w, turned = wide(X[:, :Hq])
    q.qattn_cache_append(parts[1], parts[2], c, *b.dev, rotary=q.Rotary(_dev(_freq(32))), q=parts[0], q_out=turned)
    assert bool((w[:, :8] == 7).all()) and bool((w[:, 8 + Hq * d:] == 7).all())
    for most in (max(lens), 1):
        w, out = wide(X[:, :Hq])
        q.qattn_paged_attention(turned, c, *b.dev, max_new=most, out=out)
        _check_paged(b, c, turned.cpu().numpy(), Hkv, 8, d ** -0.5, out.cpu().numpy())
        assert bool((w[:, :8] == 7).all()) and bool((w[:, 8 + Hq * d:] == 7).all())


@pytest.mark.parametrize("G,Hkv,new,d,bits", [(17, 2, [1, 1], 64, 4), (32, 1, [1, 1, 1], 128, 8), (33, 1, [1, 1], 128, 4), (20, 1, [2, 1], 64, 8),
                                             (11, 1, [3, 2, 1], 128, 4), (8, 2, [4, 5, 1], 64, 4)])
def test_rows_either_kernel_takes(G, Hkv, new, d, bits):
    """Numbers of rows on both sides of every choice of kernel: 8, 16, 32 and more per KV head."""
    b = Batch(new, [300 + 40 * i for i in range(len(new))], 16, seed=G)
    c = _filled_pool(b, Hkv, d, bits, seed=1)
    Q = _half(_rng(G), b.T, G * Hkv, d)
    for most in (None, max(new), 1):
        o = q.qattn_paged_attention(_dev(Q), c, *b.dev, max_new=most)
        _check_paged(b, c, Q, Hkv, bits, d ** -0.5, o.cpu().numpy())


@pytest.mark.parametrize("new", [[1, 2], [90, 1]])
def test_rows_before_the_first_sequence(new):
    """cu begins after rows of no sequence: they are neither read nor written, by any call."""
    d, Hq, Hkv, bits, lead, tail = 64, 4, 2, 4, 3, 2
    b = Batch(new, [n + 20 for n in new], 16, seed=1)
    c = _filled_pool(b, Hkv, d, bits, seed=2)
    x = _half(_rng(3), lead + b.T + tail, Hq + 2 * Hkv, d)
    xd = _dev(x)
    inner = xd[lead:lead + b.T].clone()
    xd[:lead] = float("nan")
    xd[lead + b.T:] = float("nan")
    cu = b.dev[1] + lead
    rotary = q.Rotary(_dev(_freq(d)))

    def run(y, cu, c):
        qh, kh, vh = y.split([Hq, Hkv, Hkv], 1)
        outs = [torch.full((y.shape[0], h, d), 7.0, dtype=torch.float16, device=DEV) for h in (Hq, Hkv, Hkv, Hq, Hq)]
        q.qattn_cache_append(kh, vh, c, b.dev[0], cu, b.dev[2], rotary=rotary, q=qh, q_out=outs[0])
        q.qattn_cache_read(c, b.dev[0], cu, b.dev[2], y.shape[0], K=outs[1], V=outs[2])
        q.qattn_paged_attention(outs[0], c, b.dev[0], cu, b.dev[2], out=outs[3])
        q.qattn_prompt_attention(qh, kh, vh, cu, out=outs[4])
        return outs

    c2 = _filled_pool(b, Hkv, d, bits, seed=2)
    for got, want in zip(run(xd, cu, c), run(inner, b.dev[1], c2)):
        assert bool((got[:lead] == 7).all()) and bool((got[lead + b.T:] == 7).all())
        assert torch.equal(_bits(got[lead:lead + b.T]), _bits(want))


@pytest.mark.parametrize("new", [[1, 1], [40, 3], [200, 150]])
def test_lengths_beyond_the_table(new):
    """Contexts longer than their row of the table: what the table does not reach is not there."""
    d, Hq, Hkv, bits, page = 128, 4, 2, 8, 16
    b = Batch(new, [500, 333], page, seed=1)
    c = _filled_pool(b, Hkv, d, bits, seed=2)
    b.table = np.ascontiguousarray(b.table[:, :13])           # 208 tokens, the middle of a key tile
    b.dev = (_dev(b.table), *b.dev[1:])
    x = _half(_rng(3), b.T, Hq + 2 * Hkv, d)
    qh, kh, vh = _dev(x).split([Hq, Hkv, Hkv], 1)
    q.qattn_cache_append(kh, vh, c, *b.dev)
    for most in (max(new), 1):
        o = q.qattn_paged_attention(qh, c, *b.dev, max_new=most)
        _check_paged(b, c, x[:, :Hq], Hkv, bits, d ** -0.5, o.cpu().numpy())
    K, V = q.qattn_cache_read(c, *b.dev, b.T)
    gone = _dev(b.pos >= 208)
    assert bool((K[gone] == 0).all()) and bool((V[gone] == 0).all())


def test_append_in_place():
    d, Hq, Hkv = 128, 5, 1
    b = Batch([3, 70], [30, 70], 32, seed=1)
    x = _dev(_half(_rng(3), b.T, Hq + 2 * Hkv, d))
    rotary = q.Rotary(_dev(_freq(64)), True, 1.1)
    pools = [_poisoned_pool(b, Hkv, d, 4) for _ in range(2)]
    qh, kh, vh = x.split([Hq, Hkv, Hkv], 1)
    want = q.qattn_cache_append(kh, vh, pools[0], *b.dev, rotary=rotary, q=qh)
    assert q.qattn_cache_append(kh, vh, pools[1], *b.dev, rotary=rotary, q=qh, q_out=qh) is qh
    assert torch.equal(_bits(qh), _bits(want))
    for s, t in zip((pools[0].k_codes, pools[0].v_codes, pools[0].k_par, pools[0].v_par),
                    (pools[1].k_codes, pools[1].v_codes, pools[1].k_par, pools[1].v_par)):
        assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))


def test_negative_lengths_and_empty_contexts():
    """Lengths of zero and below: every row sees nothing and is zero, whichever kernel has it."""
    d, Hq, Hkv = 64, 4, 1
    b = Batch([1, 40, 2, 3], [5, 60, 9, 300], 16, seed=1)
    c = _filled_pool(b, Hkv, d, 4, seed=2)
    kl = _dev(np.array([0, -5, -(1 << 31), 300], dtype=np.int32))
    Q = _half(_rng(1), b.T, Hq, d)
    b.kv = [0, -5, -5, 300]
    for most in (40, 1):
        o = q.qattn_paged_attention(_dev(Q), c, b.dev[0], b.dev[1], kl, max_new=most).cpu().numpy()
        assert not o[:43].any()
        one = Batch([3], [300], 16)
        one.table, one.pages, one.cu, one.pos = b.table[3:], b.pages, one.cu, b.pos[43:]
        _check_paged(one, c, Q[43:], Hkv, 4, d ** -0.5, o[43:])


def test_empty_calls():
    d, Hq, Hkv = 64, 4, 2
    c = q.paged_kv_cache(3, Hkv, d)
    i32 = dict(dtype=torch.int32, device=DEV)
    x = torch.empty(0, Hq + 2 * Hkv, d, dtype=torch.float16, device=DEV)
    qh, kh, vh = x.split([Hq, Hkv, Hkv], 1)
    table, cu, kl = torch.zeros(2, 1, **i32), torch.zeros(3, **i32), torch.zeros(2, **i32)
    assert q.qattn_paged_attention(qh, c, table, cu, kl).shape == (0, Hq, d)
    assert q.qattn_prompt_attention(qh, kh, vh, cu).shape == (0, Hq, d)
    assert q.qattn_cache_append(kh, vh, c, table, cu, kl) is None
    assert q.qattn_cache_read(c, table, cu, kl, 0)[0].shape == (0, Hkv, d)
    # no sequence at all: rows stay as they are
    y = torch.full((4, Hq, d), 7.0, dtype=torch.float16, device=DEV)
    q.qattn_paged_attention(y, c, torch.zeros(0, 1, **i32), cu[:1], kl[:0], out=y)
    assert bool((y == 7).all())
    # sequences, and no row of theirs
    q.qattn_paged_attention(torch.zeros_like(y), c, table, cu, kl, out=y)
    q.qattn_prompt_attention(y, y[:, :2].contiguous(), y[:, :2].contiguous(), cu, out=y)
    assert bool((y == 7).all())


def _good():
    d, Hq, Hkv, T = 64, 4, 2, 6
    i32 = dict(dtype=torch.int32, device=DEV)
    x = torch.zeros(T, Hq + 2 * Hkv, d, dtype=torch.float16, device=DEV)
    qh, kh, vh = x.split([Hq, Hkv, Hkv], 1)
    return dict(q=qh, k=kh, v=vh, c=q.paged_kv_cache(4, Hkv, d, 4, 16), table=torch.arange(4, **i32).view(2, 2),
                cu=torch.tensor([0, 2, 6], **i32), kl=torch.tensor([2, 9], **i32), rot=q.Rotary(_dev(_freq(d))),
                pos=torch.arange(T, **i32), out=None, ws=None, scale=None, max_new=None)


CALLS = {
    "rotary": lambda a: q.qattn_rotary(a["q"], a["pos"], a["rot"], out=a["out"]),
    "append": lambda a: q.qattn_cache_append(a["k"], a["v"], a["c"], a["table"], a["cu"], a["kl"], rotary=a["rot"], q=a["q"], q_out=a["out"]),
    "paged": lambda a: q.qattn_paged_attention(a["q"], a["c"], a["table"], a["cu"], a["kl"], scale=a["scale"], max_new=a["max_new"],
                                               out=a["out"], workspace=a["ws"]),
    "prompt": lambda a: q.qattn_prompt_attention(a["q"], a["k"], a["v"], a["cu"], scale=a["scale"], out=a["out"]),
}
REFUSED = [
    ("rotary append paged prompt", "q", lambda x: x.float()),
    ("rotary append paged prompt", "q", lambda x: x.cpu()),
    ("rotary append paged prompt", "q", lambda x: x[0]),
    ("rotary append paged prompt", "q", lambda x: x.transpose(0, 1)),
    ("append paged prompt", "q", lambda x: x[..., :32]),
    ("append prompt", "q", lambda x: x[:5]),
    ("append prompt", "q", lambda x: x[:, :3]),
    ("append prompt", "k", lambda x: x[:, :1]),
    ("append prompt", "v", lambda x: x.bfloat16()),
    ("rotary append paged prompt", "out", lambda x: torch.empty(6, 3, 64, dtype=torch.float16, device=DEV)),
    ("rotary append paged prompt", "out", lambda x: torch.empty(6, 4, 64, dtype=torch.float32, device=DEV)),
    ("append paged prompt", "cu", lambda x: x.long()),
    ("append paged prompt", "cu", lambda x: x.cpu()),
    ("append paged", "cu", lambda x: x[:2]),
    ("append paged", "kl", lambda x: x[:1]),
    ("append paged", "kl", lambda x: x.view(2, 1)),
    ("append paged", "table", lambda x: x.t()),
    ("append paged", "table", lambda x: x[:1]),
    ("append paged", "table", lambda x: x.float()),
    ("append paged", "c", lambda x: q.paged_kv_cache(4, 2, 128, 4, 16)),
    ("append", "c", lambda x: q.paged_kv_cache(4, 1, 64, 4, 16)),
    ("append paged", "c", lambda x: q.paged_kv_cache(4, 2, 64, 4, 16, device="cpu")),
    ("append", "rot", lambda x: None),
    ("rotary append", "rot", lambda x: q.Rotary(x.freq.float())),
    ("rotary append", "rot", lambda x: q.Rotary(x.freq[:5])),
    ("rotary append", "rot", lambda x: q.Rotary(torch.cat([x.freq, x.freq]))),
    ("rotary append", "rot", lambda x: q.Rotary(x.freq, False, float("inf"))),
    ("rotary", "pos", lambda x: x[:3]),
    ("rotary", "pos", lambda x: x.long()),
    ("paged prompt", "scale", lambda x: float("nan")),
    ("paged", "ws", lambda x: torch.empty(64, dtype=torch.uint8, device=DEV)),
    ("paged", "ws", lambda x: torch.empty(1 << 24, dtype=torch.uint8)),
    ("paged", "c", lambda x: q.paged_kv_cache(0, 2, 64, 4, 16)),
]


@pytest.mark.parametrize("call,name,change", [(c, n, f) for cs, n, f in REFUSED for c in cs.split()])
def test_refusals(call, name, change):
    a = _good()
    CALLS[call](a)
    a[name] = change(a[name])
    with pytest.raises((ValueError, q.QoQError)):
        CALLS[call](a)
    torch.cuda.synchronize()


def test_cache_refusals():
    ok = q.paged_kv_cache(2, 2, 64, 4, 16)
    for bits, d, page, pages, Hkv in ((3, 64, 16, 2, 2), (4, 96, 16, 2, 2), (4, 64, 24, 2, 2), (4, 64, 16, -1, 2), (4, 64, 16, 2, 0)):
        with pytest.raises(ValueError):
            q.paged_kv_cache(pages, Hkv, d, bits, page)
    for change in (dict(k_codes=ok.k_codes.half()), dict(v_codes=ok.v_codes[:1]), dict(k_par=ok.k_par.float()), dict(bits=5),
                   dict(v_par=ok.v_par[..., :1]), dict(k_codes=ok.k_codes.transpose(0, 1)), dict(v_codes=ok.v_codes.cpu())):
        with pytest.raises(ValueError):
            q.PagedKVCache(**{**dict(k_codes=ok.k_codes, v_codes=ok.v_codes, k_par=ok.k_par, v_par=ok.v_par, bits=4), **change})
