"""The attention operators where their inputs are unusual: copied cache handles, row tiles without
keys between others.  (The operators themselves:
test_gpu_attn.py, whose helpers are used here.)"""
import copy
import pickle

import numpy as np
import pytest
import torch

import w4a8_integer_gemm_b200 as q
from test_gpu_attn import Batch, _check_paged, _check_prompt, _dev, _filled_pool, _half, _rng

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
