"""The attention operators where their inputs are unusual: copied cache handles.  (The operators themselves:
test_gpu_attn.py, whose helpers are used here.)"""
import copy
import pickle

import pytest
import torch

import w4a8_integer_gemm_b200 as q
from test_gpu_attn import Batch, _dev, _filled_pool, _half, _rng

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
