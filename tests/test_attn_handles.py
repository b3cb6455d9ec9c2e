"""A cache handle's arguments are those of its own tensors, whatever way the handle or its tensors came about (no GPU)."""
import copy
import dataclasses
import pickle

import pytest
import torch

from w4a8_integer_gemm_b200 import PagedKVCache, paged_kv_cache


def _cache(bits=4, pages=5, page=16):
    c = paged_kv_cache(pages, 2, 64, bits, page, device="cpu")
    for t in (c.k_codes, c.v_codes, c.k_par, c.v_par):
        t.zero_()
    return c


def _addresses(c):
    return c.k_codes.data_ptr(), c.v_codes.data_ptr(), c.k_par.data_ptr(), c.v_par.data_ptr()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("way", [copy.deepcopy, copy.copy, lambda c: pickle.loads(pickle.dumps(c)),
                                 lambda c: dataclasses.replace(c, k_codes=c.k_codes.clone())])
def test_a_copy_works_on_its_own_tensors(way, bits):
    c = _cache(bits)
    before = c.args(-1)
    x = way(c)
    assert x.args(-1)[:4] == _addresses(x) and x.args(-1)[4:] == (bits, 16, 5, 2, 64)
    assert c.args(-1) == before == (*_addresses(c), bits, 16, 5, 2, 64)


def test_other_memory_under_the_same_tensors():
    c = _cache()
    c.args(-1)
    c.k_codes.data = c.k_codes.clone()
    assert c.args(-1)[:4] == _addresses(c)
    c.v_par.set_(torch.zeros_like(c.v_par))
    assert c.args(-1)[:4] == _addresses(c)
    c.v_codes.data = c.v_codes[:3].clone()                    # fewer pages than the others
    with pytest.raises(ValueError):
        c.args(-1)
    for t in (c.k_codes, c.k_par, c.v_par):
        t.data = t[:3].clone()
    assert c.args(-1) == (*_addresses(c), 4, 16, 3, 2, 64)
    c.k_codes.resize_(2, 2, 16, 32)                           # the same address, fewer pages
    with pytest.raises(ValueError):
        c.args(-1)


def test_checks_are_those_of_a_new_handle():
    c = _cache()
    with pytest.raises(ValueError):
        PagedKVCache(c.k_codes, c.v_codes[:4], c.k_par, c.v_par, 4)
    with pytest.raises(ValueError):
        c.args(0)                                             # another device
