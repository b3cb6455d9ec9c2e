"""What the workspace query answers (no GPU)."""
import itertools

import pytest


@pytest.fixture(scope="module")
def need():
    from w4a8_integer_gemm_b200 import build_lib
    build_lib.build()
    import w4a8_integer_gemm_b200 as q
    return q.qattn_paged_attention_workspace_bytes


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (32, 8, 128), (7, 1, 64), (64, 1, 128), (64, 2, 64), (4, 4, 64)])
def test_every_valid_shape_needs_some_and_smaller_calls_no_more(need, Hq, Hkv, d):
    sizes = {}
    for T, B, new in itertools.product((1, 4, 33, 300, 4096), (1, 3, 64), (1, 2, 8, 40, 4096)):
        sizes[T, B, new] = n = need(T, B, Hq, Hkv, d, 3, 64, new)
        assert n > 0 and n % 16 == 0
    for (T, B, new), n in sizes.items():
        for (T1, B1, new1), n1 in sizes.items():
            if T1 <= T and new1 <= new:
                assert n1 <= n, ((T1, B1, new1), (T, B, new))
    # neither the batch, the table nor the page size has a part in it
    assert len({need(33, B, Hq, Hkv, d, p, s, 8) for B in (1, 33) for p in (1, 100) for s in (16, 128)}) == 1


def test_work_that_cannot_be_counted_needs_none(need):
    assert need(1 << 21, 1, 1024, 16, 128, 1 << 17, 128, 1 << 21) == 0
