"""spc_kv4_store and spc_kv4_load refuse rows that overlap the cache, and a load
rows of k and v that overlap one another. Every call returns before anything is
launched; that rows which interleave pass is a GPU test's."""
import pytest

import __graft_entry__
from sparse_kv_cache_retrieval_gb300 import binding as B

K, FAR = 1 << 30, 1 << 40
ROW = 3 * 128                                               # elements of a row of 3 heads
POOL = 4 * 16 * 3 * 144


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return B.lib()


def load(lib, v, ks, vs, T=10, cache=FAR):
    return lib.spc_kv4_load(cache, 2 * FAR, K, v, ks, vs, T, 3, 128, 4, 16, None)


@pytest.mark.parametrize("v,ks,vs", [
    (K, ROW, ROW), (K + 16, ROW, ROW), (K - 16, ROW, ROW), (K + 18 * ROW, ROW, ROW),     # the same rows, or shifted
    (K + 2 * ROW - 16, 14 * 128, 14 * 128),                 # halves of a fused row that reach into one another
    (K + 2 * 14 * 128 - 16, 14 * 128, 14 * 128),            # the next row's start
    (K + 2 * ROW, ROW, 2 * ROW), (K + 2 * ROW, 14 * 128, 13 * 128)])                     # strides that bring them together
def test_a_load_refuses_rows_that_meet(lib, v, ks, vs):
    assert load(lib, v, ks, vs) == -1


@pytest.mark.parametrize("T", [1, 10])
def test_rows_refuse_the_cache(lib, T):
    span = ((T - 1) * 1024 + ROW) * 2
    for k, v in ((FAR, K), (K, FAR), (FAR - span + 16, K), (K, FAR - span + 16), (FAR + POOL - 16, K), (K, FAR + POOL - 16)):
        assert lib.spc_kv4_store(k, v, 1024, 1024, 2 * FAR, FAR, T, 3, 128, 4, 16, None) == -1
        assert lib.spc_kv4_load(FAR, 2 * FAR, k, v, 1024, 1024, T, 3, 128, 4, 16, None) == -1


def test_a_stride_beyond_any_memory_is_refused(lib):
    assert load(lib, 2 * K, (1 << 37) + 8, ROW) == -2 and load(lib, 2 * K, ROW, (1 << 37) + 8) == -2
