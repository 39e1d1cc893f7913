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


# ------------------------------------------------------------------ outputs and workspaces of the other calls
def spread(sizes):
    """Addresses far apart for buffers of these sizes."""
    return [(i + 1) << 36 for i in range(len(sizes))]


def refused_where_one_overlaps(call, addresses, sizes, outputs):
    """Each output moved so that its last 16-byte unit is another buffer's first, or the reverse."""
    for i in outputs:
        for j, (a, n) in enumerate(zip(addresses, sizes)):
            if j == i:
                continue
            low = a - (-(-sizes[i] // 256) - 1) * 256
            for at in (low, a, a + (n - 1) // 256 * 256):
                moved = list(addresses)
                moved[i] = at
                assert call(*moved) == -1, (i, j, at - a)


def test_block_map_refuses_outputs_that_overlap(lib):
    n, mb, num, slots = 3, 20, 90, 500
    sizes = [n * 4, n * 4, n * mb * 4, num * 4, 4, 4, (n + 1) * 4, slots * 4, 4]
    refused_where_one_overlaps(lambda *p: lib.spc_block_map(*p, n, mb, 16, num, slots, None), spread(sizes), sizes,
                               (2, 3, 5, 6, 7, 8))


@pytest.mark.parametrize("budget", [0, 100])
def test_decode_attn_refuses_outputs_that_overlap(lib, budget):
    n, n_q, n_kv, num, mb = 3, 64, 2, 50, 9
    ws = B.spc_kv4_decode_attn_workspace_size(n, n_q, n_kv, 128, mb, 16, budget)
    sizes = [n * n_q * 256, num * n_kv * 16 * 144, n * mb * 4, n * 4, n * n_q * 256, ws] + [n * n_kv * budget * 4] * (budget > 0)

    def call(q, cache, table, ln, out, w, sel=None):
        return lib.spc_kv4_decode_attn(q, cache, table, ln, sel, n, n_q, n_kv, 128, num, 16, mb, budget, 0.1, out, w, ws, None)

    refused_where_one_overlaps(call, spread(sizes), sizes, (4, 5))


def test_prompt_attn_refuses_outputs_that_overlap(lib):
    T, n_q, n_kv, stride = 70, 8, 2, 12 * 128
    sizes = [((T - 1) * stride + n * 128) * 2 for n in (n_q, n_kv, n_kv)] + [12, T * n_q * 256, 256]

    def call(q, k, v, cu, out, w):
        return lib.spc_prompt_attn(q, k, v, cu, T, 2, n_q, n_kv, 128, stride, stride, stride, 0.1, out, w, 256, None)

    refused_where_one_overlaps(call, spread(sizes), sizes, (4, 5))
