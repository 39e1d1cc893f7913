"""spc_kv4_load into rows of k and v that interleave without meeting: halves of
fused rows in either order, and v in every other row's gap."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from sparse_kv_cache_retrieval_gb300 import binding as spc
from tests.paged_cases import DEV, bf16, f64, i32

pytestmark = pytest.mark.gpu
T, N = 40, 3


@pytest.mark.parametrize("k_at,v_at,k_step,v_step", [(0, 3, 1, 1), (3, 0, 1, 1), (11, 2, 1, 1), (0, 7, 1, 2), (9, 4, 2, 1)])
def test_rows_that_interleave(k_at, v_at, k_step, v_step):
    # a buffer of 2 T rows of 14 heads; k and v take every first or second of them, at heads of their own
    rng = np.random.default_rng(94)
    rows = bf16(rng, T, N, 128).to(DEV)
    slots = i32(rng.permutation(64)[:T])
    cache = torch.zeros(4, N, 16, 144, dtype=torch.uint8, device=DEV)
    spc.spc_kv4_store(rows, rows.flip(0).contiguous(), slots, cache, T, N, 128, 4, 16)
    y = torch.full((2 * T, 14, 128), 9.0, dtype=torch.bfloat16, device=DEV)
    k, v = y[::k_step, k_at:k_at + N][:T], y[::v_step, v_at:v_at + N][:T]
    spc.spc_kv4_load(cache, slots, k, v, T, N, 128, 4, 16)
    want = P.values(P.records(f64(rows), f64(rows.flip(0))))
    assert np.array_equal(f64(k), want[0]) and np.array_equal(f64(v), want[1])
    assert int((y != 9).any(-1).sum()) == 2 * T * N          # and nothing else is written


def test_rows_that_meet_are_refused():
    y = torch.zeros(T, 14, 128, dtype=torch.bfloat16, device=DEV)
    cache = torch.zeros(4, N, 16, 144, dtype=torch.uint8, device=DEV)
    for a, b in ((0, 2), (5, 5), (4, 3)):
        with pytest.raises(spc.SpcError) as e:
            spc.spc_kv4_load(cache, i32(range(T)), y[:, a:a + N], y[:, b:b + N], T, N, 128, 4, 16)
        assert e.value.status == -1
    assert not y.any()
