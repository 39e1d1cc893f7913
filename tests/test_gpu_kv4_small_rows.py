"""Rows too small for the 4-bit cache's scales: stored as they are they become
zeros; stored as 2^n times themselves, with the attention's scale and output
divided by as much, they are kept like any others."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from sparse_kv_cache_retrieval_gb300 import binding as spc
from tests.paged_cases import DEV, SCALE, bf16, decode_tol, f64, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_q", [8, 64])
@pytest.mark.parametrize("amp", [1e-3, 2e-2, 1.0])
def test_rows_stored_as_a_power_of_two_times_themselves(n_q, amp):
    rng = np.random.default_rng(130)
    n, up = 700, 2.0 ** 9 if amp < 0.01 else 2.0 ** 5 if amp < 1 else 1.0
    k, v = bf16(rng, n, 1, 128, scale=amp), bf16(rng, n, 1, 128, scale=amp)
    q, scale = bf16(rng, 1, n_q, 128), SCALE / amp
    cache = torch.zeros(11, 1, 64, 144, dtype=torch.uint8, device=DEV)
    spc.spc_kv4_store((k * up).to(DEV), (v * up).to(DEV), i32(range(n)), cache, n, 1, 128, 11, 64)
    ws = torch.zeros(spc.spc_kv4_decode_attn_workspace_size(1, n_q, 1, 128, 11, 64, 0), dtype=torch.uint8, device=DEV)
    out = torch.zeros(1, n_q, 128, dtype=torch.bfloat16, device=DEV)
    spc.spc_kv4_decode_attn(q.to(DEV), cache, i32([range(11)]), i32([n]), None, 1, n_q, 1, 128, 11, 64, 11, 0, scale / up,
                            out, ws)
    got = f64(out) / up
    # the rows as the cache holds them
    kc, vc = (x / up for x in P.values(P.records(f64(k) * up, f64(v) * up)))
    want, mag = P.softmax_rows(f64(q)[0], kc[:, 0], vc[:, 0], scale)
    assert np.all(np.abs(got[0] - want) <= decode_tol(want, mag))
    # and how far that is from the rows themselves
    for a, b in ((kc, k), (vc, v)):
        err = np.linalg.norm(a - f64(b)) / np.linalg.norm(f64(b))
        assert 0.05 < err < 0.12


def test_where_rows_become_zeros():
    # largest magnitudes 6 * 2^-10 (the tie with zero) and the bf16 above it, in every group
    x = torch.zeros(2, 1, 128)
    x[0, 0, ::16], x[1, 0, ::16] = 6 * 2.0 ** -10, 6 * 2.0 ** -10 * (1 + 2.0 ** -7)
    x = x.to(torch.bfloat16).to(DEV)
    cache = torch.zeros(1, 1, 16, 144, dtype=torch.uint8, device=DEV)
    spc.spc_kv4_store(x, x, i32([0, 1]), cache, 2, 1, 128, 1, 16)
    k, v = torch.ones_like(x), torch.ones_like(x)
    spc.spc_kv4_load(cache, i32([0, 1]), k, v, 2, 1, 128, 1, 16)
    for y in (k, v):
        assert not y[0].any() and torch.all(y[1, 0, ::16] == 3 * 2.0 ** -9)
