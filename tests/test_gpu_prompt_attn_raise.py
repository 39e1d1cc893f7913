"""Prompt attention where the running maximum is raised in a block that every row
sees: the block's weights, already written against the old maximum, are written
again. Logits rise by far more than the margin from block to block, for every
head or for a single row of a warp, so that weights left from the first write
(up to infinity) would show."""
import numpy as np
import pytest
import torch

from sparse_kv_cache_retrieval_gb300 import binding as spc
import oracle.paged_oracle as P
from tests.paged_cases import DEV, bf16, f64, i32, prompt_tol

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_q,n_kv", [(1, 1), (8, 2), (64, 1)])
@pytest.mark.parametrize("step", [6.0, 20.0, 300.0])
@pytest.mark.parametrize("one_row", [False, True])
def test_raised_in_a_block_that_every_row_sees(n_q, n_kv, step, one_row):
    # logits about -1 .. 1, plus `step` (base 2) times the block's index for the rows that rise
    rng = np.random.default_rng(70 + n_q)
    n = 128 * 5 + 40
    u = np.sign(rng.standard_normal(128))
    q, k, v = (bf16(rng, n, m, 128, scale=a) for m, a in ((n_q, 1.0), (n_kv, 0.0625), (n_kv, 1.0)))
    k = (k.double() + torch.from_numpy(u * (np.arange(n)[:, None, None] // 128))).to(torch.bfloat16)
    rises = torch.ones(n, n_q, 1, dtype=torch.float64)
    if one_row:
        rises[:] = 0
        rises[5::32] = 1                                    # some tokens: one row of the warps that hold them
    along = (q.double() @ torch.from_numpy(u))[..., None] / 128 * torch.from_numpy(u)
    q = (q.double() - along + rises * torch.from_numpy(u)).to(torch.bfloat16)
    scale = step * np.log(2) / 128
    q, k, v = q.to(DEV), k.to(DEV), v.to(DEV)
    out = torch.full((n, n_q, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(spc.spc_prompt_attn_workspace_size(n, 1, n_q, n_kv, 128), dtype=torch.uint8, device=DEV)
    want, mag = P.prompt_attention(f64(q), f64(k), f64(v), [0, n], scale)
    # prompt_tol counts on small logits. Here a logit is a sum of 128 products whose magnitudes add up to A, each
    # addition off by at most 2^-24 A, and its product with the scale by as much again: 129 * 2^-24 A, which a
    # weight's numerator and the sum of the weights both have.
    A = scale * (np.abs(f64(q)).reshape(n, n_kv, -1, 128).max((1, 2)) @ np.abs(f64(k)).max(1).T).max()
    tol = prompt_tol(want, mag) + 2 * 129 * 2.0 ** -24 * A * mag
    for _ in range(3):
        spc.spc_prompt_attn(q, k, v, i32([0, n]), n, 1, n_q, n_kv, 128, scale, out, ws)
        got = f64(out)
        assert np.all(np.isfinite(got)) and np.all(np.abs(got - want) <= tol)
    assert int(ws[:4].view(torch.int32).item()) == 0
