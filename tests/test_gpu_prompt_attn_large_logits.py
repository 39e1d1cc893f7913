"""Prompt attention with logits of any finite size: the largest take all, equal
ones share, in whichever block of keys they lie."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from sparse_kv_cache_retrieval_gb300 import binding as spc
from tests.paged_cases import DEV, check, f64, i32, prompt_tol

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_q,n_kv", [(2, 1), (8, 2), (64, 1)])
@pytest.mark.parametrize("top", [2.0 ** 10, 2.0 ** 24, 2.0 ** 27, 2.0 ** 30, 2.0 ** 33, 2.0 ** 60, 2.0 ** 120])
@pytest.mark.parametrize("lens", [[1, 60], [700, 130]])
def test_logits_of_any_finite_size(n_q, n_kv, top, lens):
    # logits i / 8 top for i in -8 .. 8, exact in bf16 and fp32, the largest often: it is seen from some row on and
    # shared by more and more of its equals. The odd heads see the negatives
    rng = np.random.default_rng(92)
    T, u = sum(lens), np.sign(rng.standard_normal(128))
    step = rng.integers(-7, 8, (T, n_kv, 1))
    step[rng.random((T, n_kv, 1)) < 0.02] = 8
    step[rng.random((T, n_kv, 1)) < 0.02] = -8
    k = torch.from_numpy(step * u).to(torch.bfloat16).to(DEV)
    sign = np.where(np.arange(n_q) % 2 == 0, 1, -1)[None, :, None]
    q = torch.from_numpy(np.broadcast_to(sign * u * 2.0, (T, n_q, 128)).copy()).to(torch.bfloat16).to(DEV)
    v = torch.from_numpy(rng.standard_normal((T, n_kv, 128))).to(torch.bfloat16).to(DEV)
    scale, cu = float(np.float32(top / (8 * 2 * 128))), [0, lens[0], T]
    out = torch.full((T, n_q, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(spc.spc_prompt_attn_workspace_size(T, 2, n_q, n_kv, 128), dtype=torch.uint8, device=DEV)
    spc.spc_prompt_attn(q, k, v, i32(cu), T, 2, n_q, n_kv, 128, scale, out, ws)
    want, mag = P.prompt_attention(f64(q), f64(k), f64(v), cu, scale)
    assert int(ws[:4].view(torch.int32).item()) == 0
    check(out, want, prompt_tol(want, mag))


@pytest.mark.parametrize("sign", [1, -1])
def test_scale_times_products_beyond_fp32(sign):
    # every logit passes fp32's range (all of them negative, too), their products with the queries do not
    rng = np.random.default_rng(93)
    n, u = 300, np.sign(rng.standard_normal(128))
    k = torch.from_numpy(rng.integers(1, 9, (n, 1, 1)) * u).to(torch.bfloat16).to(DEV)
    q = torch.from_numpy(np.broadcast_to(sign * u, (n, 4, 128)).copy()).to(torch.bfloat16).to(DEV)
    v = torch.from_numpy(rng.standard_normal((n, 1, 128))).to(torch.bfloat16).to(DEV)
    out = torch.full((n, 4, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(spc.spc_prompt_attn_workspace_size(n, 1, 4, 1, 128), dtype=torch.uint8, device=DEV)
    spc.spc_prompt_attn(q, k, v, i32([0, n]), n, 1, 4, 1, 128, 2e38, out, ws)
    want, mag = P.prompt_attention(f64(q), f64(k), f64(v), [0, n], 2e38)
    check(out, want, prompt_tol(want, mag))
