"""spc_kv4_attn_mass with products q.K beyond fp32's range whose logits are ordinary
numbers, for requests on both sides of 32 rows of a KV head."""
import numpy as np
import pytest
import torch

from tests.chunk_cases import chunk, mass
from tests.paged_cases import DEV, SCALE, Cache, bf16, f64
from tests.test_gpu_kv4_mass import check, prev_of
from tests.test_gpu_kv4_mass_odd_rows import SIZES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_q,n_kv,n", SIZES + [(8, 2, 200)])
@pytest.mark.parametrize("power", [125, 110, -110, -128])
def test_products_of_any_size(n_q, n_kv, n, power):
    rng = np.random.default_rng(n_q + n + power + 200)
    c = Cache(rng, [700], n_kv, 16)
    x = f64(bf16(rng, n, n_q, 128)).clip(-3.9, 3.9)
    q = torch.from_numpy(x * 2.0 ** power).to(torch.bfloat16).to(DEV)
    scale = float(np.float32(SCALE * 2.0 ** -power))
    _, lse, _ = chunk(c, q, [n], scale=scale)
    assert torch.isfinite(lse).all()
    prev = prev_of(rng, c)
    got, _ = mass(c, q, [n], lse, prev, 1.0, scale=scale)
    check(c, q, [n], lse, prev, 1.0, got, scale=scale)
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("n_q,n_kv,n", SIZES)
@pytest.mark.parametrize("scale", [1e-40, 1.0, 1.5, 2e38])
def test_logits_of_zero_at_any_scale(n_q, n_kv, n, scale):
    rng = np.random.default_rng(n)
    c = Cache(rng, [300], n_kv, 16)
    c.rec[..., :64] &= 0xf0                                  # K: zero in even dims
    prev = prev_of(rng, c)
    for large in (0.0, 1e38, 1e-38):
        q = torch.zeros(n, n_q, 128, dtype=torch.bfloat16, device=DEV)
        q[..., 6] = large
        _, lse, _ = chunk(c, q, [n], scale=scale)
        got, _ = mass(c, q, [n], lse, prev, 1.0, scale=scale)
        check(c, q, [n], lse, prev, 1.0, got, scale=float(np.float32(scale)))
