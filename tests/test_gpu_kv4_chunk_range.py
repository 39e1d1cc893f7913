"""spc_kv4_chunk_attn with products q.K beyond fp32's range whose logits are ordinary
numbers, and with rows close to bf16's least."""
import numpy as np
import pytest
import torch

from tests.chunk_cases import check_chunk, chunk
from tests.paged_cases import DEV, SCALE, Cache, bf16, f64

pytestmark = pytest.mark.gpu

# at most a tile's rows a request; two tiles; items that are cut, the one way and the other
CASES = [(4, 1, [500], [20]), (8, 2, [700, 300], [150, 60]), (4, 1, [20000], [3]), (8, 2, [4000], [200])]


@pytest.mark.parametrize("n_q,n_kv,lens,new", CASES)
@pytest.mark.parametrize("power", [125, 110, -110, -128])
def test_products_of_any_size(n_q, n_kv, lens, new, power):
    rng = np.random.default_rng(sum(lens) + power)
    c = Cache(rng, lens, n_kv, 16)
    x = f64(bf16(rng, sum(new), n_q, 128)).clip(-3.9, 3.9)
    q = torch.from_numpy(x * 2.0 ** power).to(torch.bfloat16).to(DEV)
    scale = float(np.float32(SCALE * 2.0 ** -power))
    assert torch.isfinite(q).all()
    out, lse, _ = chunk(c, q, new, scale=scale)
    check_chunk(c, q, new, out, lse, scale=scale)
    assert torch.isfinite(lse).all()


@pytest.mark.parametrize("n_q,n_kv,lens,new", CASES)
@pytest.mark.parametrize("scale", [1.0, 1e30, 2e38])
def test_queries_of_zeros_and_the_largest_scales(n_q, n_kv, lens, new, scale):
    """lse is ln of the positions, also where the queries' factor times the scale passes fp32."""
    rng = np.random.default_rng(1)
    c = Cache(rng, lens, n_kv, 16)
    q = torch.zeros(sum(new), n_q, 128, dtype=torch.bfloat16, device=DEV)
    out, lse, _ = chunk(c, q, new, scale=scale)
    check_chunk(c, q, new, out, lse, scale=scale)
    # a large query against records whose K is zero where it is not
    c.rec[..., :64] &= 0xf0                                  # even dims
    q[..., 6] = 1e38
    out, lse, _ = chunk(c, q, new, scale=scale)
    check_chunk(c, q, new, out, lse, scale=scale)
