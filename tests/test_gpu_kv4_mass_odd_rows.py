"""spc_kv4_attn_mass where rows add nothing or hold what is not finite, for requests
on both sides of 32 rows of a KV head (two kernels): requests without new
tokens, rows whose log-sum-exp is not finite, K scales and queries that are NaN,
queries far from 1."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from tests.chunk_cases import chunk, mass
from tests.paged_cases import DEV, SCALE, Cache, bf16, f64
from tests.test_gpu_kv4_mass import check, prev_of

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
# rows of a KV head: 1, 12, 32 | 33, 36, 64
SIZES = [(1, 1, 1), (8, 2, 3), (8, 2, 8), (1, 1, 33), (8, 2, 9), (64, 1, 1)]


def nan_k(c, b, *positions):
    """K scales that are NaN in every head's record of these positions."""
    for p in positions:
        c.rec[c.table[b, p // c.bs], :, p % c.bs, 128 + p % 8] = 0x7f + 0x80 * (p & 1)


@pytest.mark.parametrize("n_q,n_kv", [(1, 1), (8, 2), (64, 1)])
@pytest.mark.parametrize("keep", [0.0, 1.0])
@pytest.mark.parametrize("new", [[0, 3], [0, 40], [0, 0]])
def test_requests_without_tokens_over_nan_records(n_q, n_kv, keep, new):
    rng = np.random.default_rng(n_q)
    c = Cache(rng, [300, 260], n_kv, 16)
    nan_k(c, 0, 0, 37, 64, 255, 299)
    q = bf16(rng, sum(new) + 1, n_q, 128).to(DEV)[:sum(new)]
    lse, prev = torch.full((sum(new), n_q), 5.0, device=DEV), prev_of(rng, c)
    got, _ = mass(c, q, new, lse, prev, keep)
    check(c, q, new, lse, prev, keep, got)
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("n_q,n_kv,n", SIZES)
def test_rows_that_add_nothing_over_nan_records(n_q, n_kv, n):
    rng = np.random.default_rng(n_q + n)
    c = Cache(rng, [300], n_kv, 16)
    nan_k(c, 0, 5, 130, 299)
    q = bf16(rng, n, n_q, 128).to(DEV)
    prev = prev_of(rng, c)
    lse = torch.full((n, n_q), -INF, device=DEV)
    got, _ = mass(c, q, [n], lse, prev, 1.0)
    check(c, q, [n], lse, prev, 1.0, got)
    assert torch.isfinite(got).all()
    # the last token adds nothing: position 299 is seen by no other one
    lse[:n - 1] = 5.0
    got, _ = mass(c, q, [n], lse, prev, 1.0)
    check(c, q, [n], lse, prev, 1.0, got)
    assert torch.isfinite(got[..., 299]).all() and bool(torch.isnan(got[..., 5]).all()) == (n > 1)


@pytest.mark.parametrize("n_q,n_kv,n", SIZES)
def test_log_sum_exps_that_are_not_finite(n_q, n_kv, n):
    rng = np.random.default_rng(2 * n_q + n)
    c = Cache(rng, [260], n_kv, 16)
    q = bf16(rng, n, n_q, 128).to(DEV)
    _, lse, _ = chunk(c, q, [n])
    prev = prev_of(rng, c)
    for odd in (-INF, INF):                                 # a weight of exp(-inf) is none either
        z = lse.clone()
        z[n // 2, n_q - 1] = z[n - 1, 0] = odd
        got, _ = mass(c, q, [n], z, prev, 0.5)
        check(c, q, [n], torch.where(z == INF, -INF, z), prev, 0.5, got)
    z = lse.clone()
    z[n // 2, 0] = NAN                                      # reaches what its row sees in its head, and no more
    got, _ = mass(c, q, [n], z, prev, 0.5)
    check(c, q, [n], z, prev, 0.5, got)
    seen = 260 - n + n // 2
    assert torch.isnan(got[0, 0, :seen + 1]).all() and torch.isfinite(got[0, 0, seen + 1:260]).all()


@pytest.mark.parametrize("n_q,n_kv,n", SIZES)
def test_nan_scales_and_queries(n_q, n_kv, n):
    rng = np.random.default_rng(3 * n_q + n)
    c = Cache(rng, [290], n_kv, 16)
    q = bf16(rng, n, n_q, 128).to(DEV)
    _, lse, _ = chunk(c, q, [n])
    prev = prev_of(rng, c)
    clean, _ = mass(c, q, [n], lse, prev, 1.0)
    nan_k(c, 0, 17, 288)
    got, _ = mass(c, q, [n], lse, prev, 1.0)
    check(c, q, [n], lse, prev, 1.0, got)
    for p in (17, 288):
        assert torch.isnan(got[..., p]).all()
        got[..., p] = clean[..., p]
    assert torch.equal(got, clean)
    x, z = q.clone(), lse.clone()
    x[n - 1, 0, 7] = NAN
    got, _ = mass(c, x, [n], lse, prev, 1.0)
    assert torch.isnan(got[0, 0, :290]).all()
    z[n - 1, 0] = -INF                                      # and none of it from a row that adds nothing
    got, _ = mass(c, x, [n], z, prev, 1.0)
    check(c, q, [n], z, prev, 1.0, got)


@pytest.mark.parametrize("n_q,n_kv,n", SIZES)
def test_infinite_queries(n_q, n_kv, n):
    """A weight is exp(inf), exp(-inf) or, where K is zero, NaN, as the formula has it."""
    rng = np.random.default_rng(5 * n_q + n)
    c = Cache(rng, [290], n_kv, 16)
    q = bf16(rng, n, n_q, 128).to(DEV)
    _, lse, _ = chunk(c, q, [n])
    prev, z = prev_of(rng, c), lse.clone()
    z[n - 1, 0] = -INF
    rest, _ = mass(c, q, [n], z, prev, 1.0)                 # without the last token's head 0
    k = np.array([P.values(c.rec[c.table[0, p // 16], 0, p % 16])[0][7] for p in range(290)])
    for odd in (INF, -INF):
        x = q.clone()
        x[n - 1, 0, 7] = odd
        got, _ = mass(c, x, [n], lse, prev, 1.0)
        s = torch.from_numpy(k * np.sign(odd)).to(DEV)
        want = rest.clone()
        want[0, 0, :290] = torch.where(s == 0, NAN, torch.where(s > 0, INF, rest[0, 0, :290]))
        assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))


@pytest.mark.parametrize("n_q,n_kv,n", SIZES)
@pytest.mark.parametrize("amp", [2.0 ** -100, 2.0 ** 30, 2.0 ** 100])
def test_queries_of_any_size(n_q, n_kv, n, amp):
    rng = np.random.default_rng(4 * n_q + n)
    c = Cache(rng, [300], n_kv, 16)
    q = (bf16(rng, n, n_q, 128).double() * amp).to(torch.bfloat16).to(DEV)
    scale = float(np.float32(SCALE / amp))
    _, lse, _ = chunk(c, q, [n], scale=scale)
    prev = prev_of(rng, c)
    got, _ = mass(c, q, [n], lse, prev, 1.0, scale=scale)
    check(c, q, [n], lse, prev, 1.0, got, scale=scale)
    assert np.isfinite(f64(got)).all()
