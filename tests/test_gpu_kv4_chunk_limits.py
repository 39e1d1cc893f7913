"""The calls over new tokens in the paged 4-bit cache at the ends of their limits:
1024 KV heads, 64 requests, the longest table, 2^24 rows."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from sparse_kv_cache_retrieval_gb300 import binding as spc
from tests.chunk_cases import check_chunk, chunk, chunk_tol, close, lse_tol, mass, workspace
from tests.paged_cases import DEV, SCALE, Cache, bf16, f64, i32
from tests.test_gpu_kv4_evict import Call, pool, sums
from tests.test_gpu_kv4_mass import check, prev_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [[1, 0], [5, 40]])
def test_the_most_kv_heads(new):
    rng = np.random.default_rng(0)
    c = Cache(rng, [70, 130], 1024, 16)
    q = bf16(rng, sum(new), 1024, 128).to(DEV)
    out, lse, _ = chunk(c, q, new)
    check_chunk(c, q, new, out, lse)
    prev = prev_of(rng, c)
    got, _ = mass(c, q, new, lse, prev, 1.0)
    check(c, q, new, lse, prev, 1.0, got)
    Call(pool(rng, [70, 130], 1024, 16), sums(rng, c), 64, 2, 16, in_place=True)().check()


def test_the_most_requests():
    rng = np.random.default_rng(1)
    lens = [int(n) for n in rng.integers(0, 90, 64)]
    new = [min(n, int(m)) for n, m in zip(lens, rng.integers(0, 20, 64))]
    new[5], lens[5] = 60, 80
    c = Cache(rng, lens, 2, 16)
    q = bf16(rng, sum(new), 8, 128).to(DEV)
    out, lse, _ = chunk(c, q, new)
    check_chunk(c, q, new, out, lse)
    prev = prev_of(rng, c)
    got, _ = mass(c, q, new, lse, prev, 0.5)
    check(c, q, new, lse, prev, 0.5, got)


@pytest.mark.parametrize("n", [1, 9])
def test_the_longest_table(n):
    rng = np.random.default_rng(2)
    L = 262144
    c = Cache(rng, [1600], 1, 16)                            # its hundred blocks over and over
    c.table = np.tile(c.table, (1, -(-L // 1600)))[:, :L // 16].copy()
    c.max_blocks, c.lens = L // 16, [L]
    q = bf16(rng, n, 4, 128).to(DEV)
    out, lse, _ = chunk(c, q, [n])
    check_chunk(c, q, [n], out, lse)
    prev = prev_of(rng, c)
    got, _ = mass(c, q, [n], lse, prev, 1.0)
    check(c, q, [n], lse, prev, 1.0, got)


def test_the_most_rows():
    """2^24 rows of which the last 300 see something."""
    rng = np.random.default_rng(3)
    T, L = 1 << 24, 300
    c = Cache(rng, [L], 1, 16)
    g = torch.Generator(device=DEV).manual_seed(3)
    q = torch.randn(T, 2, 128, generator=g, device=DEV, dtype=torch.bfloat16)
    out = torch.full((T, 2, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, 2), 7.0, device=DEV)
    ws = workspace(spc.spc_kv4_chunk_attn_workspace_size(T, 1, 2, 1, 128))
    table, cu, lens, cache = i32(c.table), i32([0, T]), i32([L]), torch.from_numpy(c.rec).to(DEV)
    chunk(c, q, None, out=out, lse=lse, ws=ws, cache=cache, table=table, cu=cu, lens=lens)
    assert not out[:T - L].any() and bool((lse[:T - L] == -torch.inf).all())
    want, mag, want_lse, err, vsum = P.chunk_attention(f64(q[T - L:]), c.rec, c.table, [L], [0, L], SCALE)
    close(out[T - L:], want, chunk_tol(want, mag, err, vsum), "out")
    close(lse[T - L:], want_lse, lse_tol(want_lse, err), "lse")
    prev = prev_of(rng, c)
    got, _ = mass(c, q, None, lse, prev, 1.0, cache=cache, table=table, cu=cu, lens=lens)
    check(c, q[T - L:], [L], lse[T - L:], prev, 1.0, got)
