"""spc_kv4_chunk_attn where a request has at most a tile's rows on average (the
kernel with one Q tile), and next to that limit: the inputs of
test_gpu_kv4_chunk.py that are harder than random ones, requests with several
tiles among ones with a token, contexts that many CTAs share; and
spc_kv4_attn_mass over many requests of either kind at once."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from sparse_kv_cache_retrieval_gb300 import binding as spc
from tests.chunk_cases import check_chunk, chunk, close, cu_of, mass, mass_tol, workspace
from tests.paged_cases import DEV, SCALE, Cache, bf16, f64

pytestmark = pytest.mark.gpu


def run(seed, lens, new, n_q, n_kv, bs, tail=0):
    rng = np.random.default_rng(seed)
    c = Cache(rng, lens, n_kv, bs)
    q = bf16(rng, sum(new) + tail, n_q, 128).to(DEV)
    out, lse, _ = chunk(c, q, new)
    check_chunk(c, q, new, out, lse)


@pytest.mark.parametrize("G", [1, 4, 16, 64])
@pytest.mark.parametrize("more", [0, 1])
def test_rows_on_both_sides_of_a_tile_a_request(G, more):
    n = 128 // G
    run(G + more, [700, 300], [n + more, n], G, 1, 16)


@pytest.mark.parametrize("n_q,n_kv", [(8, 1), (16, 2), (64, 1)])
def test_several_tiles_among_single_tokens(n_q, n_kv):
    # B = 16: one request has 400 rows or more, the others a token's
    lens = [900] + [37 * b % 400 + 1 for b in range(15)]
    new = [50 if n_q < 64 else 7] + [1] * 15
    run(n_q, lens, new, n_q, n_kv, 16, tail=3)


@pytest.mark.parametrize("n_q,n_kv,n", [(8, 1, 3), (64, 8, 4), (4, 4, 30), (8, 1, 40)])
def test_a_context_that_many_ctas_share(n_q, n_kv, n):
    run(n, [20000], [n], n_q, n_kv, 64)


@pytest.mark.parametrize("n", [17, 33, 90, 150])
def test_pairs_and_a_single_tile_of_requests_that_are_cut(n):
    run(n, [3000, 5000], [n, n // 2], 16, 2, 32)


def test_blocks_outside_the_pool():
    rng = np.random.default_rng(5)
    for bs in (16, 64):
        c = Cache(rng, [700, 700, 700], 2, bs)
        c.table[0, [0, 2, 3, 8, 10]] = -1
        c.table[1, :] = c.num_blocks
        c.table[2, 9:] = 2 ** 31 - 1
        new = [30, 20, 9]
        q = bf16(rng, 59, 8, 128).to(DEV)
        out, lse, _ = chunk(c, q, new)
        check_chunk(c, q, new, out, lse)


def test_nan_scales_reach_the_rows_that_see_them():
    rng = np.random.default_rng(6)
    lens, new = [400, 900], [20, 12]
    c = Cache(rng, lens, 1, 16)

    def at(b, p):
        return c.rec[c.table[b, p // 16], 0, p % 16]
    at(0, 390)[136 + 3] = 0x7f                              # V, a position among the new ones
    at(0, 395)[136 + 7] = 0xff
    at(1, 100)[136] = 0x7f                                  # V, one that all rows see, in an even block
    at(1, 130)[136 + 1] = 0x7f                              # and in an odd one
    at(1, 893)[128 + 1] = 0x7f                              # K: its whole logit
    q = bf16(rng, 32, 8, 128).to(DEV)
    out, lse, _ = chunk(c, q, new)
    check_chunk(c, q, new, out, lse)
    o = f64(out)
    assert np.isnan(o[10:20, 0, 48:64]).all() and np.isfinite(o[:10, 0, 48:64]).all() and np.isfinite(o[:15, 0, 112:]).all()
    assert np.isnan(o[20:, 0, :32]).all() and np.isnan(o[25:]).all() and np.isfinite(o[20:25, 0, 32:]).all()


def test_queries_that_are_not_finite():
    rng = np.random.default_rng(8)
    c = Cache(rng, [300, 700], 2, 16)
    q = bf16(rng, 22, 8, 128)
    odd = ((3, 2), (4, 1), (9, 7), (15, 0))
    for t, h in odd:
        q[t, h, 5 * t] = float("nan") if h & 1 else float("inf")
    q = q.to(DEV)
    out, lse, _ = chunk(c, q, [10, 12])
    q2 = q.clone()
    for t, h in odd:
        q2[t, h] = 0
        assert torch.isnan(out[t, h]).all() and torch.isnan(lse[t, h])
    out2, lse2, _ = chunk(c, q2, [10, 12])
    check_chunk(c, q2, [10, 12], out2, lse2)
    same = np.ones((22, 8), bool)
    for t, h in odd:
        same[t, h] = False
    assert np.array_equal(f64(out)[same], f64(out2)[same]) and np.array_equal(f64(lse)[same], f64(lse2)[same])


@pytest.mark.parametrize("amp", [2.0 ** -120, 2.0 ** 100])
def test_queries_of_any_size(amp):
    rng = np.random.default_rng(10)
    c = Cache(rng, [1500], 1, 32)
    q = (bf16(rng, 30, 4, 128).double() * amp).to(torch.bfloat16).to(DEV)
    scale = SCALE / amp if amp < 2.0 ** 99 else 2.0 ** -100
    out, lse, _ = chunk(c, q, [30], scale=scale)
    check_chunk(c, q, [30], out, lse, scale=float(np.float32(scale)))


def test_logits_beyond_any_exponential_pick_the_largest():
    rng = np.random.default_rng(11)
    c = Cache(rng, [900], 1, 16)
    q = torch.from_numpy(rng.integers(-3, 4, (20, 4, 128)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    for scale in (1e6, 1e30):
        out, _, _ = chunk(c, q, [20], scale=scale)
        check_chunk(c, q, [20], out, None, scale=scale)


@pytest.mark.parametrize("n", [8, 30, 80])
def test_small_weights_beside_a_dominating_one(n):
    """A position that takes nearly all the weight and whose V is zero, in a piece, a block and a half of its own."""
    rng = np.random.default_rng(13)
    c = Cache(rng, [6000], 1, 16)
    for p in (0, 2500):
        rec = c.rec[c.table[0, p // 16], 0, p % 16]
        rec[:64], rec[128:136] = 0x77, 0x50                  # K: 6 * 16 in every dim
        rec[64:128], rec[136:] = 0, 0
    q = bf16(rng, n, 4, 128, scale=0.01)
    q += 18.0 * np.sqrt(128) / (96 * 128)                    # 18 nats above the others
    q = q.to(DEV)
    out, lse, _ = chunk(c, q, [n])
    check_chunk(c, q, [n], out, lse)


@pytest.mark.parametrize("n", [6, 30, 300])
@pytest.mark.parametrize("sign", [1, -1])
def test_maxima_that_rise_or_fall_with_the_position(n, sign):
    rng = np.random.default_rng(14)
    m = 2500
    c = Cache(rng, [m], 1, 16)
    grow = sign * (np.arange(m) / m * 80.0)[:, None] * np.ones(128) / 128 + rng.standard_normal((m, 128)) * 0.05
    rows = P.records(grow, rng.standard_normal((m, 128)))
    for p in range(m):
        c.rec[c.table[0, p // 16], 0, p % 16] = rows[p]
    q = torch.full((n, 4, 128), float(np.sqrt(128)), dtype=torch.bfloat16, device=DEV)
    out, lse, _ = chunk(c, q, [n])
    check_chunk(c, q, [n], out, lse)


def test_shapes_take_turns_on_one_workspace():
    """Few new tokens, many, none that are cut, many again: the same bits as on a workspace of their own."""
    rng = np.random.default_rng(15)
    shapes = [([9000], [4], 8, 1), ([5000, 300], [400, 20], 8, 1), ([50], [1], 8, 1), ([3000], [200], 64, 1), ([700] * 9, [2] * 9, 16, 2)]
    calls = []
    for lens, new, n_q, n_kv in shapes:
        c = Cache(rng, lens, n_kv, 32)
        q = bf16(rng, sum(new), n_q, 128).to(DEV)
        out, lse, _ = chunk(c, q, new)
        check_chunk(c, q, new, out, lse)
        calls.append((c, q, new, out, lse))
    ws = workspace(max(spc.spc_kv4_chunk_attn_workspace_size(q.shape[0], len(c.lens), q.shape[1], c.n_kv, 128) for c, q, _, _, _ in calls))
    for i in (0, 1, 2, 1, 3, 0, 4, 1, 0):
        c, q, new, want, want_lse = calls[i]
        out, lse, _ = chunk(c, q, new, ws=ws)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("n_q,n_kv", [(8, 2), (16, 1)])
def test_weight_of_requests_of_either_kind(n_q, n_kv):
    """64 requests: a step's token, none, drafts, windows and chunks, over gaps in their tables."""
    rng = np.random.default_rng(16)
    lens = [int(n) for n in rng.integers(1, 1500, 64)]
    new = [min(n, (1, 0, 4, 64, 200, 1, 33, 2)[b % 8]) for b, n in enumerate(lens)]
    c = Cache(rng, lens, n_kv, 16)
    for b in range(0, 64, 3):
        c.table[b, rng.integers(0, c.max_blocks, 30)] = -1
    q = bf16(rng, sum(new) + 2, n_q, 128).to(DEV)
    _, lse, _ = chunk(c, q, new)
    prev = torch.from_numpy(rng.random((64, n_kv, c.max_blocks * 16)).astype(np.float32)).to(DEV)
    first = None
    for _ in range(3):
        got, _ = mass(c, q, new, lse, prev, 0.5)
        first = got if first is None else first
        assert torch.equal(got, first)
    want, rel = P.attn_mass(f64(q), c.rec, c.table, c.lens, cu_of(new), f64(lse), f64(prev), 0.5, got.shape[2], SCALE)
    for b, n in enumerate(lens):
        close(got[b, :, :n], want[b, :, :n], mass_tol(want, rel)[b, :, :n], f"mass of request {b}")


def test_weight_of_a_context_that_many_ctas_share():
    rng = np.random.default_rng(17)
    c = Cache(rng, [30000, 12000], 1, 64)
    for n_q, new in ((4, [3, 64]), (16, [100, 2]), (64, [5, 300])):
        q = bf16(rng, sum(new), n_q, 128).to(DEV)
        _, lse, _ = chunk(c, q, new)
        got, _ = mass(c, q, new, lse, None, 0.0)
        prev = np.zeros(got.shape)
        want, rel = P.attn_mass(f64(q), c.rec, c.table, c.lens, cu_of(new), f64(lse), prev, 0.0, got.shape[2], SCALE)
        for b, n in enumerate(c.lens):
            close(got[b, :, :n], want[b, :, :n], mass_tol(want, rel)[b, :, :n], f"mass of request {b}")
