"""spc_kv4_chunk_attn against the float64 oracle: every group size, lengths at
the tiles' edges, requests without tokens, rows that see nothing, blocks outside
the pool, values that are not finite, extreme logits, strides, workspaces,
streams and graphs."""
import numpy as np
import pytest
import torch

from sparse_kv_cache_retrieval_gb300 import binding as spc
from tests.chunk_cases import check_chunk, chunk, cu_of, workspace
from tests.paged_cases import DEV, SCALE, Cache, bf16, f64, i32

pytestmark = pytest.mark.gpu


def run(seed, lens, new, n_q, n_kv, bs, tail=0, amp=1.0, **kw):
    rng = np.random.default_rng(seed)
    c = Cache(rng, lens, n_kv, bs)
    q = bf16(rng, sum(new) + tail, n_q, 128, scale=amp).to(DEV)
    out, lse, _ = chunk(c, q, new, **kw)
    check_chunk(c, q, new, out, lse)


@pytest.mark.parametrize("n_q,n_kv", [(1, 1), (2, 1), (8, 2), (8, 1), (16, 1), (32, 1), (64, 1), (12, 3)])
@pytest.mark.parametrize("lens,new", [([1], [1]), ([300], [1]), ([300], [7]), ([129], [129]), ([200, 31, 640], [40, 31, 3])])
def test_groups(n_q, n_kv, lens, new):
    run(n_q * 7 + len(lens), lens, new, n_q, n_kv, 16)


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 128, 130, 257])
def test_lengths_at_the_edges_of_tiles(bs, n):
    run(bs + n, [n, n + 127, n + 128, n + 1000], [n, n, n, n], 4, 1, bs, tail=3)


@pytest.mark.parametrize("n_q,n_kv,lens,new", [
    (8, 2, [2500], [700]), (32, 8, [5000, 40, 900], [5, 40, 300]), (64, 1, [3500], [130]), (4, 4, [1100, 1100], [1, 700]),
    (8, 8, [20000], [2]), (64, 8, [9000, 1], [4, 1])])
def test_longer_contexts(n_q, n_kv, lens, new):
    run(sum(lens), lens, new, n_q, n_kv, 64, tail=2)


def test_requests_without_tokens_and_without_context():
    run(1, [50, 0, 70, 0, 33], [3, 0, 0, 0, 33], 8, 2, 16, tail=5)
    run(2, [0, 0], [0, 0], 8, 2, 16, tail=4)
    run(3, [5] * 64, [1] * 64, 8, 2, 16)


@pytest.mark.parametrize("n_q", [1, 4, 64])
def test_tokens_before_position_zero_see_nothing(n_q):
    run(4, [10, 0, 200], [17, 3, 260], n_q, 1, 16)


def test_blocks_outside_the_pool_are_left_out():
    rng = np.random.default_rng(5)
    c = Cache(rng, [700, 700, 700], 2, 16)
    c.table[0, [0, 7, 8, 9, 10, 11, 12, 13, 14, 15, 16, 43]] = -1
    c.table[1, :] = [c.num_blocks, 2 ** 31 - 1, -2 ** 31, -1] * 11
    c.table[2, 40:] = c.num_blocks
    new = [150, 20, 90]
    q = bf16(rng, 260, 8, 128).to(DEV)
    out, lse, _ = chunk(c, q, new)
    check_chunk(c, q, new, out, lse)
    assert np.all(f64(out[150:170]) == 0) and np.all(f64(lse[150:170]) == -np.inf)


def test_lengths_beyond_the_table_and_below_zero_are_cut():
    rng = np.random.default_rng(6)
    c = Cache(rng, [160, 160, 160], 1, 16)
    q = bf16(rng, 60, 4, 128).to(DEV)
    for lens in ([5000, -3, 2 ** 31 - 1], [160, -2 ** 31, 161]):
        out, lse, _ = chunk(c, q, [20, 20, 20], lens=i32(lens))
        check_chunk(c, q, [20, 20, 20], out, lse, lens=lens)


# ------------------------------------------------------------------ values that are not finite
@pytest.mark.parametrize("n_q,n_kv", [(4, 1), (16, 2), (64, 1)])
def test_nan_scales_reach_the_rows_that_see_them(n_q, n_kv):
    rng = np.random.default_rng(n_q)
    lens, new = [400, 150], [200, 150]
    c = Cache(rng, lens, n_kv, 16)

    def at(b, p):
        return c.rec[c.table[b, p // 16], 0, p % 16]
    at(0, 333)[136 + 3] = 0x7f                              # V: 16 values of a position among the new ones
    at(0, 390)[136 + 3] = 0xff
    at(0, 361)[136 + 7] = 0x7f
    at(1, 100)[128 + 1] = 0x7f                              # K: its whole logit
    q = bf16(rng, 350, n_q, 128).to(DEV)
    out, lse, _ = chunk(c, q, new)
    check_chunk(c, q, new, out, lse)
    o = f64(out)
    assert np.isnan(o[133:200, 0, 48:64]).all() and np.isfinite(o[:133, 0, 48:64]).all() and np.isfinite(o[:161, 0, 112:]).all()
    assert np.isnan(o[300:, 0]).all() and np.isfinite(o[200:300]).all()


def test_queries_that_are_not_finite():
    rng = np.random.default_rng(8)
    c = Cache(rng, [300, 40], 2, 16)
    q = bf16(rng, 60, 8, 128)
    q[3, 2, 5], q[4, 1, 0], q[9, 7, 127] = float("nan"), float("inf"), float("-inf")
    q[45, 0, 3], q[46, 1, 7] = float("nan"), float("inf")   # positions 25 and 26 of request 1
    q[12, 0, 3], q[13, 1, 7] = float("nan"), float("inf")   # rows 10 to 19 are before its position 0
    q = q.to(DEV)
    out, lse, _ = chunk(c, q, [10, 50])
    o, z = f64(out), f64(lse)
    odd = ((3, 2), (4, 1), (9, 7), (45, 0), (46, 1))
    for t, h in odd:
        assert np.isnan(o[t, h]).all() and np.isnan(z[t, h])
    q2 = q.clone()
    for t, h in odd + ((12, 0), (13, 1)):
        q2[t, h] = 0
    out2, lse2, _ = chunk(c, q2, [10, 50])
    check_chunk(c, q2, [10, 50], out2, lse2)
    same = np.ones((60, 8), bool)
    for t, h in odd:
        same[t, h] = False
    assert np.array_equal(o[same], f64(out2)[same]) and np.array_equal(z[same], f64(lse2)[same])
    # a shorter request: rows 10 to 51 see nothing, whatever their queries hold
    out, lse, _ = chunk(c, q, [10, 50], lens=i32([300, 8]))
    assert np.all(f64(out)[10:52] == 0) and np.all(f64(lse)[10:52] == -np.inf)


def test_rows_of_others_that_are_not_finite_do_not_reach_a_row():
    rng = np.random.default_rng(9)
    c = Cache(rng, [90, 90], 1, 16)
    q = bf16(rng, 64, 2, 128)
    q[30:] = float("nan")
    q = q.to(DEV)
    out, lse, _ = chunk(c, q, [30, 0], lens=i32([90, 0]))
    check_chunk(c, q, [30, 0], out, lse, lens=[90, 0])


# ------------------------------------------------------------------ logits of any size
@pytest.mark.parametrize("amp", [2.0 ** -120, 2.0 ** -40, 2.0 ** 20, 2.0 ** 100])
def test_queries_of_any_size(amp):
    rng = np.random.default_rng(10)
    c = Cache(rng, [500], 1, 32)
    q = (bf16(rng, 150, 4, 128).double() * amp).to(torch.bfloat16).to(DEV)
    out, lse, _ = chunk(c, q, [150], scale=SCALE / amp if amp < 2.0 ** 99 else 2.0 ** -100)
    check_chunk(c, q, [150], out, lse, scale=float(np.float32(SCALE / amp if amp < 2.0 ** 99 else 2.0 ** -100)))


def test_logits_beyond_any_exponential_pick_the_largest():
    # integer queries: the products are whole multiples of 2^-10, ties and all, so that the result is a
    # mean of V over the largest logits
    rng = np.random.default_rng(11)
    c = Cache(rng, [400], 1, 16)
    q = torch.from_numpy(rng.integers(-3, 4, (60, 4, 128)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    for scale in (1e6, 1e30):
        out, _, _ = chunk(c, q, [60], scale=scale)
        check_chunk(c, q, [60], out, None, scale=scale)


def test_zero_queries_average():
    rng = np.random.default_rng(12)
    c = Cache(rng, [777], 1, 16)
    q = torch.zeros(200, 4, 128, dtype=torch.bfloat16, device=DEV)
    for scale in (SCALE, 1e-38):
        out, lse, _ = chunk(c, q, [200], scale=scale)
        check_chunk(c, q, [200], out, lse, scale=scale)


def test_small_weights_beside_a_dominating_one():
    """A position that takes nearly all the weight and whose V is zero: the others' weights, 2^-26 of it, are the result."""
    rng = np.random.default_rng(13)
    c = Cache(rng, [4000], 1, 16)
    rec = c.rec[c.table[0, 0], 0, 0]
    rec[:64], rec[128:136] = 0x77, 0x50                      # K: 6 * 16 in every dim
    rec[64:128], rec[136:] = 0, 0
    q = bf16(rng, 200, 4, 128, scale=0.01)
    q += 18.0 * np.sqrt(128) / (96 * 128)                    # 18 nats above the others
    q = q.to(DEV)
    out, lse, _ = chunk(c, q, [200])
    check_chunk(c, q, [200], out, lse)


def test_rising_maxima():
    """Keys whose logits grow with the position, so that the running maximum rises in every block."""
    rng = np.random.default_rng(14)
    n = 1500
    c = Cache(rng, [n], 1, 16)
    grow = (np.arange(n) / n * 60.0)[:, None] * np.ones(128) / 128 + rng.standard_normal((n, 128)) * 0.05
    from oracle.paged_oracle import records
    rows = records(grow, rng.standard_normal((n, 128)))
    for p in range(n):
        c.rec[c.table[0, p // 16], 0, p % 16] = rows[p]
    q = torch.full((300, 4, 128), float(np.sqrt(128)), dtype=torch.bfloat16, device=DEV)
    out, lse, _ = chunk(c, q, [300])
    check_chunk(c, q, [300], out, lse)


# ------------------------------------------------------------------ how it is called
def test_rows_inside_fused_projections_and_no_lse():
    rng = np.random.default_rng(15)
    c = Cache(rng, [300, 300], 2, 32)
    fused = bf16(rng, 90, 8 + 4 + 3, 128).to(DEV)
    for q in (fused[:, :8], fused[:, 7:15]):
        out, lse, ws = chunk(c, q, [50, 33])
        check_chunk(c, q, [50, 33], out, lse)
        again, none, _ = chunk(c, q, [50, 33], lse=None, ws=ws)
        assert none is None and torch.equal(again, out)


def test_an_address_on_a_16_byte_boundary():
    rng = np.random.default_rng(16)
    c = Cache(rng, [300], 1, 16)
    q = bf16(rng, 41, 4, 128).to(DEV)

    def shifted(numel, dtype, off):
        t = torch.zeros(numel + 256, dtype=dtype, device=DEV)
        assert t.data_ptr() % 256 == 0
        return t[off:off + numel]
    q1 = shifted(q.numel(), torch.bfloat16, 8).view(41, 4, 128).copy_(q)
    out = shifted(q.numel(), torch.bfloat16, 24).view(41, 4, 128).fill_(7)
    lse = shifted(164, torch.float32, 1).view(41, 4).fill_(7)
    cache = shifted(c.rec.size, torch.uint8, 16).copy_(torch.from_numpy(c.rec).flatten().to(DEV))
    chunk(c, q1, [41], out=out, lse=lse, cache=cache)
    check_chunk(c, q, [41], out, lse)


def test_the_same_bits_every_time_and_on_a_used_workspace():
    rng = np.random.default_rng(17)
    ws = workspace(max(spc.spc_kv4_chunk_attn_workspace_size(*s, 128) for s in ((600, 4, 32, 8), (600, 4, 64, 1), (8, 1, 4, 1))))
    for lens, new, n_q, n_kv in (([4000, 100, 9, 1500], [300, 100, 9, 1], 32, 8), ([6000, 10, 0, 64], [2, 1, 0, 5], 64, 1),
                                 ([20000], [8], 4, 1)):
        c = Cache(rng, lens, n_kv, 32)
        q = bf16(rng, sum(new), n_q, 128).to(DEV)
        first = chunk(c, q, new)
        for _ in range(3):
            out, lse, _ = chunk(c, q, new, ws=ws)
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
        check_chunk(c, q, new, *first[:2])
        assert not ws[:4].any()


def test_streams_at_once():
    rng = np.random.default_rng(18)
    jobs = []
    for i in range(4):
        c = Cache(rng, [3000 - 500 * i, 200], 2, 32)
        q = bf16(rng, 90, 8, 128).to(DEV)
        jobs.append((c, q, torch.from_numpy(c.rec).to(DEV), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for c, q, cache, st in jobs:
        with torch.cuda.stream(st):
            for _ in range(3):
                r = chunk(c, q, [60, 30], cache=cache)
            got.append(r)
    torch.cuda.synchronize()
    for (c, q, _, _), r in zip(jobs, got):
        check_chunk(c, q, [60, 30], *r[:2])


def test_a_captured_call_follows_lengths_and_tables():
    rng = np.random.default_rng(19)
    c = Cache(rng, [900, 900], 2, 16)
    q = bf16(rng, 64, 8, 128).to(DEV)
    cache, table, lens, cu = torch.from_numpy(c.rec).to(DEV), i32(c.table), i32(c.lens), i32(cu_of([40, 24]))
    out, lse, ws = chunk(c, q, [40, 24], cache=cache, table=table, lens=lens, cu=cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chunk(c, q, None, out=out, lse=lse, ws=ws, cache=cache, table=table, lens=lens, cu=cu)
    for new_lens, new in (([900, 900], [40, 24]), ([64, 500], [1, 63]), ([900, 0], [64, 0]), ([129, 777], [0, 64])):
        lens.copy_(i32(new_lens))
        cu.copy_(i32(cu_of(new)))
        out.fill_(7)
        lse.fill_(7)
        graph.replay()
        graph.replay()
        check_chunk(c, q, new, out, lse, lens=new_lens)


def test_cu_seqlens_that_leave_the_rows_are_cut():
    rng = np.random.default_rng(20)
    c = Cache(rng, [300, 300], 1, 16)
    q = bf16(rng, 20, 4, 128).to(DEV)
    out, lse, _ = chunk(c, q, None, cu=i32([0, 12, 40]))     # rows 20 .. 39 are not there
    want, want_lse, _ = chunk(c, q, [12, 8], cu=i32([0, 12, 20]))
    assert torch.isfinite(out.float()).all() and torch.equal(out[:12], want[:12]) and torch.equal(lse[:12], want_lse[:12])


def test_a_pool_beyond_32_bits():
    """Records whose byte offsets pass 2^32."""
    rng = np.random.default_rng(21)
    c = Cache(rng, [700], 2, 128)
    n = (1 << 33) // (2 * 128 * 144) + 10                    # blocks: 8.6 GB
    cache = torch.zeros(n, 2, 128, 144, dtype=torch.uint8, device=DEV)
    far = [n - 1 - 3 * i for i in range(6)]
    for i, blk in enumerate(c.table[0]):
        cache[far[i]] = torch.from_numpy(c.rec[blk]).to(DEV)
    q = bf16(rng, 40, 8, 128).to(DEV)
    out = torch.full((40, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((40, 8), 7.0, device=DEV)
    ws = workspace(spc.spc_kv4_chunk_attn_workspace_size(40, 1, 8, 2, 128))
    spc.spc_kv4_chunk_attn(q, cache, i32([far]), i32([700]), i32([0, 40]), 40, 1, 8, 2, 128, n, 128, 6, SCALE, out, lse, ws)
    check_chunk(c, q, [40], out, lse)
