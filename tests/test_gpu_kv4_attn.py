"""spc_kv4_decode_attn against the float64 oracle on the same records, codes and
scales included, with the tolerance derived in paged_cases."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from sparse_kv_cache_retrieval_gb300 import binding as spc
from tests.paged_cases import DEV, SCALE, Cache, bf16, check, decode, decode_tol, f64, i32

pytestmark = pytest.mark.gpu


def run(c, q, selected=None, scale=SCALE, **kw):
    sel = None if selected is None else i32(selected)
    got, ws = decode(c, q.to(DEV), sel, scale=scale, **kw)
    want, mag = P.decode_attention(f64(q), c.rec, c.table, c.lens, selected, scale)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32).item()) == 0
    check(got, want, decode_tol(want, mag))
    return got, want


@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [17], [63], [64], [65], [127], [129], [1000], [4097],
                                  [0, 1, 0, 300], [5, 700, 64, 128, 1, 1999, 0, 33]])
def test_lengths(lens):
    rng = np.random.default_rng(sum(lens) + len(lens))
    c = Cache(rng, lens, 2, 64)
    got, _ = run(c, bf16(rng, len(lens), 16, 128))
    for b, n in enumerate(lens):
        if n == 0:
            assert torch.all(got[b] == 0)


@pytest.mark.parametrize("n_q,n_kv", [(1, 1), (2, 2), (2, 1), (8, 2), (16, 2), (16, 1), (32, 1), (64, 1), (128, 2),
                                      (8, 8), (40, 5)])
def test_head_layouts(n_q, n_kv):
    rng = np.random.default_rng(n_q * 7 + n_kv)
    run(Cache(rng, [700, 33], n_kv, 32), bf16(rng, 2, n_q, 128))


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("n_kv", [1, 8])
def test_block_sizes(bs, n_kv):
    rng = np.random.default_rng(bs)
    run(Cache(rng, [777, bs, bs + 1, 3], n_kv, bs), bf16(rng, 4, 8 * n_kv, 128))


@pytest.mark.parametrize("lens,n_q,n_kv", [([40000], 8, 1), ([30000, 5, 9000], 16, 2), ([20011], 64, 1)])
def test_long_contexts_split_over_the_gpu(lens, n_q, n_kv):
    rng = np.random.default_rng(lens[0])
    run(Cache(rng, lens, n_kv, 64), bf16(rng, len(lens), n_q, 128, scale=2.0))


def test_full_batch():
    rng = np.random.default_rng(64)
    lens = [int(x) for x in rng.integers(0, 500, 64)]
    run(Cache(rng, lens, 4, 16), bf16(rng, 64, 16, 128))


def test_peaked_and_late_maxima():
    # logits that grow along the context, so the running maximum moves all the time, and a last position that takes all
    rng = np.random.default_rng(9)
    c = Cache(rng, [3000], 1, 64)
    q = bf16(rng, 1, 8, 128)
    k = np.zeros((1, 3000, 128))
    d = f64(q)[0].sum(0)
    k[0] = d / np.linalg.norm(d) * np.linspace(-20, 60, 3000)[:, None] + rng.standard_normal((3000, 128))
    rec = P.records(k, rng.standard_normal((1, 3000, 128)))
    for i, blk in enumerate(c.table[0]):
        m = min(64, 3000 - i * 64)
        c.rec[blk, :, :m] = rec[:, i * 64:i * 64 + m]
    run(c, q, scale=0.5)


@pytest.mark.parametrize("amp", [1e-3, 300.0])
def test_cache_values_at_the_ends_of_the_scales(amp):
    rng = np.random.default_rng(10)
    run(Cache(rng, [500], 2, 64, amp=amp), bf16(rng, 1, 8, 128), scale=SCALE if amp < 1 else SCALE / amp)


@pytest.mark.parametrize("qscale", [1e-30, 1e-6, 1e4, 1e30])
def test_queries_of_any_size(qscale):
    rng = np.random.default_rng(11)
    q = bf16(rng, 2, 16, 128)
    q[0, 3] *= 2.0 ** -12                                   # heads of one group differ by far
    q = (q.float() * qscale).to(torch.bfloat16)
    run(Cache(rng, [400, 90], 2, 64), q, scale=SCALE / qscale)


@pytest.mark.parametrize("n_q", [8, 64])
def test_addresses_on_16_byte_boundaries(n_q):
    rng = np.random.default_rng(23)
    c = Cache(rng, [333, 0], 1, 16)
    q = bf16(rng, 2 * n_q * 128 + 8).to(DEV)[8:].view(2, n_q, 128)
    cache = torch.zeros(c.rec.size + 16, dtype=torch.uint8, device=DEV)[16:]
    cache.copy_(torch.from_numpy(c.rec.reshape(-1)))
    out = torch.full((2 * n_q * 128 + 8,), 7.0, dtype=torch.bfloat16, device=DEV)[8:].view(2, n_q, 128)
    run(c, q, out=out, cache=cache)
    run(c, q, selection(rng, c.lens, 1, 50), out=out, cache=cache)


def test_zero_queries_average_the_values():
    rng = np.random.default_rng(12)
    c = Cache(rng, [100], 1, 16)
    run(c, torch.zeros(1, 4, 128, dtype=torch.bfloat16))


@pytest.mark.parametrize("n_q", [8, 32])
@pytest.mark.parametrize("scale", [1e-9, 1e-37])
def test_zero_and_tiny_queries_at_a_small_scale(n_q, scale):
    # every logit vanishes, the masked ones must not: 100 of 128 positions, and 37 selected ones of a tile
    rng = np.random.default_rng(22)
    c = Cache(rng, [100], 1, 16)
    q = torch.zeros(1, n_q, 128, dtype=torch.bfloat16)
    q[0, 1:] = (bf16(rng, n_q - 1, 128).float() * 1e-36).to(torch.bfloat16)
    run(c, q, scale=scale)
    run(c, q, selection(rng, [100], 1, 37), scale=scale)


def test_what_lies_behind_the_context_does_not_count():
    # every byte behind the lengths is 0xff: codes -6 under NaN scales (Cache fills it so); longer tables too
    rng = np.random.default_rng(13)
    c = Cache(rng, [70, 1, 0], 2, 64, max_blocks=9)
    c.table[c.table < 0] = c.num_blocks - 1                 # entries behind the requests name a real block
    run(c, bf16(rng, 3, 16, 128))


def test_length_beyond_the_table_counts_up_to_it():
    rng = np.random.default_rng(14)
    c = Cache(rng, [64, 128], 1, 64)
    q = bf16(rng, 2, 8, 128)
    c.lens = [1000, -3]
    c.table[0, 1] = c.table[1, 0]
    run(c, q)


@pytest.mark.parametrize("bs", [16, 64])
def test_table_entries_outside_the_pool_are_left_out(bs):
    rng = np.random.default_rng(15)
    c = Cache(rng, [500, 200, 64], 2, bs)
    c.table[0, 1], c.table[0, 3], c.table[1, 0] = -1, c.num_blocks, 1 << 30
    c.table[2, :] = -(1 << 31)                              # nothing left: zeros
    got, _ = run(c, bf16(rng, 3, 16, 128))
    assert torch.all(got[2] == 0)


def test_two_requests_may_share_blocks():
    rng = np.random.default_rng(16)
    c = Cache(rng, [300, 300], 2, 64)
    c.table[1, :3] = c.table[0, :3]
    run(c, bf16(rng, 2, 16, 128))


# ------------------------------------------------------------------ selected positions
def selection(rng, lens, n_kv, budget):
    sel = np.full((len(lens), n_kv, budget), -1, np.int32)
    for b, n in enumerate(lens):
        for g in range(n_kv):
            k = min(n, budget)
            sel[b, g, :k] = np.sort(rng.choice(n, k, replace=False)) if n else []
    return sel


@pytest.mark.parametrize("lens,budget,n_q,n_kv", [([1000], 96, 8, 1), ([3000, 50, 0, 700], 257, 16, 2), ([9000], 4096, 64, 8),
                                                  ([500], 1, 4, 4), ([5000, 5000], 1000, 64, 1), ([400, 10], 4096, 32, 2)])
def test_selected(lens, budget, n_q, n_kv):
    rng = np.random.default_rng(budget)
    c = Cache(rng, lens, n_kv, 64)
    run(c, bf16(rng, len(lens), n_q, 128), selection(rng, lens, n_kv, budget))


def test_selected_in_any_order_with_gaps_repeats_and_strays():
    rng = np.random.default_rng(20)
    lens = [600, 300]
    c = Cache(rng, lens, 2, 16)
    sel = rng.integers(-3, 700, (2, 2, 150)).astype(np.int32)   # unsorted, repeated, some behind the context
    sel[0, 1] = -1                                              # a head that keeps nothing
    sel[1, 0, 1:] = -1
    sel[1, 0, 0] = 299
    sel[1, 1, 7], sel[1, 1, 8] = (1 << 31) - 1, -(1 << 31)
    got, _ = run(c, bf16(rng, 2, 16, 128), sel)
    assert torch.all(got[0, 8:] == 0)


def test_selecting_everything_equals_the_whole_context():
    rng = np.random.default_rng(21)
    c = Cache(rng, [900], 2, 64)
    q = bf16(rng, 1, 16, 128)
    run(c, q, np.broadcast_to(np.arange(900, dtype=np.int32), (1, 2, 900)).copy())
    run(c, q)


# ------------------------------------------------------------------ how it is called
def test_same_result_every_time_and_on_another_stream():
    rng = np.random.default_rng(30)
    c = Cache(rng, [9000, 17], 2, 64)
    q = bf16(rng, 2, 16, 128).to(DEV)
    first, ws = decode(c, q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    cache, table, lens = torch.from_numpy(c.rec).to(DEV), i32(c.table), i32(c.lens)
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        again, _ = decode(c, q, ws=ws, cache=cache, table=table, lens=lens)
        assert torch.equal(first, again)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other, _ = decode(c, q, ws=ws, cache=cache, table=table, lens=lens)
    s.synchronize()
    assert torch.equal(first, other)


def test_two_graphs_share_a_workspace_and_follow_the_lengths():
    rng = np.random.default_rng(31)
    c = Cache(rng, [5000, 800], 2, 64)
    q = bf16(rng, 2, 16, 128).to(DEV)
    sel = i32(selection(rng, c.lens, 2, 500))
    cache, table, lens = torch.from_numpy(c.rec).to(DEV), i32(c.table), i32(c.lens)
    n = max(spc.spc_kv4_decode_attn_workspace_size(2, 16, 2, 128, c.max_blocks, 64, k) for k in (0, 500))
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    outs, graphs = [], []
    for s in (None, sel):
        out, _ = decode(c, q, s, ws=ws, cache=cache, table=table, lens=lens)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            decode(c, q, s, out=out, ws=ws, cache=cache, table=table, lens=lens)
        outs.append(out)
        graphs.append(g)
    for new in ([4000, 0], [64, 800], [5000, 799]):
        lens.copy_(i32(new))
        for _ in range(2):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        for out, s in zip(outs, (None, sel)):
            want, mag = P.decode_attention(f64(q), c.rec, c.table, new, None if s is None else s.cpu().numpy(), SCALE)
            check(out, want, decode_tol(want, mag))


def test_a_pool_beyond_32_bit_offsets():
    rng = np.random.default_rng(32)
    c = Cache(rng, [300], 1, 128, spare=0)
    num = 250000                                            # 4.6 GB of records
    cache = torch.empty(num, 1, 128, 144, dtype=torch.uint8, device=DEV)
    where = np.array([num - 1, 240000, num - 2])
    cache[torch.from_numpy(where).to(DEV)] = torch.from_numpy(c.rec[c.table[0]]).to(DEV)
    q = bf16(rng, 1, 8, 128)
    want, mag = P.decode_attention(f64(q), c.rec, c.table, c.lens, None, SCALE)
    c.num_blocks = num
    got, _ = decode(c, q.to(DEV), cache=cache, table=i32(where[None]))
    check(got, want, decode_tol(want, mag))


# ------------------------------------------------------------------ how the work is cut
@pytest.mark.parametrize("n_q,budget", [(8, 0), (8, 1500), (128, 0), (256, 0)])
def test_more_long_segments_than_ctas(n_q, budget):
    # 160 segments, too long to go whole: runs that end inside segments and hold pieces of two
    rng = np.random.default_rng(50 + n_q)
    lens = [int(x) for x in rng.integers(1100, 1900, 20)]
    c = Cache(rng, lens, 8, 64)
    run(c, bf16(rng, 20, n_q, 128), selection(rng, lens, 8, budget) if budget else None)


def test_one_long_segment_over_all_ctas_and_heads_in_two_halves():
    rng = np.random.default_rng(51)
    run(Cache(rng, [30001], 1, 128), bf16(rng, 1, 64, 128))


def test_a_long_request_among_empty_and_short_ones():
    rng = np.random.default_rng(52)
    lens = [0, 3, 9000, 0, 0, 64, 1] + [5] * 20 + [0]
    run(Cache(rng, lens, 4, 16), bf16(rng, len(lens), 16, 128))


def test_calls_of_different_shapes_take_turns_on_one_workspace():
    rng = np.random.default_rng(53)
    calls, size = [], 0
    for lens, n_q, n_kv, budget in (([3000, 40], 64, 1, 0), ([3000, 40], 64, 1, 500), ([2500] * 40, 16, 2, 0),
                                    ([9000], 8, 1, 0), ([1500] * 12, 128, 4, 0), ([100, 7000], 32, 2, 3000)):
        c = Cache(rng, lens, n_kv, 64)
        sel = selection(rng, lens, n_kv, budget) if budget else None
        calls.append((c, bf16(rng, len(lens), n_q, 128), sel))
        size = max(size, spc.spc_kv4_decode_attn_workspace_size(len(lens), n_q, n_kv, 128, c.max_blocks, 64, budget))
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        for c, q, sel in calls:
            run(c, q, sel, ws=ws)
