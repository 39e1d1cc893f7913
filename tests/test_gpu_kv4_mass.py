"""spc_kv4_attn_mass against the float64 oracle: group sizes, lengths at the
tiles' edges, windows of a request's last tokens, the earlier sums kept, faded
and not read, rows that see nothing, values that are not finite, and how it is
called."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from sparse_kv_cache_retrieval_gb300 import binding as spc
from tests.chunk_cases import chunk, close, cu_of, mass, mass_tol, workspace
from tests.paged_cases import DEV, SCALE, Cache, bf16, f64, i32

pytestmark = pytest.mark.gpu


def prev_of(rng, c, cap=None):
    return torch.from_numpy(rng.random((len(c.lens), c.n_kv, cap or c.max_blocks * c.bs)).astype(np.float32) * 3).to(DEV)


def check(c, q, new, lse, prev, keep, got, scale=SCALE, table=None, lens=None):
    with np.errstate(invalid="ignore", over="ignore"):
        want, rel = P.attn_mass(f64(q), c.rec, c.table if table is None else table, c.lens if lens is None else lens,
                                cu_of(new), f64(lse), f64(prev), keep, got.shape[2], scale)
    got = got.clone()
    lens = np.clip(c.lens if lens is None else lens, 0, c.max_blocks * c.bs)
    for b, n in enumerate(lens):
        assert np.all(f64(got[b, :, n:]) == 7)              # entries behind the request are left as they were
        close(got[b, :, :n], want[b, :, :n], mass_tol(want, rel)[b, :, :n], f"mass of request {b}")


def run(seed, lens, new, n_q, n_kv, bs, keep=1.0, tail=0, cap=None):
    rng = np.random.default_rng(seed)
    c = Cache(rng, lens, n_kv, bs)
    q = bf16(rng, sum(new) + tail, n_q, 128).to(DEV)
    _, lse, _ = chunk(c, q, new)
    prev = prev_of(rng, c, cap)
    got, _ = mass(c, q, new, lse, prev, keep, cap=cap)
    check(c, q, new, lse, prev, keep, got)


@pytest.mark.parametrize("n_q,n_kv", [(1, 1), (2, 1), (8, 2), (8, 1), (16, 1), (32, 1), (64, 1), (12, 3)])
@pytest.mark.parametrize("lens,new", [([1], [1]), ([300], [1]), ([300], [7]), ([129], [129]), ([200, 31, 640], [40, 31, 3])])
def test_groups(n_q, n_kv, lens, new):
    run(n_q * 7 + len(lens), lens, new, n_q, n_kv, 16)


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 128, 130, 257])
def test_lengths_at_the_edges_of_tiles(bs, n):
    run(bs + n, [n, n + 127, n + 128, n + 1000], [n, n, n, n], 4, 1, bs, keep=0.5, tail=3)


@pytest.mark.parametrize("n_q,n_kv,lens,new,keep", [
    (8, 2, [1500], [700], 0.0), (32, 8, [5000, 40, 900], [1, 1, 1], 1.0), (64, 1, [3500], [130], 0.25), (4, 4, [700, 1100], [1, 64], 1.0),
    (8, 8, [20000], [2], 0.0), (64, 8, [9000, 1], [4, 1], 1.0)])
def test_longer_contexts(n_q, n_kv, lens, new, keep):
    run(sum(lens), lens, new, n_q, n_kv, 64, keep=keep, tail=2)


def test_requests_without_tokens_keep_their_sums():
    run(1, [50, 0, 70, 0, 33], [3, 0, 0, 0, 33], 8, 2, 16, tail=5)
    run(2, [40, 300], [0, 0], 8, 2, 16, keep=0.5, tail=4)
    run(3, [5] * 64, [1] * 64, 8, 2, 16)


def test_no_rows_at_all():
    rng = np.random.default_rng(4)
    c = Cache(rng, [40, 200], 2, 16)
    prev = prev_of(rng, c)
    q = torch.zeros(0, 8, 128, dtype=torch.bfloat16, device=DEV)
    got, _ = mass(c, q, [0, 0], torch.zeros(0, 8, device=DEV), prev, 0.5)
    check(c, q, [0, 0], torch.zeros(0, 8), prev, 0.5, got)


def test_a_row_longer_than_the_table():
    run(5, [100, 40], [20, 1], 8, 2, 16, cap=1000)


@pytest.mark.parametrize("n_q", [1, 4, 64])
def test_tokens_before_position_zero_add_nothing(n_q):
    run(6, [10, 0, 200], [17, 3, 260], n_q, 1, 16)


def test_blocks_outside_the_pool():
    rng = np.random.default_rng(7)
    c = Cache(rng, [700, 700, 700], 2, 16)
    c.table[0, [0, 7, 8, 9, 10, 11, 12, 13, 14, 15, 16, 43]] = -1
    c.table[1, :] = [c.num_blocks, 2 ** 31 - 1, -2 ** 31, -1] * 11
    c.table[2, 40:] = c.num_blocks
    new = [150, 20, 90]
    q = bf16(rng, 260, 8, 128).to(DEV)
    _, lse, _ = chunk(c, q, new)
    prev = prev_of(rng, c)
    got, _ = mass(c, q, new, lse, prev, 1.0)
    check(c, q, new, lse, prev, 1.0, got)


def test_earlier_sums_are_not_read_where_nothing_is_kept():
    rng = np.random.default_rng(8)
    c = Cache(rng, [300], 2, 16)
    q = bf16(rng, 5, 8, 128).to(DEV)
    _, lse, _ = chunk(c, q, [5])
    prev = torch.full((1, 2, 304), float("nan"), device=DEV)
    got, ws = mass(c, q, [5], lse, prev, 0.0)
    check(c, q, [5], lse, torch.zeros(1, 2, 304), 0.0, got)
    none, _ = mass(c, q, [5], lse, None, 0.0, ws=ws)
    assert torch.equal(none, got)


def test_sums_in_place():
    rng = np.random.default_rng(9)
    c = Cache(rng, [1000, 30], 2, 16)
    q = bf16(rng, 40, 8, 128).to(DEV)
    _, lse, _ = chunk(c, q, [20, 20])
    prev = prev_of(rng, c)
    got, _ = mass(c, q, [20, 20], lse, prev, 0.5)
    own = prev.clone()
    mass(c, q, [20, 20], lse, own, 0.5, out=own)
    assert torch.equal(own[0, :, :1000], got[0, :, :1000]) and torch.equal(own[1, :, :30], got[1, :, :30])
    assert torch.equal(own[1, :, 30:], prev[1, :, 30:])


def test_sums_of_windows_add_up():
    """The tokens in pieces, each over the context that its last one sees, are the tokens at once."""
    rng = np.random.default_rng(10)
    c = Cache(rng, [500], 2, 16)
    q = bf16(rng, 300, 8, 128).to(DEV)
    _, lse, _ = chunk(c, q, [300])
    whole, _ = mass(c, q, [300], lse, None, 0.0)
    acc = torch.zeros_like(whole)
    for i, j in ((0, 1), (1, 130), (130, 300)):
        mass(c, q[i:j], [j - i], lse[i:j].contiguous(), acc, 1.0, out=acc, lens=i32([200 + j]))
    check(c, q, [300], lse, torch.zeros_like(acc), 0.0, torch.where(torch.arange(512, device=DEV) < 500, acc, 7.0))


# ------------------------------------------------------------------ values that are not finite
def test_lse_of_minus_infinity_adds_nothing_and_nan_reaches_what_its_row_sees():
    rng = np.random.default_rng(11)
    c = Cache(rng, [260], 1, 16)
    q = bf16(rng, 200, 4, 128)
    q[7, 1, 3] = float("nan")
    q = q.to(DEV)
    _, lse, _ = chunk(c, torch.nan_to_num(q), [200])
    lse[7, 1] = lse[50, 2] = lse[199, 3] = -float("inf")
    prev = prev_of(rng, c)
    got, _ = mass(c, q, [200], lse, prev, 1.0)
    check(c, torch.nan_to_num(q), [200], lse, prev, 1.0, got)
    lse[20, 0] = float("nan")                               # its row is at position 80
    got, _ = mass(c, q, [200], lse, prev, 1.0)
    g = f64(got)[0, 0]
    assert np.isnan(g[:81]).all() and np.isfinite(g[81:]).all()


def test_what_a_row_does_not_see_does_not_change():
    rng = np.random.default_rng(12)
    c = Cache(rng, [300, 200], 2, 16)
    q = bf16(rng, 170, 4, 128)
    clean = q.clone().to(DEV)
    q[150:] = float("nan")                                  # rows of no request
    q[40, 0, 0] = float("inf")                              # head 0 of the token at position 240 of request 0
    q = q.to(DEV)
    new = [100, 50]
    _, lse, _ = chunk(c, clean, new)
    prev = prev_of(rng, c)
    got, _ = mass(c, q, new, lse, prev, 1.0)
    want, _ = mass(c, clean, new, lse, prev, 1.0)
    assert torch.equal(got[0, :, 241:300], want[0, :, 241:300]) and torch.equal(got[0, 1], want[0, 1])
    assert torch.equal(got[1], want[1])
    c.rec[c.table[0, 2], 0, 5, 128:136] = 0x7f              # K of position 37: NaN, its own sum alone
    got, _ = mass(c, clean, new, lse, prev, 1.0)
    g, w = f64(got), f64(want)
    assert np.isnan(g[0, 0, 37])
    g[0, 0, 37] = w[0, 0, 37]
    assert np.array_equal(g, w)


@pytest.mark.parametrize("amp", [2.0 ** -100, 2.0 ** 30, 2.0 ** 100])
def test_queries_of_any_size(amp):
    rng = np.random.default_rng(13)
    c = Cache(rng, [300], 1, 16)
    q = (bf16(rng, 60, 4, 128).double() * amp).to(torch.bfloat16).to(DEV)
    scale = float(np.float32(SCALE / amp))
    _, lse, _ = chunk(c, q, [60], scale=scale)
    prev = prev_of(rng, c)
    got, _ = mass(c, q, [60], lse, prev, 1.0, scale=scale)
    check(c, q, [60], lse, prev, 1.0, got, scale=scale)


# ------------------------------------------------------------------ how it is called
def test_rows_inside_fused_projections():
    rng = np.random.default_rng(14)
    c = Cache(rng, [300, 300], 2, 32)
    fused = bf16(rng, 90, 8 + 4 + 3, 128).to(DEV)
    for q in (fused[:, :8], fused[:, 7:15]):
        _, lse, _ = chunk(c, q, [50, 33])
        prev = prev_of(rng, c)
        got, _ = mass(c, q, [50, 33], lse, prev, 1.0)
        check(c, q, [50, 33], lse, prev, 1.0, got)


def test_the_same_bits_every_time_and_on_a_used_workspace():
    rng = np.random.default_rng(15)
    ws = workspace(max(spc.spc_kv4_attn_mass_workspace_size(*s, 128) for s in ((600, 4, 32, 8), (600, 4, 64, 1), (8, 1, 4, 1))))
    for lens, new, n_q, n_kv in (([2000, 100, 9, 500], [300, 100, 9, 1], 32, 8), ([2000, 10, 0, 64], [200, 1, 0, 5], 64, 1),
                                 ([20000], [8], 4, 1)):
        c = Cache(rng, lens, n_kv, 32)
        q = bf16(rng, sum(new), n_q, 128).to(DEV)
        _, lse, _ = chunk(c, q, new)
        prev = prev_of(rng, c)
        first, _ = mass(c, q, new, lse, prev, 1.0)
        for _ in range(3):
            got, _ = mass(c, q, new, lse, prev, 1.0, ws=ws)
            assert torch.equal(got, first)
        check(c, q, new, lse, prev, 1.0, first)
        assert not ws[:4].any()


def test_streams_at_once():
    rng = np.random.default_rng(16)
    jobs = []
    for i in range(4):
        c = Cache(rng, [1500 - 300 * i, 200], 2, 32)
        q = bf16(rng, 90, 8, 128).to(DEV)
        _, lse, _ = chunk(c, q, [60, 30])
        jobs.append((c, q, lse, prev_of(rng, c), torch.from_numpy(c.rec).to(DEV), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for c, q, lse, prev, cache, st in jobs:
        with torch.cuda.stream(st):
            for _ in range(3):
                r, _ = mass(c, q, [60, 30], lse, prev, 1.0, cache=cache)
            got.append(r)
    torch.cuda.synchronize()
    for (c, q, lse, prev, _, _), r in zip(jobs, got):
        check(c, q, [60, 30], lse, prev, 1.0, r)


def test_a_captured_call_follows_lengths():
    rng = np.random.default_rng(17)
    c = Cache(rng, [900, 900], 2, 16)
    q = bf16(rng, 64, 8, 128).to(DEV)
    lens, cu = i32(c.lens), i32(cu_of([40, 24]))
    cache, table = torch.from_numpy(c.rec).to(DEV), i32(c.table)
    lse = torch.full((64, 8), 6.0, device=DEV)
    prev = prev_of(rng, c)
    got, ws = mass(c, q, None, lse, prev, 1.0, lens=lens, cu=cu, cache=cache, table=table)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mass(c, q, None, lse, prev, 1.0, out=got, ws=ws, lens=lens, cu=cu, cache=cache, table=table)
    for new_lens, new in (([900, 900], [40, 24]), ([64, 500], [1, 63]), ([900, 0], [64, 0]), ([129, 777], [0, 64])):
        lens.copy_(i32(new_lens))
        cu.copy_(i32(cu_of(new)))
        got.fill_(7)
        graph.replay()
        graph.replay()
        check(c, q, new, lse, prev, 1.0, got, lens=new_lens)


def test_lengths_beyond_the_table_and_below_zero_are_cut():
    rng = np.random.default_rng(18)
    c = Cache(rng, [160, 160, 160], 1, 16)
    q = bf16(rng, 60, 4, 128).to(DEV)
    lse, prev = torch.full((60, 4), 5.0, device=DEV), prev_of(rng, c)
    for lens in ([5000, -3, 2 ** 31 - 1], [160, -2 ** 31, 161]):
        got, _ = mass(c, q, [20, 20, 20], lse, prev, 1.0, lens=i32(lens))
        check(c, q, [20, 20, 20], lse, prev, 1.0, got, lens=lens)
