"""spc_kv4_evict against the oracle, bit for bit: budgets and lengths at the
ranks' edges, equal sums, forced positions, in place and into other blocks,
requests with blocks outside the pool, and how it is called."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from sparse_kv_cache_retrieval_gb300 import binding as spc
from tests.paged_cases import DEV, Cache, i32

pytestmark = pytest.mark.gpu


def pool(rng, lens, n_kv, bs, spare=3, max_blocks=None):
    """A Cache whose records are random bytes (eviction does not look into them)."""
    c = Cache(rng, [0] * len(lens), n_kv, bs, spare=sum(-(-n // bs) for n in lens) + spare,
              max_blocks=max_blocks or max(-(-n // bs) for n in list(lens) + [1]))
    c.rec[:] = rng.integers(0, 256, c.rec.shape, dtype=np.uint8)
    perm, at = rng.permutation(c.num_blocks), 0
    for b, n in enumerate(lens):
        u = -(-n // bs)
        c.table[b, :u] = perm[at:at + u]
        at += u
    c.lens = list(lens)
    return c


class Call:
    def __init__(self, c, mass, budget, n_sink=0, n_recent=0, table_next=None, lens=None, in_place=False, kept=True, cap=None):
        B = len(c.lens)
        self.c, self.budget, self.n_sink, self.n_recent = c, budget, n_sink, n_recent
        self.cap = cap or c.max_blocks * c.bs
        self.mass_np, self.lens_np = mass, c.lens if lens is None else lens
        self.cache = torch.from_numpy(c.rec).to(DEV)
        self.table, self.len = i32(c.table), i32(self.lens_np)
        self.table_next = self.table if table_next is None else i32(table_next)
        self.next_np = c.table if table_next is None else table_next
        self.len_next = i32([-9] * B)
        self.mass = torch.from_numpy(mass).to(DEV)
        self.mass_next = self.mass if in_place else torch.full_like(self.mass, 7.0)
        self.kept = torch.full((B, c.n_kv, budget), -5, dtype=torch.int32, device=DEV) if kept else None
        self.status = i32([0])

    def __call__(self, stream=None):
        c = self.c
        spc.spc_kv4_evict(self.cache, self.table, self.table_next, self.len, self.len_next, self.mass, self.mass_next, self.kept,
                          self.status, len(c.lens), c.n_kv, 128, c.num_blocks, c.bs, c.max_blocks, self.cap, self.budget,
                          self.n_sink, self.n_recent, stream=stream)
        return self

    def check(self):
        c = self.c
        rec, kept, nxt, mass, ok = P.evict(c.rec, c.table, self.next_np, self.lens_np, self.mass_np, self.budget, self.n_sink,
                                           self.n_recent)
        if self.mass_next is not self.mass:
            for b, n in enumerate(self.lens_np):
                mass[b, :, max(0, min(n, c.max_blocks * c.bs)):] = 7
            assert np.array_equal(self.mass.cpu().numpy(), self.mass_np, equal_nan=True)
        assert int(self.status.item()) == (0 if ok else -1)
        assert np.array_equal(self.len_next.cpu().numpy(), nxt)
        if self.kept is not None:
            got = self.kept.cpu().numpy()
            assert np.array_equal(got, kept), np.argwhere(got != kept)[:4]
        got = self.mass_next.cpu().numpy()
        assert np.array_equal(got, mass, equal_nan=True), np.argwhere(got != mass)[:4]
        got = self.cache.cpu().numpy()
        assert np.array_equal(got, rec), np.argwhere(got != rec)[:4]


def sums(rng, c, cap=None, kind="wide"):
    shape = (len(c.lens), c.n_kv, cap or c.max_blocks * c.bs)
    if kind == "wide":
        x = np.exp(rng.standard_normal(shape) * 4)
    elif kind == "ties":
        x = rng.integers(0, 4, shape) / 8
    elif kind == "equal":
        x = np.full(shape, 0.25)
    elif kind == "near":                                    # keys that differ in their last bits alone
        x = 1 + rng.integers(0, 700, shape) * 2.0 ** -23
    else:
        x = np.zeros(shape)
    return x.astype(np.float32)


@pytest.mark.parametrize("kind", ["wide", "ties", "equal", "near", "zero"])
@pytest.mark.parametrize("n,budget,n_sink,n_recent", [(1000, 1, 0, 0), (1000, 7, 3, 4), (1000, 100, 4, 64), (1000, 999, 4, 64),
                                                      (5000, 1024, 4, 64), (4097, 4096, 0, 1)])
@pytest.mark.parametrize("in_place", [True, False])
def test_kept_sets(kind, n, budget, n_sink, n_recent, in_place):
    rng = np.random.default_rng(n + budget)
    c = pool(rng, [n, n // 2 + 1], 2, 16)
    Call(c, sums(rng, c, kind=kind), budget, n_sink, n_recent, in_place=in_place)().check()


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("budget", [1, 8, 15, 16, 17, 255, 256, 257, 511, 513])
def test_lengths_and_budgets_at_the_edges(bs, budget):
    rng = np.random.default_rng(bs * budget)
    c = pool(rng, [0, 1, budget - 1, budget, budget + 1, 2 * budget + 31, 700], 3, bs)
    Call(c, sums(rng, c), budget, min(2, budget // 2), min(5, budget // 2), in_place=budget % 2 == 0)().check()


def other_blocks(c, budget):
    """A table of blocks that no request holds."""
    free = sorted(set(range(c.num_blocks)) - set(c.table[c.table >= 0].tolist()))
    nxt, at = np.full_like(c.table, -7), 0
    for b, n in enumerate(c.lens):
        u = -(-min(n, budget) // c.bs)
        assert at + u <= len(free)
        nxt[b, :u] = free[at:at + u]
        at += u
    return nxt


@pytest.mark.parametrize("budget", [40, 200, 3000])
def test_into_other_blocks(budget):
    rng = np.random.default_rng(budget)
    lens = [900, 10, 2500, 0, 333]
    c = pool(rng, lens, 2, 32, spare=200)
    Call(c, sums(rng, c), budget, 4, 16, table_next=other_blocks(c, budget))().check()


def test_into_blocks_that_are_partly_its_own():
    """Some of the request's blocks keep their places, the others are new."""
    rng = np.random.default_rng(1)
    c = pool(rng, [1000, 600], 2, 16, spare=40)
    nxt = other_blocks(c, 300)
    nxt[0, :10], nxt[1, 3:6] = c.table[0, :10], c.table[1, 3:6]
    Call(c, sums(rng, c), 300, 4, 16, table_next=nxt)().check()


def test_the_largest():
    rng = np.random.default_rng(2)
    c = pool(rng, [262144], 1, 128)
    Call(c, sums(rng, c), 4096, 4, 64)().check()
    c = pool(rng, [70000, 262144 // 4], 4, 64, max_blocks=4096)
    Call(c, sums(rng, c, kind="near"), 4096, 0, 0, in_place=True)().check()


@pytest.mark.parametrize("n", [16384, 16385, 32768, 40000, 65536, 70000, 131072, 140000])
@pytest.mark.parametrize("in_place", [True, False])
def test_every_number_of_ranks(n, in_place):
    """A rank has 16384 positions: one to eight ranks, the last ones with little or nothing."""
    rng = np.random.default_rng(n)
    c = pool(rng, [n, n // 3], 1, 16)
    m = sums(rng, c)
    m[0, 0, n - 5000:] *= 1e6                                # most of what is kept lies behind
    for budget in (100, 2100, 4096):
        Call(c, m.copy(), budget, 4, 64, in_place=in_place)().check()


def test_many_requests_and_heads():
    rng = np.random.default_rng(3)
    c = pool(rng, [17 + 3 * b for b in range(64)], 16, 16)
    Call(c, sums(rng, c), 60, 2, 8, in_place=True)().check()


def test_sums_that_are_odd():
    rng = np.random.default_rng(4)
    c = pool(rng, [600], 2, 16)
    m = sums(rng, c)
    m[0, 0, ::7], m[0, 0, 1::11], m[0, 0, 5::29], m[0, 1, :] = np.nan, -1.0, np.inf, np.nan
    m[0, 0, 3::13] = -0.0
    m[0, 0, 9::17] = 1e-42                                  # subnormal
    Call(c, m, 100, 2, 3, in_place=True)().check()
    Call(c, m, 500, 2, 3)().check()


def test_forced_positions_fill_the_budget():
    rng = np.random.default_rng(5)
    c = pool(rng, [300, 69, 68, 67], 2, 16)
    Call(c, sums(rng, c), 68, 4, 64)().check()
    Call(c, sums(rng, c), 68, 68, 0)().check()
    Call(c, sums(rng, c), 68, 0, 68, in_place=True)().check()


def test_blocks_outside_the_pool_leave_the_request():
    rng = np.random.default_rng(6)
    c = pool(rng, [500, 400, 300, 200], 2, 16)
    c.table[0, 20] = -1
    c.table[2, 18] = c.num_blocks
    c.table[3, 13:] = -1                                     # behind its 200 positions: not looked at
    Call(c, sums(rng, c), 100, 4, 16)().check()
    Call(c, sums(rng, c), 100, 4, 16, in_place=True)().check()
    c = pool(rng, [500, 400], 2, 16, spare=20)
    nxt = other_blocks(c, 100)
    nxt[1, 6] = 2 ** 31 - 1
    nxt[0, 7] = -1                                           # behind its 100 positions
    Call(c, sums(rng, c), 100, 4, 16, table_next=nxt)().check()


def test_lengths_beyond_the_table_and_below_zero_are_cut():
    rng = np.random.default_rng(7)
    c = pool(rng, [160, 160, 160], 1, 16)
    for lens in ([5000, -3, 2 ** 31 - 1], [160, -2 ** 31, 161]):
        Call(c, sums(rng, c), 50, 2, 8, lens=lens)().check()


def test_without_kept_and_with_longer_rows():
    rng = np.random.default_rng(8)
    c = pool(rng, [700, 90], 2, 16)
    Call(c, sums(rng, c, cap=1500), 64, 2, 8, kept=False, cap=1500)().check()


def test_twice_is_once():
    rng = np.random.default_rng(9)
    c = pool(rng, [700, 90], 2, 16)
    x = Call(c, sums(rng, c), 64, 2, 8, in_place=True)()
    x.check()
    rec, m, n = x.cache.clone(), x.mass.clone(), x.len_next.clone()
    x.len.copy_(n)
    x()
    assert torch.equal(x.cache, rec) and torch.equal(x.mass, m) and torch.equal(x.len_next, n)
    assert torch.equal(x.kept[0, 0].cpu(), torch.arange(64, dtype=torch.int32))


def test_streams_and_graphs():
    rng = np.random.default_rng(10)
    calls = []
    for i in range(3):
        c = pool(rng, [1500 + i, 300], 2, 32, spare=60)
        calls.append(Call(c, sums(rng, c), 256, 4, 32, table_next=other_blocks(c, 256)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for x, s in zip(calls, streams):
        for _ in range(3):
            x(stream=s)
    torch.cuda.synchronize()
    for x in calls:
        x.check()
    x = calls[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x()
    for n in (1500, 256, 40, 0):
        x.lens_np = [n, 300]
        x.len.copy_(i32(x.lens_np))
        x.cache.copy_(torch.from_numpy(x.c.rec))
        x.mass_next.fill_(7)
        graph.replay()
        graph.replay()
        x.check()
