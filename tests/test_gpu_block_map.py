"""spc_block_map against the oracle: every output equal, on seeded scenarios and
at the edges (nothing to do, exact block ends, blocks that go round within one
call, a stack that runs out)."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from sparse_kv_cache_retrieval_gb300 import binding as spc
from tests.paged_cases import DEV, i32

pytestmark = pytest.mark.gpu


def call(lens, nxt, table, free, n_free, bs, n_slots, status=0):
    B, mb = table.shape
    t = dict(len=i32(lens), nxt=i32(nxt), table=i32(table), free=i32(free), n=i32([n_free]), n2=i32([-7]),
             cu=torch.full((B + 2,), -9, dtype=torch.int32, device=DEV),
             slots=torch.full((n_slots + 5,), -9, dtype=torch.int32, device=DEV), status=i32([status]))

    def go():
        spc.spc_block_map(t["len"], t["nxt"], t["table"], t["free"], t["n"], t["n2"], t["cu"], t["slots"], t["status"],
                          B, mb, bs, len(free), n_slots)
    go()
    return t, go


def same(t, want, n_slots):
    wt, wf, wn, wcu, ws, ok = want
    B = wt.shape[0]
    assert int(t["status"].item()) == (0 if ok else -6)
    assert np.array_equal(t["table"].cpu().numpy(), wt)
    assert np.array_equal(t["free"].cpu().numpy(), wf)
    assert int(t["n2"].item()) == wn
    assert np.array_equal(t["cu"].cpu().numpy(), list(wcu) + [-9])
    s = t["slots"].cpu().numpy()
    assert np.array_equal(s[:n_slots], ws)
    assert np.all(s[n_slots:] == -9)                       # nothing behind the map is touched


def state(rng, lens, need, bs, max_blocks, spare=5):
    used = [-(-n // bs) for n in lens]
    num = sum(used) + need + spare
    perm = rng.permutation(num)
    table = np.full((len(lens), max_blocks), -1, np.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = perm[at:at + u]
        at += u
    free = np.full(num, -1, np.int32)
    free[:num - at] = perm[at:]
    return table, free, num - at


@pytest.mark.parametrize("seed", range(12))
def test_random_scenarios(seed):
    rng = np.random.default_rng(seed)
    B = int(rng.integers(1, 65))
    bs = int(rng.choice([16, 32, 64, 128]))
    hi = int(rng.choice([40, 700, 5000]))
    lens = rng.integers(0, hi, B) * (rng.random(B) < 0.7)
    nxt = np.where(rng.random(B) < 0.4, rng.integers(0, hi, B), lens + rng.integers(0, 3, B))
    mb = -(-int(max(lens.max(), nxt.max(), 1)) // bs) + int(rng.integers(0, 3))
    table, free, n_free = state(rng, lens, int(sum(-(-nxt // bs))), bs, mb)
    new = int(np.maximum(nxt - lens, 0).sum())
    n_slots = max(1, new + int(rng.integers(0, 50)))
    t, go = call(lens, nxt, table, free, n_free, bs, n_slots)
    want = P.block_map(lens, nxt, table, free, n_free, bs, n_slots)
    assert want[-1]
    same(t, want, n_slots)
    go()                                                   # the same lengths again: the same result
    same(t, want, n_slots)


@pytest.mark.parametrize("lens,nxt", [
    ([0], [0]),                      # nothing
    ([0], [1]), ([0], [64]), ([0], [65]), ([63], [64]), ([64], [65]), ([64], [64]),
    ([65], [64]), ([64], [63]), ([64], [0]), ([1], [0]),
    ([200, 0, 100], [0, 300, 100]),  # blocks given back are taken in the same call
    ([0, 0, 0], [0, 1, 0]),
    ([64] * 64, [65] * 64),          # every request needs a block
])
def test_edges(lens, nxt):
    rng = np.random.default_rng(3)
    table, free, n_free = state(rng, lens, sum(-(-n // 64) for n in nxt), 64, 6)
    n_slots = max(1, sum(max(0, b - a) for a, b in zip(lens, nxt)))
    t, _ = call(lens, nxt, table, free, n_free, 64, n_slots)
    same(t, P.block_map(lens, nxt, table, free, n_free, 64, n_slots), n_slots)


def test_only_blocks_given_back_are_free():
    # an empty stack: request 1 lives on the blocks of request 0, in the order of the stack
    table = np.array([[4, 2, 0], [-1, -1, -1]], np.int32)
    free = np.array([-1, -1, -1, -1, -1], np.int32)
    t, _ = call([40, 0], [0, 48], table, free, 0, 16, 48)
    same(t, P.block_map([40, 0], [0, 48], table, free, 0, 16, 48), 48)
    assert list(t["table"].cpu().numpy()[1]) == [0, 2, 4]


@pytest.mark.parametrize("lens,nxt,n_free,n_slots", [
    ([10, 0], [10, 65], 4, 65),          # one block too few on the stack
    ([10, 0], [10, 64], 4, 63),          # one slot too few
    ([10, 0], [10, -1], 4, 65),          # a negative length
    ([10, 0], [10, 16 * 6 + 1], 40, 200),  # longer than the table
    ([-1, 0], [10, 5], 4, 65),
    ([10, 0], [10, 5], -1, 65),          # a broken stack height
    ([10, 0], [10, 5], 41, 65),
    ([40, 0], [0, 5], 39, 65),           # blocks given back would pass the end of the stack
])
def test_refused_on_the_device(lens, nxt, n_free, n_slots):
    rng = np.random.default_rng(4)
    table = rng.permutation(40)[:12].reshape(2, 6).astype(np.int32)
    free = rng.permutation(40).astype(np.int32)
    want = P.block_map(lens, nxt, table, free, n_free, 16, n_slots)
    assert not want[-1]
    t, _ = call(lens, nxt, table, free, n_free, 16, n_slots)
    same(t, want, n_slots)


def test_the_first_error_of_a_status_word_stays():
    t, _ = call([0], [100], np.full((1, 2), -1, np.int32), np.zeros(4, np.int32), 4, 16, 100, status=-4)
    assert int(t["status"].item()) == -4
    assert np.all(t["slots"].cpu().numpy()[:100] == -1)


def test_a_table_entry_outside_the_pool_gives_no_slot():
    table = np.array([[99, -1], [2, -1], [-5, -1]], np.int32)
    t, _ = call([3, 3, 3], [5, 5, 5], table, np.zeros(4, np.int32), 0, 16, 6)
    assert list(t["slots"].cpu().numpy()[:6]) == [-1, -1, 2 * 16 + 3, 2 * 16 + 4, -1, -1]


def test_longest_requests():
    # 64 requests of 2^18 positions in 128-position blocks: 2^24 slots
    B, n, bs = 64, 1 << 18, 128
    nb = n // bs
    table = np.full((B, nb), -1, np.int32)
    free = np.arange(B * nb, dtype=np.int32)[::-1].copy()
    t, _ = call([0] * B, [n] * B, table, free, B * nb, bs, B * n)
    assert int(t["status"].item()) == 0 and int(t["n2"].item()) == 0
    assert torch.equal(t["slots"][:B * n], torch.arange(B * n, dtype=torch.int32, device=DEV))
    assert np.array_equal(t["table"].cpu().numpy().ravel(), np.arange(B * nb))


def test_captured_and_replayed_with_new_lengths():
    rng = np.random.default_rng(8)
    lens, nxt = [100, 0, 37, 64], [101, 70, 0, 65]
    table, free, n_free = state(rng, lens, 12, 16, 9)
    t, go = call(lens, nxt, table, free, n_free, 16, 80)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    nxt = [0, 70, 40, 66]
    t["nxt"].copy_(i32(nxt))
    t["table"].copy_(i32(table))
    t["free"].copy_(i32(free))
    graph.replay()
    torch.cuda.synchronize()
    same(t, P.block_map(lens, nxt, table, free, n_free, 16, 80), 80)
