"""spc_kv4_evict where nothing is selected and a head has several ranks: requests
not longer than the budget in tables that are much longer, and sinks and recent
positions that fill the budget. The ranks' first words to each other are then
their counts."""
import numpy as np
import pytest

from tests.test_gpu_kv4_evict import Call, other_blocks, pool, sums

pytestmark = pytest.mark.gpu


# positions of the table: one, two, four and eight ranks
@pytest.mark.parametrize("table", [8192, 20000, 60000, 131072])
@pytest.mark.parametrize("budget,lens", [(4096, [0, 1, 31, 300, 2500, 4095, 4096]), (200, [7, 199, 200]), (4096, [5000, 3, 4096])])
def test_requests_not_longer_than_the_budget(table, budget, lens):
    rng = np.random.default_rng(table + budget)
    c = pool(rng, lens, 2, 16, spare=3 + sum(-(-min(n, budget) // 16) for n in lens), max_blocks=table // 16)
    m = sums(rng, c)
    Call(c, m.copy(), budget, 4, 64, in_place=True)().check()
    Call(c, m, budget, 4, 64, table_next=other_blocks(c, budget))().check()


@pytest.mark.parametrize("table", [8192, 20000, 60000, 131072])
@pytest.mark.parametrize("n_sink,n_recent", [(4, 1020), (1024, 0), (0, 1024)])
def test_forced_positions_that_fill_the_budget(table, n_sink, n_recent):
    rng = np.random.default_rng(table + n_sink)
    c = pool(rng, [7000, 1025, 1024, 10], 2, 16, max_blocks=table // 16)
    Call(c, sums(rng, c), 1024, n_sink, n_recent, in_place=True)().check()


@pytest.mark.parametrize("budget", [300, 600, 4096])
def test_few_heads_with_long_budgets(budget):
    """The ranks that a long budget has, in a short table."""
    rng = np.random.default_rng(budget)
    c = pool(rng, [budget, budget // 2, 0], 1, 16)
    for _ in range(20):
        Call(c, sums(rng, c), budget, 4, 64, in_place=True)().check()


def test_blocks_outside_the_pool_in_a_long_table():
    rng = np.random.default_rng(1)
    c = pool(rng, [500, 400, 300], 2, 16, max_blocks=8192)
    c.table[1, 20] = -1
    Call(c, sums(rng, c), 1000, 4, 16)().check()
    Call(c, sums(rng, c), 100, 4, 16, in_place=True)().check()
