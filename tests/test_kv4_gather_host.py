"""The barrier protocol of the selected-position decode attention, as a model on
the CPU: copying warps fill rings of tiles that computing warps empty, and both
wait on the parity of a phase. A phase and the one two before it have the same
parity, so a wait is only right while the waiter is at most one phase ahead. The
numbers of warps and stages are read from the kernel's source."""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_kv_cache_retrieval_gb300", "csrc")


def configs():
    """(computing warps, copying warps, stages) of one head tile and of more, positions selected."""
    src = open(os.path.join(CSRC, "kv4_attn.cu")).read()
    pick = lambda name: re.search(rf"static constexpr int {name} = ([^;]*);", src).group(1)  # noqa: E731

    def value(expr, one):
        # C's conditional expressions over HT and SEL, nested to the right; SEL is true
        m = re.fullmatch(r"(.*?) \? (.*?) : (.*)", expr.strip())
        if not m:
            return int(expr)
        cond = {"!SEL": False, "SEL": True, "HT == 1": one, "HT > 1": not one}[m.group(1).strip()]
        return value(m.group(2) if cond else m.group(3), one)

    out = []
    for one in (True, False):
        every, copy, stages = (value(pick(n), one) for n in ("kAll", "kCopy", "kStages"))
        out.append((every - copy, copy, stages))
    return out


def violations(W, N, S, tiles, seed):
    """Runs the protocol with warps of changing speeds; the number of tiles that were overwritten before they were read
    (the run ends at the first)."""
    rng = random.Random(seed)
    filled = [[0] * S for _ in range(W)]                    # phases completed: stage's full barrier
    emptied = [[0] * S for _ in range(W)]                   # and its empty one
    read = [0] * W                                          # tiles that warp r has read
    done = lambda phases, parity: (phases & 1) != parity    # noqa: E731  (what a parity wait can tell)
    copy_at, end = list(range(N)), tiles
    speed = [1.0] * (W + N)
    while any(t < end for t in copy_at) or any(r + read[r] * W < end for r in range(W)):
        if rng.random() < 0.02:
            speed = [rng.choice((0.02, 1.0, 1.0)) for _ in speed]
        moved = False
        for i in rng.sample(range(W + N), W + N):
            if rng.random() > speed[i]:
                moved = True
                continue
            if i < W:
                k = read[i]
                if i + k * W < end and done(filled[i][k % S], (k // S) & 1):
                    emptied[i][k % S] += 1
                    read[i] += 1
                    moved = True
            else:
                t = copy_at[i - W]
                if t >= end:
                    continue
                r, use = t % W, t // W
                if use >= S and not done(emptied[r][use % S], ((use // S) & 1) ^ 1):
                    continue
                if use - S >= read[r]:
                    return 1                                # the stage's tile has not been read
                filled[r][use % S] += 1
                copy_at[i - W] += N
                moved = True
        if not moved:
            return 1                                        # nobody can move: every wait would run out
    return 0


@pytest.mark.parametrize("which", [0, 1], ids=["one head tile", "more"])
def test_no_tile_is_overwritten_before_it_is_read(which):
    W, N, S = configs()[which]
    assert sum(violations(W, N, S, 600, seed) for seed in range(60)) == 0


def test_the_model_finds_rings_that_several_warps_fill():
    # 11 rings filled by five warps in turn: a warp comes to a ring five tiles after its last one there
    assert sum(violations(11, 5, 2, 600, seed) for seed in range(60)) > 0
    assert sum(violations(10, 5, 2, 600, seed) for seed in range(60)) == 0
