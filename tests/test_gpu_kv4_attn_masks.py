"""The masks of a tile in the tcgen05 decode attention: four words, each written
by a lane of its own for 32 of the tile's 128 positions. Table entries outside
the pool make every pattern of words that blocks of 16 to 128 positions can, on
tiles that follow one another, so that a word of another tile would show."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from tests.paged_cases import DEV, SCALE, Cache, bf16, check, decode, decode_tol, f64, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_q", [32, 64])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
def test_every_word_of_a_tiles_mask(n_q, bs):
    rng = np.random.default_rng(60 + bs)
    c = Cache(rng, [5003, 1290, 77], 1, bs)
    bad = np.array([-1, c.num_blocks, 1 << 30, -(1 << 31)])
    drop = rng.random(c.table.shape) < 0.5
    if bs == 32:
        # a word a block: all sixteen patterns of the first tiles in turn
        for t in range(16):
            drop[0, 4 * t:4 * t + 4] = [(t >> w) & 1 for w in range(4)]
    c.table[drop] = rng.choice(bad, int(drop.sum()))
    q = bf16(rng, 3, n_q, 128)
    want, mag = P.decode_attention(f64(q), c.rec, c.table, c.lens, None, SCALE)
    first, ws = decode(c, q.to(DEV))
    check(first, want, decode_tol(want, mag))
    cache, table, lens = torch.from_numpy(c.rec).to(DEV), i32(c.table), i32(c.lens)
    for _ in range(20):
        again, _ = decode(c, q.to(DEV), ws=ws, cache=cache, table=table, lens=lens)
        assert torch.equal(first, again)
    assert int(ws[:4].view(torch.int32).item()) == 0
