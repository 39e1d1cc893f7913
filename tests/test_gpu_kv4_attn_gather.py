"""The gather of selected positions under warps of uneven speed: contexts whose
tiles alternate between nothing to do, a part of their positions, and maxima that
rise, called many times. Every call ends without a wait running out, with the same
bits."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from tests.paged_cases import DEV, Cache, check, decode, decode_tol, f64, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_q,n_kv", [(4, 4), (8, 1), (16, 1), (64, 1)])
@pytest.mark.parametrize("lens", [[20000], [9000, 300, 15000, 4000]])
def test_uneven_tiles(n_q, n_kv, lens):
    rng = np.random.default_rng(140 + n_q)
    c = Cache(rng, lens, n_kv, 32)
    budget = 4096
    sel = np.full((len(lens), n_kv, budget), -1, np.int32)
    u = np.sign(rng.standard_normal(128))
    for b, n in enumerate(lens):
        size = np.cumsum(rng.random(n) < 20 / n) * 0.25          # logits that rise in some 20 steps
        for i, blk in enumerate(c.table[b, :-(-n // 32)]):
            m = min(32, n - 32 * i)
            k = u * size[32 * i:32 * i + m, None] + 0.2 * rng.standard_normal((n_kv, m, 128))
            c.rec[blk, :, :m] = P.records(k, rng.standard_normal((n_kv, m, 128)))
        for g in range(n_kv):
            pos = np.sort(rng.choice(n, min(n, budget), replace=False))
            kind = rng.integers(0, 4, budget // 32)              # a tile: whole, empty, a few, every second
            keep = np.ones(len(pos), bool)
            for t, kd in enumerate(kind):
                s = slice(32 * t, min(32 * t + 32, len(pos)))
                if kd == 1:
                    keep[s] = False
                elif kd == 2:
                    keep[s] = rng.random(len(keep[s])) < 0.1
                elif kd == 3:
                    keep[s] = np.arange(len(keep[s])) % 2 == 0
            sel[b, g, :len(pos)] = np.where(keep, pos, -1)
    q = torch.from_numpy(u + 0.3 * rng.standard_normal((len(lens), n_q, 128))).to(torch.bfloat16)
    scale = 0.1
    cache, table, ln, sd = torch.from_numpy(c.rec).to(DEV), i32(c.table), i32(c.lens), i32(sel)
    first, ws = decode(c, q.to(DEV), sd, scale=scale, cache=cache, table=table, lens=ln)
    want, mag = P.decode_attention(f64(q), c.rec, c.table, c.lens, sel, scale)
    # logits up to 128 * 5 * 0.1 here: a sum of 128 products of magnitudes 830 at most, off by 129 * 2^-24 of that
    # times the scale, for a weight and for their sum
    check(first, want, decode_tol(want, mag) + 2 * 129 * 2.0 ** -24 * 83 * mag)
    qd = q.to(DEV)
    for _ in range(300):
        again, _ = decode(c, qd, sd, ws=ws, scale=scale, cache=cache, table=table, lens=ln)
        assert torch.equal(first, again)
    assert int(ws[:4].view(torch.int32).item()) == 0
