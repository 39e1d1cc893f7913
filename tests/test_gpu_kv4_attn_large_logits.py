"""Decode attention over the 4-bit cache with logits of any finite size: the
largest take all, equal ones share, whichever tile, warp or CTA holds them."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from tests.paged_cases import DEV, Cache, check, decode, decode_tol, f64, i32
from tests.test_gpu_kv4_attn_sink import small_weights_tol

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_q", [8, 16, 32, 64])
@pytest.mark.parametrize("top", [2.0 ** 10, 2.0 ** 24, 2.0 ** 28, 2.0 ** 33, 2.0 ** 60, 2.0 ** 110])
@pytest.mark.parametrize("n", [300, 20000])
def test_logits_of_any_finite_size(n_q, top, n):
    # logits i / 6 top for i in -6 .. 6 (exact: K's values are e2m1 times a power of two), the largest at three
    # positions far apart; the odd heads see the negatives
    rng = np.random.default_rng(91)
    u = np.sign(rng.standard_normal(128))
    c = Cache(rng, [n], 1, 64)
    step = rng.choice([0, .5, 1, 1.5, 2, 3, 4, -.5, -1, -1.5, -2, -3, -4], n)
    step[[3, n // 2, n - 2]] = 6
    step[[10, n - 1]] = -6
    k, v = u * step[None, :, None], rng.standard_normal((1, n, 128))
    # a group whose largest is below 6 would get a smaller scale; the first value of each pins it, and the
    # queries there are zero
    k[:, :, ::16] = 6
    rec = P.records(k, v)
    for i in range(-(-n // 64)):
        m = min(64, n - i * 64)
        c.rec[c.table[0, i], :, :m] = rec[:, i * 64:i * 64 + m]
    q = np.where(np.arange(n_q) % 2 == 0, 1, -1)[None, :, None] * u * 2.0
    q[:, :, ::16] = 0
    q = torch.from_numpy(q).to(torch.bfloat16)
    scale = float(np.float32(top / (6 * 2 * 120)))
    sel = np.arange(1, n, max(1, n // 4000), dtype=np.int32)[:3900]
    sel = np.concatenate([sel, [3, n - 2, 10]]).astype(np.int32)[None, None]
    for s in (None, sel):
        got, ws = decode(c, q.to(DEV), None if s is None else i32(s), scale=scale)
        want, mag = P.decode_attention(f64(q), c.rec, c.table, c.lens, s, scale)
        assert int(ws[:4].view(torch.int32).item()) == 0
        # where the largest one's V is zero, weights of 2^-100 and less of the largest are the whole result; they
        # are lost, which moves it by at most their half step, 2^-36 sum |v|
        check(got, want, decode_tol(want, mag) + small_weights_tol(c, n_q))
