"""Decode attention over the 4-bit cache with a scale and queries whose product
passes fp32's range: logits that are zero stay zero, and the largest takes all."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from tests.paged_cases import DEV, Cache, check, decode, decode_tol, f64, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_q", [8, 16, 64])
@pytest.mark.parametrize("qamp,scale", [(3.0, 2e38), (1e38, 1e3), (3e38, 3.0)])
def test_scale_times_queries_beyond_fp32(n_q, qamp, scale):
    rng = np.random.default_rng(90)
    n, u = 300, np.sign(rng.standard_normal(128))
    c = Cache(rng, [n, n], 1, 64)
    k, v = np.zeros((1, n, 128)), rng.standard_normal((1, n, 128))
    rec0 = P.records(k, v)                                  # request 0: every logit is zero
    k[0, 177] = 2 * u
    rec1 = P.records(k, v)                                  # request 1: but for one position
    for b, rec in ((0, rec0), (1, rec1)):
        for i in range(-(-n // 64)):
            m = min(64, n - i * 64)
            c.rec[c.table[b, i], :, :m] = rec[:, i * 64:i * 64 + m]
    # that position takes all of the even heads and nothing of the odd ones
    q = torch.from_numpy(np.where(np.arange(n_q) % 2 == 0, 1, -1)[None, :, None] * u * qamp).to(torch.bfloat16)
    q = q.expand(2, n_q, 128).contiguous()
    sel = np.stack([np.sort(rng.choice(n, 200, replace=False)) for _ in range(2)])[:, None].astype(np.int32)
    sel[1, 0, 7] = 177
    for s in (None, sel):
        got, ws = decode(c, q.to(DEV), None if s is None else i32(s), scale=scale)
        want, mag = P.decode_attention(f64(q), c.rec, c.table, c.lens, s, scale)
        assert int(ws[:4].view(torch.int32).item()) == 0
        check(got, want, decode_tol(want, mag))
