"""The decode attention's rarer branches for every kind of group: one head tile
(8 heads), two (16), and the tcgen05 kernel (32, 64; four head tiles where
positions are selected). Maxima that are found late, that rise in every tile or
in one, tiles where nothing counts, and what must not count."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from tests.gpu_cases import ScoreRun, check_score_call, oracle_score, workload
from tests.paged_cases import DEV, SCALE, Cache, bf16, check, decode, decode_tol, f64, i32
from tests.test_gpu_kv4_attn_sink import small_weights_tol

pytestmark = pytest.mark.gpu
GROUPS = [4, 8, 16, 32, 64]


def run(c, q, selected=None, scale=SCALE):
    got, ws = decode(c, q.to(DEV), None if selected is None else i32(selected), scale=scale)
    want, mag = P.decode_attention(f64(q), c.rec, c.table, c.lens, selected, scale)
    assert int(ws[:4].view(torch.int32).item()) == 0
    # decode_tol counts on logits off by 2^-13. A logit is a sum of 128 products whose magnitudes add up to at most A;
    # each addition is off by at most 2^-24 A, the product with the factor by as much: twice 129 * 2^-24 A, for a
    # weight and for their sum.
    k = np.abs(P.values(c.rec[c.table[(c.table >= 0) & (c.table < c.num_blocks)]])[0])
    k = np.where(np.isnan(k), 0, k).reshape(-1, 128)
    A = scale * (np.abs(f64(q)).max((0, 1)) * k).sum(-1).max()
    check(got, want, decode_tol(want, mag) + 2 * 129 * 2.0 ** -24 * A * mag + small_weights_tol(c, q.shape[1]))
    return got


def fill(c, b, k, v):
    rec = P.records(k, v)
    n = k.shape[1]
    for i in range(-(-n // c.bs)):
        m = min(c.bs, n - i * c.bs)
        c.rec[c.table[b, i], :, :m] = rec[:, i * c.bs:i * c.bs + m]


def along(rng, n, size, n_q, lean=1.0):
    """Keys of the given sizes along a direction of signs, and queries that lean on it."""
    u = np.sign(rng.standard_normal(128))
    k = u * np.asarray(size)[None, :, None] + 0.1 * rng.standard_normal((1, n, 128))
    q = torch.from_numpy(lean * u + 0.3 * rng.standard_normal((1, n_q, 128))).to(torch.bfloat16)
    return k, q


@pytest.mark.parametrize("n_q", GROUPS)
@pytest.mark.parametrize("n", [500, 3000, 25000])
@pytest.mark.parametrize("nats", [8.0, 100.0])
def test_maxima_that_rise_all_along(n_q, n, nats):
    # logits grow by `nats` over the context and rise again and again: over several tiles of one CTA (500, 3000),
    # of a run (25000), with the largest last
    rng = np.random.default_rng(100 + n_q)
    c = Cache(rng, [n], 1, 64)
    k, q = along(rng, n, np.linspace(-3, 3, n), n_q)
    fill(c, 0, k, rng.standard_normal((1, n, 128)))
    run(c, q, scale=nats / 768)
    budget = min(n, 4096)
    sel = np.sort(rng.choice(n, budget, replace=False)).astype(np.int32)[None, None]
    run(c, q, sel, scale=nats / 768)
    run(c, q, sel[:, :, ::-1].copy(), scale=nats / 768)


@pytest.mark.parametrize("n_q", GROUPS)
@pytest.mark.parametrize("at", [127, 128, 400, 1999])
def test_one_late_maximum(n_q, at):
    # in one tile, for the even heads alone
    rng = np.random.default_rng(101 + n_q)
    n = 2000
    c = Cache(rng, [n], 1, 32)
    size = np.zeros(n)
    size[at] = 3
    k, q = along(rng, n, size, n_q)
    q[:, 1::2] = bf16(rng, 1, n_q // 2, 128)
    fill(c, 0, k, rng.standard_normal((1, n, 128)))
    run(c, q, scale=20 / 384)
    sel = np.sort(np.concatenate([[at], rng.choice(np.delete(np.arange(n), at), 999, replace=False)]))
    run(c, q, sel[None, None].astype(np.int32), scale=20 / 384)


@pytest.mark.parametrize("n_q", GROUPS)
@pytest.mark.parametrize("gone", [(0, 1), (0, 3), (3, 5), (0, 23), (5, 24), (0, 24)])
def test_tiles_where_nothing_counts(n_q, gone):
    # 3000 positions, 24 tiles of 128: those of a span have no block; the first to count is late, or none is
    rng = np.random.default_rng(102 + n_q)
    c = Cache(rng, [3000, 700], 1, 64)
    c.table[0, 2 * gone[0]:2 * gone[1]] = rng.choice([-1, c.num_blocks, 1 << 30])
    c.table[1, 4:6] = -1
    got = run(c, bf16(rng, 2, n_q, 128))
    if gone == (0, 24):
        assert torch.all(got[0] == 0)
    sel = np.stack([np.sort(rng.choice(n, 600, replace=False)) for n in (3000, 700)])[:, None].astype(np.int32)
    run(c, bf16(rng, 2, n_q, 128), sel)


@pytest.mark.parametrize("n_q", GROUPS)
def test_every_second_tile_counts_and_maxima_rise(n_q):
    rng = np.random.default_rng(103 + n_q)
    n = 9000
    c = Cache(rng, [n], 1, 128)
    k, q = along(rng, n, np.linspace(-3, 3, n), n_q)
    fill(c, 0, k, rng.standard_normal((1, n, 128)))
    c.table[0, ::2] = -1
    run(c, q, scale=60 / 768)


@pytest.mark.parametrize("n_q", GROUPS)
def test_what_lies_behind_the_context_does_not_count(n_q):
    # every byte behind the lengths is 0xff: codes -6 under NaN scales
    rng = np.random.default_rng(104)
    c = Cache(rng, [70, 1, 0, 1300], 2, 64, max_blocks=25)
    c.table[c.table < 0] = c.num_blocks - 1
    run(c, bf16(rng, 4, 2 * n_q, 128))


@pytest.mark.parametrize("n_q", GROUPS)
@pytest.mark.parametrize("bs", [16, 64, 128])
def test_lengths_beyond_the_table_and_below_zero(n_q, bs):
    rng = np.random.default_rng(105)
    c = Cache(rng, [5 * bs, 5 * bs], 1, bs)
    q = bf16(rng, 2, n_q, 128)
    c.lens = [1000000, -3]
    got, _ = decode(c, q.to(DEV))
    want, mag = P.decode_attention(f64(q), c.rec, c.table, c.lens, None, SCALE)
    check(got, want, decode_tol(want, mag))
    assert torch.all(got[1] == 0)


@pytest.mark.parametrize("n_q", GROUPS)
@pytest.mark.parametrize("qscale", [1e-30, 1e-6, 1e4, 1e30])
def test_queries_of_any_size(n_q, qscale):
    rng = np.random.default_rng(106)
    q = bf16(rng, 2, 2 * n_q, 128)
    q[0, 3] *= 2.0 ** -12                                   # heads of one group differ by far
    q[1, n_q - 1] = 0
    q = (q.float() * qscale).to(torch.bfloat16)
    c = Cache(rng, [400, 900], 2, 64)
    run(c, q, scale=SCALE / qscale)
    sel = np.stack([np.stack([np.sort(rng.choice(n, 300, replace=False)) for _ in range(2)]) for n in (400, 900)])
    run(c, q, sel.astype(np.int32), scale=SCALE / qscale)


@pytest.mark.parametrize("n_q", GROUPS)
def test_one_head_of_a_group_is_not_finite(n_q):
    # a query of NaN or infinities spoils its own head and no other
    rng = np.random.default_rng(107)
    c = Cache(rng, [1500], 1, 64)
    q = bf16(rng, 1, n_q, 128)
    want, mag = P.decode_attention(f64(q), c.rec, c.table, c.lens, None, SCALE)
    bad = {1: float("nan"), 2: float("inf")}
    for h, x in bad.items():
        q[0, h, 5] = x
    got, _ = decode(c, q.to(DEV))
    keep = [h for h in range(n_q) if h not in bad]
    check(got[:, keep], want[:, keep], decode_tol(want, mag)[:, keep])
    assert not torch.isfinite(got[0, list(bad)].float()).all(-1).any()


@pytest.mark.parametrize("n_q", GROUPS)
def test_the_same_call_gives_the_same_bits(n_q):
    rng = np.random.default_rng(108)
    c = Cache(rng, [9000, 17, 2500], 2, 64)
    q = bf16(rng, 3, 2 * n_q, 128).to(DEV)
    sel = i32(rng.integers(0, 2500, (3, 2, 700)))
    cache, table, lens = torch.from_numpy(c.rec).to(DEV), i32(c.table), i32(c.lens)
    for s in (None, sel):
        first, ws = decode(c, q, s, cache=cache, table=table, lens=lens)
        for _ in range(30):
            again, _ = decode(c, q, s, ws=ws, cache=cache, table=table, lens=lens)
            assert torch.equal(first, again)


@pytest.mark.parametrize("n_q,n_kv", [(16, 2), (32, 1), (64, 1)])
def test_over_the_positions_that_a_retrieval_head_selected(n_q, n_kv):
    # a step of sparse decoding: spc_score_select picks the positions from its own keys, and the attention reads them
    # out of the 4-bit cache that holds the same requests; the selection tensor goes from one call to the other
    lens = (1500, 129, 700, 40)
    cfg = workload(name="kv4", B=4, lens=lens, n_q=n_q, n_kv=n_kv, H=256, budget=96, steps=2)
    head = ScoreRun(cfg)
    K0, rng = head.inp.K_dlm.copy(), np.random.default_rng(109)
    c = Cache(rng, lens, n_kv, 64)
    for t in range(2):
        gq, gs, gsel, glen, _ = head.call(t, 0)
        oq, _, _, olens, os_all, osel = oracle_score(cfg, K0, head.inp.lens, head.inp.x[t], head.inp.Wq, head.inp.Wk, False)
        check_score_call(cfg, gq, gs, gsel, glen, oq, olens, os_all, osel)
        q = bf16(rng, 4, n_q, 128)
        got, ws = decode(c, q.to(DEV), head.sel, lens=head.len)
        want, mag = P.decode_attention(f64(q), c.rec, c.table, lens, gsel, SCALE)
        assert int(ws[:4].view(torch.int32).item()) == 0
        check(got, want, decode_tol(want, mag))
