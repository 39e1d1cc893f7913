"""Decode attention over the 4-bit cache where one position takes nearly all the
weight and has a V of zero (an attention sink): the result is what the small
weights of all the others make of their V, so none of them may be lost, and their
roundings must not add up."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from tests.paged_cases import DEV, Cache, check, decode, decode_tol, f64, i32

pytestmark = pytest.mark.gpu


def sink_case(seed, lens, n_q, n_kv, gap, spread, at=0, bs=64):
    """(cache, q, scale): position `at` of every context about `gap` nats above the others, whose logits
    spread by about `spread` nats, and its V zero."""
    rng = np.random.default_rng(seed)
    c = Cache(rng, lens, n_kv, bs)
    u = np.sign(rng.standard_normal(128))
    q = torch.from_numpy(2 * u + 0.25 * rng.standard_normal((len(lens), n_q, 128))).to(torch.bfloat16)
    scale = gap / 1024                                      # q . (4 u) = 8 * 128
    # the others: along q by +-w, which 16 values of one magnitude a group hold exactly enough
    for b, n in enumerate(lens):
        w = spread / scale / 256
        k = u * (rng.choice([-1.0, 1.0], (n_kv, n, 1)) * w * rng.random((n_kv, n, 1))) + 1e-3
        k[:, at] = 4 * u
        v = rng.standard_normal((n_kv, n, 128)) + 0.5
        v[:, at] = 0
        rec = P.records(k, v)
        for i in range(-(-n // bs)):
            m = min(bs, n - i * bs)
            c.rec[c.table[b, i], :, :m] = rec[:, i * bs:i * bs + m]
    return c, q, scale


def small_weights_tol(c, n_q):
    """decode_tol counts on weights with 11 bits. Fp16 has them down to 2^-14 and steps of 2^-24 below; the weights
    are kept at least 2^11 times those against the running maximum, so that a step is at most 2^-35 of the largest,
    and the n positions' half steps come to at most 2^-36 sum |v|."""
    tol = np.zeros((len(c.lens), n_q, 128))
    for b, n in enumerate(c.lens):
        pos = np.arange(n)
        blk = c.table[b, pos // c.bs]
        ok = (blk >= 0) & (blk < c.num_blocks)
        _, v = P.values(c.rec[blk[ok], :, (pos % c.bs)[ok]])                    # [positions][n_kv][128]
        tol[b] = 2.0 ** -36 * np.repeat(np.abs(v).sum(0), n_q // c.n_kv, 0)
    return tol


def compare(c, q, scale, selected=None):
    got, ws = decode(c, q.to(DEV), None if selected is None else i32(selected), scale=scale)
    want, mag = P.decode_attention(f64(q), c.rec, c.table, c.lens, selected, scale)
    assert int(ws[:4].view(torch.int32).item()) == 0
    check(got, want, decode_tol(want, mag) + small_weights_tol(c, q.shape[1]))


@pytest.mark.parametrize("n_q", [4, 16, 32, 64])
@pytest.mark.parametrize("gap", [10, 14, 16, 18])
@pytest.mark.parametrize("spread", [0.0, 1.0])
def test_one_context(n_q, gap, spread):
    c, q, scale = sink_case(80 + gap, [4096], n_q, 1, gap, spread)
    compare(c, q, scale)


@pytest.mark.parametrize("n_q,n_kv", [(8, 1), (64, 1), (64, 2)])
@pytest.mark.parametrize("gap", [14, 18])
def test_long_contexts(n_q, n_kv, gap):
    c, q, scale = sink_case(81 + gap, [65536, 300], n_q, n_kv, gap, 0.0)
    compare(c, q, scale)


@pytest.mark.parametrize("n_q", [8, 32])
@pytest.mark.parametrize("lens", [[200], [31], [130] * 30])
def test_contexts_that_one_cta_holds(n_q, lens):
    c, q, scale = sink_case(82, lens, n_q, 1, 16, 0.0, bs=16)
    compare(c, q, scale)


@pytest.mark.parametrize("n_q", [8, 32])
@pytest.mark.parametrize("at", [1, 2047, 4095])
def test_the_large_one_comes_late(n_q, at):
    # what was summed before is scaled down by 2^-26, in fp32
    c, q, scale = sink_case(83, [4096], n_q, 1, 18, 0.5, at=at)
    compare(c, q, scale)


@pytest.mark.parametrize("n_q", [8, 16, 32, 64])
@pytest.mark.parametrize("gap", [14, 18])
def test_selected(n_q, gap):
    rng = np.random.default_rng(84)
    c, q, scale = sink_case(84, [9000, 5000], n_q, 1, gap, 0.0)
    sel = np.stack([np.sort(np.concatenate([[0], 1 + rng.choice(n - 1, 4095, replace=False)])) for n in c.lens])
    compare(c, q, scale, sel[:, None].astype(np.int32))
