"""spc_prompt_attn against the float64 oracle, with the tolerance derived in
paged_cases."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from sparse_kv_cache_retrieval_gb300 import binding as spc
from tests.paged_cases import DEV, SCALE, bf16, check, f64, i32, prompt_tol

pytestmark = pytest.mark.gpu


def call(q, k, v, cu, scale=SCALE, out=None, ws=None, stream=None):
    T, n_q, _ = q.shape
    B = len(cu) - 1
    if ws is None:
        ws = torch.zeros(spc.spc_prompt_attn_workspace_size(T, B, n_q, k.shape[1], 128), dtype=torch.uint8, device=DEV)
    if out is None:
        out = torch.full((T, n_q, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    spc.spc_prompt_attn(q, k, v, cu if torch.is_tensor(cu) else i32(cu), T, B, n_q, k.shape[1], 128, scale, out, ws,
                        stream=stream)
    return out, ws


def offsets(lens, first=0):
    return [first + sum(lens[:i]) for i in range(len(lens) + 1)]


def compare(got, q, k, v, cu, scale=SCALE):
    want, mag = P.prompt_attention(f64(q), f64(k), f64(v), cu, scale)
    inside = ~np.isnan(mag[:, 0, 0])
    check(got[torch.from_numpy(inside).to(got.device)], want[inside], prompt_tol(want, mag)[inside])
    assert torch.all(got[torch.from_numpy(~inside).to(got.device)] == 7)


def run(rng, lens, n_q, n_kv, scale=SCALE, tail=0, first=0, amp=1.0):
    T = first + sum(lens) + tail
    q, k, v = (bf16(rng, T, n, 128, scale=amp).to(DEV) for n in (n_q, n_kv, n_kv))
    cu = offsets(lens, first)
    got, ws = call(q, k, v, cu, scale)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32).item()) == 0
    compare(got, q, k, v, cu, scale)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257, 384, 500, 1025])
def test_one_sequence(n):
    run(np.random.default_rng(n), [n], 4, 1)


@pytest.mark.parametrize("n_q,n_kv", [(1, 1), (3, 3), (2, 1), (8, 2), (16, 2), (16, 1), (32, 1), (64, 1), (40, 5), (128, 2)])
@pytest.mark.parametrize("n", [70, 300])
def test_head_layouts(n_q, n_kv, n):
    run(np.random.default_rng(n_q + n), [n, 13], n_q, n_kv)


@pytest.mark.parametrize("lens", [[1, 1, 1, 1], [0, 5, 0, 0, 200, 1, 0], [128, 128], [129, 127, 300, 1], [700, 3, 64, 2]])
def test_packed(lens):
    run(np.random.default_rng(len(lens)), lens, 8, 2)


def test_full_batch_of_short_and_long():
    rng = np.random.default_rng(7)
    run(rng, [int(x) for x in rng.integers(0, 90, 62)] + [900, 0], 8, 4)


def test_long_sequence():
    run(np.random.default_rng(8), [3500], 4, 2)


def test_rows_outside_the_sequences_stay():
    run(np.random.default_rng(9), [40, 200], 8, 2, tail=37, first=5)


def test_no_sequence_has_a_row():
    rng = np.random.default_rng(10)
    q = bf16(rng, 9, 4, 128).to(DEV)
    got, _ = call(q, q, q, [3, 3, 3])
    assert torch.all(got == 7)


def test_peaked_softmax():
    run(np.random.default_rng(11), [400], 4, 2, scale=2.0)


def test_maxima_that_keep_rising():
    # keys along one direction with growing size: the running maximum moves at every tile
    rng = np.random.default_rng(12)
    n = 900
    q, v = bf16(rng, n, 4, 128).to(DEV), bf16(rng, n, 1, 128).to(DEV)
    d = rng.standard_normal(128)
    k = torch.from_numpy((d * np.linspace(-3, 9, n)[:, None] + rng.standard_normal((n, 128)))[:, None]).to(torch.bfloat16).to(DEV)
    q = (q.float() + torch.from_numpy(d).float().to(DEV)).to(torch.bfloat16)
    got, _ = call(q, k, v, [0, n], 0.2)
    compare(got, q, k, v, [0, n], 0.2)


def test_rows_of_one_fused_projection():
    rng = np.random.default_rng(13)
    x = bf16(rng, 333, 14, 128).to(DEV)
    q, k, v = x[:, :8], x[:, 8:11][:, :2], x[:, 12:]
    got, _ = call(q, k, v, [0, 100, 333])
    compare(got, q, k, v, [0, 100, 333])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_later_rows_and_other_sequences_do_not_reach_a_row(bad):
    rng = np.random.default_rng(14)
    lens = [150, 201, 90]
    cu = offsets(lens)
    q, k, v = (bf16(rng, sum(lens) + 20, n, 128).to(DEV) for n in (8, 2, 2))
    want, mag = P.prompt_attention(f64(q), f64(k), f64(v), cu, SCALE)
    k[150 + 180, 1], v[150 + 180, 1] = bad, bad             # row 180 of the second sequence, KV head 1
    v[150 + 60, 0, 7] = bad                                 # one value of row 60, KV head 0
    q[150 + 199, 2] = bad                                   # one query
    k[sum(lens):], v[sum(lens):] = bad, bad                 # behind the last sequence
    got, _ = call(q, k, v, cu)
    g = f64(got)
    clean = np.zeros(g.shape, bool)
    clean[:sum(lens)] = True
    clean[330:351, 4:] = False                              # what row 180 reaches
    clean[210:351, :4, 7] = False                           # what row 60's value reaches
    clean[349, 2] = False
    assert np.all(np.isfinite(g[clean]))
    assert np.all(np.abs(g - want)[clean] <= prompt_tol(want, mag)[clean])
    assert not np.any(np.isfinite(g[210:349, :4, 7]))       # and what they reach, they reach
    assert np.all(torch.isnan(got[349, 2]).cpu().numpy())
    assert not np.any(np.isfinite(g[331:351, 4:])) or not np.isnan(bad)
    assert np.all(g[sum(lens):] == 7)


def test_values_that_are_not_finite_stay_in_their_dims():
    # dim 3 of the first row reaches every row, dim 9 of row 700 those from 700 on: the other dims, and dim 9
    # of the rows before (70 of them in its block of keys), are as if both were finite
    rng = np.random.default_rng(18)
    n = 900
    q, k, v = (bf16(rng, n, m, 128).to(DEV) for m in (4, 1, 1))
    want, mag = P.prompt_attention(f64(q), f64(k), f64(v), [0, n], SCALE)
    v[0, 0, 3], v[700, 0, 9] = float("nan"), float("inf")
    got, _ = call(q, k, v, [0, n])
    g = f64(got)
    bad = np.zeros(g.shape, bool)
    bad[:, :, 3] = True
    bad[700:, :, 9] = True
    assert not np.any(np.isfinite(g[bad]))
    assert np.all(np.abs(g - want)[~bad] <= prompt_tol(want, mag)[~bad])


def test_values_near_the_largest():
    # weights are summed before they are divided by their sum: a few hundred values of 3e38 pass fp32's range there
    rng = np.random.default_rng(19)
    n = 300
    q, k = bf16(rng, n, 2, 128).to(DEV), bf16(rng, n, 1, 128).to(DEV)
    v = (torch.from_numpy(rng.uniform(2.5, 3.3, (n, 1, 128)) * 1e38)).to(torch.bfloat16).to(DEV)
    v[:, :, 1::2] *= -1
    got, _ = call(q, k, v, [0, n])
    compare(got, q, k, v, [0, n])


def test_addresses_on_16_byte_boundaries():
    rng = np.random.default_rng(20)
    lens = [70, 333]
    q, k, v = (bf16(rng, 403 * n * 128 + 8).to(DEV)[8:].view(403, n, 128) for n in (8, 2, 2))
    out = torch.full((403 * 8 * 128 + 8,), 7.0, dtype=torch.bfloat16, device=DEV)[8:].view(403, 8, 128)
    got, _ = call(q, k, v, offsets(lens), out=out)
    compare(got, q, k, v, offsets(lens))


def test_rows_far_apart():
    # row strides that put the rows beyond 32-bit offsets
    rng = np.random.default_rng(15)
    stride = 1 << 22
    x = torch.empty(600 * stride, dtype=torch.bfloat16, device=DEV)
    rows = x.view(600, stride)[:, :10 * 128].view(600, 10, 128)
    rows.copy_(bf16(rng, 600, 10, 128))
    q, k, v = rows[:, :8], rows[:, 8:9], rows[:, 9:]
    got, _ = call(q, k, v, [0, 250, 600])
    compare(got, q.contiguous(), k.contiguous(), v.contiguous(), [0, 250, 600])


def test_same_result_every_time_and_on_another_stream():
    rng = np.random.default_rng(16)
    lens = [700, 30, 1100]
    q, k, v = (bf16(rng, sum(lens), n, 128).to(DEV) for n in (8, 2, 2))
    cu = i32(offsets(lens))
    first, ws = call(q, k, v, cu)
    for _ in range(3):
        again, _ = call(q, k, v, cu, ws=ws)
        assert torch.equal(first, again)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other, _ = call(q, k, v, cu, ws=ws)
    s.synchronize()
    assert torch.equal(first, other)


def test_captured_and_replayed_with_other_sequences():
    rng = np.random.default_rng(17)
    T = 900
    q, k, v = (bf16(rng, T, n, 128).to(DEV) for n in (8, 2, 2))
    cu = i32([0, 300, 900])
    out, ws = call(q, k, v, cu)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(q, k, v, cu, out=out, ws=ws)
    for new in ([0, 300, 900], [0, 0, 899], [10, 11, 500]):
        cu.copy_(i32(new))
        out.fill_(7)
        g.replay()
        g.replay()
        torch.cuda.synchronize()
        compare(out, q, k, v, new)
