"""spc_kv4_store and spc_kv4_load against the oracle: the records' bytes equal
(the rounding is a function of the exact quotient), the rows exact."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from sparse_kv_cache_retrieval_gb300 import binding as spc
from tests.paged_cases import DEV, bf16, f64, i32

pytestmark = pytest.mark.gpu


def same_records(got, want):
    """Equal bytes; the codes of a group whose scale is NaN say nothing."""
    nan = (want[..., 128:] & 127) == 127
    mask = np.repeat(nan, 8, -1)
    got, want = got.copy(), want.copy()
    got[..., :128][mask], want[..., :128][mask] = 0, 0
    assert np.array_equal(got, want)


def store(k, v, slots, num_blocks, bs):
    n_kv = k.shape[1]
    cache = torch.full((num_blocks, n_kv, bs, 144), 0x5a, dtype=torch.uint8, device=DEV)
    spc.spc_kv4_store(k, v, slots, cache, k.shape[0], n_kv, 128, num_blocks, bs)
    return cache


@pytest.mark.parametrize("T,n_kv,bs", [(1, 1, 16), (1, 8, 64), (7, 2, 32), (33, 8, 16), (300, 3, 128), (1000, 8, 64),
                                       (5000, 1, 64)])
def test_round_trip(T, n_kv, bs):
    rng = np.random.default_rng(T)
    k, v = bf16(rng, T, n_kv, 128), bf16(rng, T, n_kv, 128, scale=0.05)
    k *= torch.from_numpy(10.0 ** rng.integers(-4, 4, (T, n_kv, 1))).to(torch.bfloat16)
    num_blocks = -(-T // bs) + 2
    slots = rng.permutation(num_blocks * bs)[:T].astype(np.int32)
    cache = store(k.to(DEV), v.to(DEV), i32(slots), num_blocks, bs)
    got = cache.cpu().numpy()
    want = np.full_like(got, 0x5a)
    want[slots // bs, :, slots % bs] = P.records(f64(k), f64(v))
    same_records(got, want)
    ko = torch.full((T, n_kv, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    vo = torch.full((T, n_kv, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    spc.spc_kv4_load(cache, i32(slots), ko, vo, T, n_kv, 128, num_blocks, bs)
    wk, wv = P.values(want[slots // bs, :, slots % bs])
    assert np.array_equal(f64(ko), wk) and np.array_equal(f64(vo), wv)


def test_ties_and_special_values():
    # every e4m3 scale s, with values at the ties of e2m1 (exact in bf16 for these s) and one step beside them
    s = P.E4M3[1:127]
    rows = np.zeros((126, 128))
    steps = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5])
    for i in range(126):
        rows[i, 0] = 6 * s[i]
        rows[i, 1:8], rows[i, 8:15] = steps * s[i], -steps * s[i]
        rows[i, 16] = 6 * s[i]
        rows[i, 17:24] = steps * s[i] * (1 + 2.0 ** -7)
        rows[i, 24:31] = steps * s[i] * (1 - 2.0 ** -7)
    k = torch.from_numpy(rows).to(torch.bfloat16)[:, None]
    # scales at the ties of e4m3: largest magnitudes 6 times a midpoint
    mid = (P.E4M3[:126] + P.E4M3[1:127]) / 2
    v = torch.zeros(126, 1, 128, dtype=torch.bfloat16)
    v[:, 0, ::16] = torch.from_numpy(6 * mid).to(torch.bfloat16)[:, None]
    v[:, 0, 3::16] = torch.from_numpy(-5 * mid).to(torch.bfloat16)[:, None]
    slots = np.arange(126, dtype=np.int32)
    got = store(k.to(DEV), v.to(DEV), i32(slots), 8, 16).cpu().numpy()
    same_records(got[slots // 16, :, slots % 16], P.records(f64(k), f64(v)))


def test_extremes():
    x = torch.zeros(9, 1, 128)
    x[0, 0, 5] = float("nan")
    x[1, 0, 20], x[1, 0, 21] = float("inf"), -1.0
    x[2, 0, 40], x[2, 0, 41] = -float("inf"), float("nan")
    x[3, 0, 60] = 3e38
    x[4] = 1e-38                                            # scale 0: zeros
    x[5] = 2.0 ** -10 * 6                                   # rounds up from the tie below the smallest scale
    x[6, 0, 0] = 2689.0
    x[7] = -0.0
    x[8] = torch.linspace(-3000, 3000, 128)
    x = x.to(torch.bfloat16)
    slots = np.arange(9, dtype=np.int32)
    cache = store(x.to(DEV), x.flip(0).to(DEV), i32(slots), 1, 16)
    got = cache.cpu().numpy()[0].transpose(1, 0, 2)[:9]
    want = P.records(f64(x), f64(x.flip(0)))
    same_records(got, want)
    ko, vo = torch.zeros(9, 1, 128, dtype=torch.bfloat16, device=DEV), torch.zeros(9, 1, 128, dtype=torch.bfloat16, device=DEV)
    spc.spc_kv4_load(cache, i32(slots), ko, vo, 9, 1, 128, 1, 16)
    wk, wv = P.values(want)
    assert np.array_equal(f64(ko), wk, equal_nan=True) and np.array_equal(f64(vo), wv, equal_nan=True)


def test_every_byte_pattern_loads():
    # all codes under all scale bytes, NaN and negative scales among them
    rec = np.zeros((256, 1, 16, 144), np.uint8)
    rec[..., 128:] = np.arange(256)[:, None, None, None]
    rec[..., :128] = np.arange(128) * 2 + np.arange(16)[:, None]
    slots = np.arange(4096, dtype=np.int32)
    ko, vo = (torch.zeros(4096, 1, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    spc.spc_kv4_load(torch.from_numpy(rec).to(DEV), i32(slots), ko, vo, 4096, 1, 128, 256, 16)
    wk, wv = P.values(rec.reshape(4096, 1, 144))
    assert np.array_equal(f64(ko), wk, equal_nan=True) and np.array_equal(f64(vo), wv, equal_nan=True)


def test_slots_outside_the_cache_are_skipped():
    rng = np.random.default_rng(1)
    k = bf16(rng, 6, 2, 128).to(DEV)
    slots = np.array([-1, 5, 32, 31, -(1 << 31), (1 << 31) - 1], np.int32)
    cache = store(k, k, i32(slots), 2, 16)
    got = cache.cpu().numpy()
    want = np.full_like(got, 0x5a)
    for t, s in ((1, 5), (3, 31)):
        want[s // 16, :, s % 16] = P.records(f64(k[t]), f64(k[t]))
    same_records(got, want)
    ko, vo = (torch.full((6, 2, 128), 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    spc.spc_kv4_load(cache, i32(slots), ko, vo, 6, 2, 128, 2, 16)
    assert torch.all(ko[[0, 2, 4, 5]] == 3) and torch.all(vo[[0, 2, 4, 5]] == 3)
    assert np.array_equal(f64(ko[1]), P.values(want[0, :, 5])[0])


def test_rows_of_a_fused_projection():
    rng = np.random.default_rng(2)
    x = bf16(rng, 50, 14, 128).to(DEV)
    k, v = x[:, 8:11], x[:, 11:]
    slots = np.arange(50, dtype=np.int32)[::-1].copy()
    cache = store(k, v, i32(slots), 4, 16)
    want = P.records(f64(k), f64(v))
    got = cache.cpu().numpy()
    same_records(got[slots // 16, :, slots % 16], want)
    y = torch.full_like(x, 9.0)
    spc.spc_kv4_load(cache, i32(slots), y[:, 8:11], y[:, 11:], 50, 3, 128, 4, 16)
    assert np.array_equal(f64(y[:, 8:11]), P.values(want)[0]) and torch.all(y[:, :8] == 9)


def test_a_pool_beyond_32_bit_offsets():
    # 4.6 GB of records: block ids whose byte offset needs more than 32 bits
    bs, n_kv = 128, 1
    num_blocks = 250000
    cache = torch.empty(num_blocks, n_kv, bs, 144, dtype=torch.uint8, device=DEV)
    slots = np.array([num_blocks * bs - 1, 0, num_blocks * bs - 128, (1 << 32) // 144 + 3], np.int32)
    rng = np.random.default_rng(3)
    k, v = bf16(rng, 4, 1, 128).to(DEV), bf16(rng, 4, 1, 128).to(DEV)
    spc.spc_kv4_store(k, v, i32(slots), cache, 4, 1, 128, num_blocks, bs)
    same_records(cache.view(-1, 1, 144)[torch.from_numpy(slots).long().to(DEV)].cpu().numpy(), P.records(f64(k), f64(v)))
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    spc.spc_kv4_load(cache, i32(slots), ko, vo, 4, 1, 128, num_blocks, bs)
    assert np.array_equal(f64(ko), P.values(P.records(f64(k), f64(v)))[0])


def test_on_another_stream_and_replayed():
    rng = np.random.default_rng(5)
    k = bf16(rng, 40, 4, 128).to(DEV)
    slots = i32(np.arange(40))
    want = P.records(f64(k), f64(k))
    cache = torch.zeros(3, 4, 16, 144, dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    spc.spc_kv4_store(k, k, slots, cache, 40, 4, 128, 3, 16, stream=s)
    s.synchronize()
    flat = lambda c: c.cpu().numpy().transpose(0, 2, 1, 3).reshape(48, 4, 144)[:40]  # noqa: E731
    same_records(flat(cache), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        spc.spc_kv4_store(k, k, slots, cache, 40, 4, 128, 3, 16)
    k.neg_()
    graph.replay()
    torch.cuda.synchronize()
    same_records(flat(cache), P.records(f64(k), f64(k)))
