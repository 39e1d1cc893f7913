"""Host-side checks of the paged 4-bit cache calls (no GPU needed): the
oracle's own pins, and every refusal of the C entry points and of the binding.
Each rejected call returns before anything is launched."""
import numpy as np
import pytest
import torch

import __graft_entry__
import oracle.paged_oracle as P
from sparse_kv_cache_retrieval_gb300 import binding as B

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return B.lib()


# ------------------------------------------------------------------ oracle pins
def test_e4m3_table_matches_torch():
    b = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(b), np.isnan(P.E4M3))
    assert np.array_equal(b[~np.isnan(b)], P.E4M3[~np.isnan(b)])


def test_quantise_rounds_to_nearest_even():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 128)) * 10.0 ** rng.integers(-3, 3, (50, 1))
    codes, sb = P.quantise(x)
    s = np.repeat(P.E4M3[sb], 16, -1)
    y = np.where(s > 0, np.abs(x) / np.where(s > 0, s, 1), 0)
    got = np.abs(P.E2M1[codes])
    # no entry of the table is nearer, and ties sit on an even code
    best = np.abs(np.minimum(y, 6)[..., None] - P.E2M1[:8]).min(-1)
    assert np.allclose(np.abs(np.minimum(y, 6) - got), best, atol=0, rtol=1e-12)
    ties = np.zeros((1, 128))
    ties[0, :9] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -2.5]
    c, sb = P.quantise(ties)
    assert P.E4M3[sb[0, 0]] == 1
    assert list(P.E2M1[c[0, :9]]) == [6, 0, 1, 1, 2, 2, 4, 4, -2]
    # the largest of a group keeps its scale's rounding: e4m3 of 1.0625 is the even 1.0
    ties[0, 0] = 6 * 1.0625
    assert P.E4M3[P.quantise(ties)[1][0, 0]] == 1
    ties[0, 0] = 6 * 1.1875
    assert P.E4M3[P.quantise(ties)[1][0, 0]] == 1.25


def test_records_round_trip_and_special_values():
    x = np.zeros((5, 128))
    x[0, :16], x[1, 0], x[2, 3], x[3, 0] = 1e-5, np.nan, -np.inf, 5000.0
    k, v = P.values(P.records(x, x[::-1]))
    assert np.all(k[0] == 0) and np.isnan(k[1, 0]) and k[2, 3] == -2688 and k[3, 0] == 2688
    assert np.array_equal(v[::-1], k, equal_nan=True)


def test_block_map_oracle_on_a_worked_example():
    # blocks of 16: request 0 ends (3 blocks go onto the stack), request 1 grows from 16 to 40 (2 blocks come off it)
    table = np.array([[7, 5, 3, -1], [9, -1, -1, -1]], np.int32)
    free = np.array([1, 2, 0, 0, 0, 0, 0, 0, 0, 0], np.int32)
    t, f, n, cu, slots, ok = P.block_map([33, 16], [0, 40], table, free, 2, 16, 30)
    assert ok and n == 3 and list(f[:5]) == [1, 2, 7, 5, 3]
    assert list(t[1]) == [9, 3, 5, -1] and list(t[0]) == [7, 5, 3, -1]
    assert list(cu) == [0, 0, 24]
    assert list(slots) == [3 * 16 + i for i in range(16)] + [5 * 16 + i for i in range(8)] + [-1] * 6


# ------------------------------------------------------------------ C refusals
def _refused(fn, args, changes):
    for i, v, code in changes:
        bad = list(args)
        bad[i] = v
        assert fn(*bad) == code, (i, v)


def test_block_map_refusals(lib):
    ok = [FAKE, FAKE, FAKE, FAKE, FAKE, FAKE + 64, FAKE, FAKE, FAKE, 4, 16, 64, 100, 50, None]
    _refused(lib.spc_block_map, ok,
             [(i, None, -1) for i in range(9)] + [(i, FAKE + 2, -1) for i in range(9)] +
             [(5, FAKE, -1), (9, 0, -2), (9, 65, -2), (10, 0, -2), (10, 4097, -2), (11, 48, -2), (11, 8, -2),
              (12, 0, -2), (12, 1 << 25, -2), (13, 0, -2), (13, (1 << 24) + 1, -2)])


def test_kv4_rows_refusals(lib):
    ok = [FAKE, FAKE, 1024, 1024, FAKE, FAKE, 10, 8, 128, 100, 64, None]
    _refused(lib.spc_kv4_store, ok,
             [(0, None, -1), (1, None, -1), (4, None, -1), (5, None, -1), (0, FAKE + 8, -1), (1, FAKE + 2, -1),
              (4, FAKE + 1, -1), (5, FAKE + 8, -1), (2, 1016, -2), (3, 1028, -2), (6, -1, -2), (6, (1 << 24) + 1, -2),
              (7, 0, -2), (8, 64, -2), (9, 0, -2), (10, 256, -2), (9, 1 << 25, -2)])
    assert lib.spc_kv4_store(None, None, 1024, 1024, None, None, 0, 8, 128, 100, 64, None) == 0    # nothing to do
    ok = [FAKE, FAKE, FAKE, FAKE, 1024, 1024, 10, 8, 128, 100, 64, None]
    _refused(lib.spc_kv4_load, ok, [(0, None, -1), (1, None, -1), (2, None, -1), (3, None, -1), (0, FAKE + 8, -1),
                                    (2, FAKE + 8, -1), (4, 1000, -2), (5, 1025, -2), (8, 96, -2), (10, 0, -2)])


def test_kv4_decode_attn_refusals(lib):
    ws = B.spc_kv4_decode_attn_workspace_size(2, 32, 8, 128, 16, 64, 0)
    assert ws > 0
    for bad in ((0, 32, 8, 128, 16, 64, 0), (65, 32, 8, 128, 16, 64, 0), (2, 30, 8, 128, 16, 64, 0),
                (2, 32, 8, 64, 16, 64, 0), (2, 32, 8, 128, 0, 64, 0), (2, 32, 8, 128, 5000, 64, 0),
                (2, 32, 8, 128, 16, 63, 0), (2, 129, 129, 128, 16, 64, 0), (2, 32, 8, 128, 16, 64, 5000), (2, 32, 8, 128, 16, 64, -1)):
        assert B.spc_kv4_decode_attn_workspace_size(*bad) == 0, bad
    ok = [FAKE, FAKE, FAKE, FAKE, None, 2, 32, 8, 128, 100, 64, 16, 0, 0.1, FAKE, FAKE, ws, None]
    nan, inf = float("nan"), float("inf")
    _refused(lib.spc_kv4_decode_attn, ok,
             [(0, None, -1), (1, None, -1), (2, None, -1), (3, None, -1), (14, None, -1), (0, FAKE + 8, -1),
              (1, FAKE + 8, -1), (14, FAKE + 8, -1), (2, FAKE + 2, -1), (4, FAKE, -1), (12, 64, -1), (5, 0, -2),
              (5, 65, -2), (6, 24, -2), (8, 64, -2), (9, 0, -2), (10, 20, -2), (11, 5000, -2), (13, 0.0, -1),
              (13, -1.0, -1), (13, nan, -1), (13, inf, -1), (15, None, -5), (16, ws - 1, -5), (15, FAKE + 64, -1)])
    sel = list(ok)
    sel[4], sel[12], sel[16] = FAKE, 4097, 1 << 40
    assert lib.spc_kv4_decode_attn(*sel) == -2


def test_prompt_attn_refusals(lib):
    ws = B.spc_prompt_attn_workspace_size(100, 2, 32, 8, 128)
    assert ws > 0 and B.spc_prompt_attn_workspace_size(0, 1, 1, 1, 128) > 0
    for bad in ((-1, 2, 32, 8, 128), (100, 0, 32, 8, 128), (100, 65, 32, 8, 128), (100, 2, 20, 8, 128),
                (100, 2, 32, 8, 64), ((1 << 24) + 1, 2, 32, 8, 128), (100, 2, 2048, 64, 128)):
        assert B.spc_prompt_attn_workspace_size(*bad) == 0, bad
    ok = [FAKE, FAKE, FAKE, FAKE, 100, 2, 32, 8, 128, 4096, 1024, 1024, 0.1, FAKE, FAKE, ws, None]
    _refused(lib.spc_prompt_attn, ok,
             [(i, None, -1) for i in (0, 1, 2, 3, 13)] + [(i, FAKE + 8, -1) for i in (0, 1, 2, 13)] +
             [(3, FAKE + 2, -1), (4, -1, -2), (5, 0, -2), (5, 65, -2), (6, 20, -2), (8, 64, -2), (9, 4088, -2),
              (9, 4100, -2), (10, 1000, -2), (11, 1028, -2), (12, 0.0, -1), (12, float("nan"), -1),
              (12, float("inf"), -1), (14, None, -5), (15, ws - 1, -5), (14, FAKE + 64, -1)])
    empty = [None, None, None, None, 0, 2, 32, 8, 128, 4096, 1024, 1024, 0.1, None, FAKE, ws, None]
    assert lib.spc_prompt_attn(*empty) == 0


def test_attention_refuses_overlapping_output_and_overflowing_scale(lib):
    # addresses that no call reads: every one of these is refused before a launch
    far = FAKE + (1 << 30)
    dec = [FAKE, far, far, far, None, 2, 32, 8, 128, 100, 64, 16, 0, 0.1, FAKE + (1 << 28), FAKE, 1 << 40, None]
    for out in (FAKE, FAKE + 2 * 32 * 256 - 16, FAKE - 2 * 32 * 256 + 16):
        assert lib.spc_kv4_decode_attn(*dec[:14], out, *dec[15:]) == -1, out
    assert lib.spc_kv4_decode_attn(*dec[:13], 2.5e38, *dec[14:]) == -1
    pro = [FAKE, far, 2 * far, FAKE, 100, 2, 32, 8, 128, 8192, 1024, 1024, 0.1, 4 * far, FAKE, 1 << 40, None]
    q_end = FAKE + (99 * 8192 + 4096) * 2
    for out in (FAKE, q_end - 16, far, far + (99 * 1024 + 1024) * 2 - 16, 2 * far - 100 * 8192 + 16):
        assert lib.spc_prompt_attn(*pro[:13], out, *pro[14:]) == -1, out
    assert lib.spc_prompt_attn(*pro[:12], 2.5e38, *pro[13:]) == -1


# ------------------------------------------------------------------ binding refusals
def test_binding_refuses_wrong_tensors(lib):
    k = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    cache = torch.zeros(2, 8, 16, 144, dtype=torch.uint8)
    slots = torch.zeros(4, dtype=torch.int32)

    def store(k=k, v=k, slots=slots, cache=cache, T=4, **kw):
        B.spc_kv4_store(k, v, slots, cache, T, 8, 128, 2, 16, stream=0, **kw)

    for bad in (dict(k=k.float()), dict(k=k.half()), dict(k=k[:, :4]), dict(k=k.transpose(0, 1)), dict(T=5),
                dict(k=k.view(4, 1024)), dict(k=k[:, :, ::2]), dict(k_stride=2048), dict(k=k)):
        with pytest.raises(ValueError):
            store(**bad)                                    # (the last one: right shape, but host memory)
    B._device()
    fused = torch.zeros(4, 20, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        store(k=fused[:, :8])                               # row stride and shape pass, host memory does not
    for name, t, dt, n in (("cache", cache.float(), B._BYTES, 1), ("cache", cache[:1], B._BYTES, cache.numel()),
                           ("slot_map", slots.long(), B._I32, 1), ("slot_map", slots[:3], B._I32, 4),
                           ("block_table", slots.view(2, 2).t(), B._I32, 4), ("slot_map", slots, B._I32, 4)):
        with pytest.raises(ValueError, match=name):
            B._dev(name, t, dt, n, -2)
    with pytest.raises(B.SpcError) as e:
        B.spc_prompt_attn(FAKE, FAKE, FAKE, FAKE, 4, 1, 8, 8, 64, 0.1, FAKE, FAKE, 1 << 20, stream=0)
    assert e.value.status == -2


def test_row_strides_come_from_the_tensor():
    class OnDevice:                                         # a tensor's face without its memory
        dtype, device = torch.bfloat16, torch.device("cuda:0")

        def __init__(self, shape, strides):
            self.shape, self._s = shape, strides

        def stride(self):
            return self._s

        def get_device(self):
            return 0

        def data_ptr(self):
            return FAKE

    B._device()
    assert B._rows("k", OnDevice((4, 8, 128), (2048, 128, 1)), 4, 8, 128, None, 0) == (FAKE, 2048)
    assert B._rows("k", OnDevice((4, 1, 128), (512, 7, 1)), 4, 1, 128, None, 0) == (FAKE, 512)
    assert B._rows("k", OnDevice((1, 2, 128), (3, 128, 1)), 1, 2, 128, None, 0) == (FAKE, 256)
    for shape, strides, dev in (((4, 8, 128), (128, 512, 1), 0), ((4, 8, 128), (2048, 128, 1), 1),
                                ((4, 8, 128), (2048, 128, 1), -2)):
        with pytest.raises(ValueError):
            B._rows("k", OnDevice(shape, strides), 4, 8, 128, None, dev)
    assert B._rows("k", FAKE, 4, 8, 128, None, -2) == (FAKE, 1024)
    assert B._rows("k", FAKE, 4, 8, 128, 4096, -2) == (FAKE, 4096)
