"""Host-side checks of the calls over new tokens in the paged 4-bit cache
(chunk attention, accumulated attention weight, eviction), no GPU needed: the
oracle's pins, and every refusal of the C entry points and of the binding. Each
rejected call returns before anything is launched."""
import numpy as np
import pytest
import torch

import __graft_entry__
import oracle.paged_oracle as P
from sparse_kv_cache_retrieval_gb300 import binding as B

FAKE, FAR = 0x10000, 1 << 36


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return B.lib()


def _cache(rng, lens, n_kv, bs):
    used = [-(-n // bs) for n in lens]
    table = np.full((len(lens), max(used)), -1, np.int32)
    perm, at = rng.permutation(sum(used)), 0
    cache = np.full((sum(used), n_kv, bs, 144), 0xff, np.uint8)
    for b, n in enumerate(lens):
        table[b, :used[b]] = perm[at:at + used[b]]
        at += used[b]
        for p in range(n):
            cache[table[b, p // bs], :, p % bs] = P.records(*rng.standard_normal((2, n_kv, 128)))
    return cache, table


# ------------------------------------------------------------------ oracle pins
def test_a_single_new_token_is_the_decode_attention():
    rng = np.random.default_rng(0)
    cache, table = _cache(rng, [70, 5], 2, 16)
    q = rng.standard_normal((2, 4, 128))
    want, _ = P.decode_attention(q, cache, table, [70, 5], None, 0.1)
    out, _, lse, *_ = P.chunk_attention(q, cache, table, [70, 5], [0, 1, 2], 0.1)
    assert np.allclose(out, want, rtol=1e-12)
    k, _ = P.values(cache[table[1, 0], 1, :5])
    assert np.allclose(lse[1, 2], np.log(np.exp(k @ q[1, 2] * 0.1).sum()), rtol=1e-12)


def test_a_whole_prompt_is_the_prompt_attention_of_the_cached_values():
    rng = np.random.default_rng(1)
    cache, table = _cache(rng, [40], 2, 16)
    q = rng.standard_normal((40, 4, 128))
    rows = cache[table[0]].transpose(0, 2, 1, 3).reshape(-1, 2, 144)[:40]
    k, v = P.values(rows)
    want, _ = P.prompt_attention(q, k, v, [0, 40], 0.1)
    out, _, lse, *_ = P.chunk_attention(q, cache, table, [40], [0, 40], 0.1)
    assert np.allclose(out, want, rtol=1e-12)
    # every row's weights are a distribution: the positions' sums add up to the rows
    mass, _ = P.attn_mass(q, cache, table, [40], [0, 40], lse, np.zeros((1, 2, 48)), 0.0, 48, 0.1)
    assert np.allclose(np.nansum(mass[0], -1), 80) and np.all(np.isnan(mass[..., 40:]))
    # the last position is seen by the last token alone
    x = np.exp(np.einsum("hd,d->h", q[39, :2], k[39, 0]) * 0.1 - lse[39, :2]).sum()
    assert np.isclose(mass[0, 0, 39], x)


def test_rows_before_position_zero_and_blocks_outside_the_pool():
    rng = np.random.default_rng(2)
    cache, table = _cache(rng, [33], 1, 16)
    q = rng.standard_normal((40, 1, 128))
    out, _, lse, *_ = P.chunk_attention(q, cache, table, [33], [0, 40], 0.1)
    assert np.all(out[:7] == 0) and np.all(lse[:7] == -np.inf) and np.all(np.isfinite(lse[7:]))
    cut = table.copy()
    cut[0, 0] = -1
    out2, _, lse2, *_ = P.chunk_attention(q, cache, cut, [33], [0, 40], 0.1)
    assert np.all(out2[:23] == 0) and np.all(lse2[:23] == -np.inf) and np.all(lse2[23:] < lse[23:])


def test_evict_oracle_on_a_worked_example():
    cache = np.arange(4 * 16, dtype=np.uint8).reshape(4, 1, 16, 1).repeat(144, -1)
    table = np.array([[2, 0, -1]], np.int32)
    mass = np.zeros((1, 1, 48), np.float32)
    mass[0, 0, [3, 5, 7, 9, 20, 30]] = [1, 5, 1, np.nan, 4, 2]       # 40 and on are forced with 2 recent ones
    mass[0, 0, 6] = -3
    new, kept, nxt, after, ok = P.evict(cache, table, table, [32], mass, 6, 1, 2)
    # sink 0, recent 30 and 31, then 5, 20, and of the equal sums at 3 and 7 the lower
    assert ok and list(kept[0, 0]) == [0, 3, 5, 20, 30, 31] and nxt[0] == 6
    assert list(new[2, 0, :6, 0]) == [32, 35, 37, 4, 14, 15] and np.array_equal(new[0], cache[0])
    assert list(after[0, 0, :7]) == [0, 1, 5, 4, 2, 0, 0] and np.all(after[0, 0, 6:] == 0)
    # nothing to evict: as it was
    new, kept, nxt, after, ok = P.evict(cache, table, table, [5], mass, 6, 1, 2)
    assert ok and list(kept[0, 0]) == [0, 1, 2, 3, 4, -1] and nxt[0] == 5 and np.array_equal(new, cache)
    bad = np.array([[2, -1, 0]], np.int32)
    new, kept, nxt, after, ok = P.evict(cache, bad, table, [32], mass, 6, 1, 2)
    assert not ok and nxt[0] == 32 and np.all(kept == -1) and np.array_equal(after, mass, equal_nan=True)


# ------------------------------------------------------------------ C refusals
def _refused(fn, args, changes):
    for i, v, code in changes:
        bad = list(args)
        bad[i] = v
        assert fn(*bad) == code, (i, v)


SIZES_REFUSED = ((-1, 2, 32, 8, 128), (100, 0, 32, 8, 128), (100, 65, 32, 8, 128), (100, 2, 20, 8, 128), (100, 2, 32, 8, 64),
                 ((1 << 24) + 1, 2, 32, 8, 128), (100, 2, 2048, 64, 128), (100, 2, 32, 0, 128))
COMMON = [(0, None, -1), (1, None, -1), (2, None, -1), (3, None, -1), (4, None, -1), (0, FAKE + 8, -1), (1, FAKE + 8, -1),
          (2, FAKE + 2, -1), (3, FAKE + 1, -1), (4, FAKE + 2, -1)]


def _shapes(at, stride, scale):
    """Refusals of T, B, n_q, n_kv, d, num_blocks, block_size, max_blocks from `at` on, of the stride and the scale."""
    return [(at, -1, -2), (at, (1 << 24) + 1, -2), (at + 1, 0, -2), (at + 1, 65, -2), (at + 2, 20, -2), (at + 2, 2048, -2),
            (at + 3, 0, -2), (at + 4, 64, -2), (at + 5, 0, -2), (at + 5, 1 << 28, -2), (at + 6, 8, -2), (at + 6, 48, -2),
            (at + 7, 0, -2), (at + 7, 5000, -2), (stride, 4088, -2), (stride, 4100, -2), (stride, (1 << 32) + 8, -2),
            (scale, 0.0, -1), (scale, -1.0, -1), (scale, float("nan"), -1), (scale, float("inf"), -1), (scale, 2.5e38, -1)]


def test_chunk_attn_refusals(lib):
    ws = B.spc_kv4_chunk_attn_workspace_size(100, 2, 32, 8, 128)
    assert ws > 0 and B.spc_kv4_chunk_attn_workspace_size(0, 1, 1, 1, 128) > 0
    for bad in SIZES_REFUSED:
        assert B.spc_kv4_chunk_attn_workspace_size(*bad) == 0, bad
    ok = [FAKE, FAKE, FAKE, FAKE, FAKE, 100, 2, 32, 8, 128, 50, 64, 16, 4096, 0.1, FAKE, FAKE, FAKE, ws, None]
    _refused(lib.spc_kv4_chunk_attn, ok, COMMON + _shapes(5, 13, 14) +
             [(15, None, -1), (15, FAKE + 8, -1), (16, FAKE + 2, -1), (17, None, -5), (18, ws - 1, -5), (17, FAKE + 64, -1)])
    empty = list(ok)
    empty[0], empty[5], empty[15] = None, 0, None
    assert lib.spc_kv4_chunk_attn(*empty) == 0


def test_attn_mass_refusals(lib):
    ws = B.spc_kv4_attn_mass_workspace_size(100, 2, 32, 8, 128)
    assert ws > 0
    for bad in SIZES_REFUSED:
        assert B.spc_kv4_attn_mass_workspace_size(*bad) == 0, bad
    ok = [FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 100, 2, 32, 8, 128, 50, 64, 16, 1024, 4096, 0.1, 1.0, FAKE, ws, None]
    _refused(lib.spc_kv4_attn_mass, ok, COMMON + _shapes(8, 17, 18) +
             [(5, None, -1), (5, FAKE + 2, -1), (6, None, -1), (6, FAKE + 2, -1), (7, None, -1), (7, FAKE + 2, -1),
              (16, 1023, -2), (16, 262145, -2), (19, -0.5, -1), (19, float("nan"), -1), (19, float("inf"), -1),
              (20, None, -5), (21, ws - 1, -5), (20, FAKE + 64, -1)])


def test_evict_refusals(lib):
    ok = [FAKE] * 9 + [2, 8, 128, 50, 64, 16, 1024, 512, 4, 64, None]
    _refused(lib.spc_kv4_evict, ok,
             [(i, None, -1) for i in (0, 1, 2, 3, 4, 5, 6, 8)] + [(0, FAKE + 8, -1)] + [(i, FAKE + 2, -1) for i in range(1, 9)] +
             [(9, 0, -2), (9, 65, -2), (10, 0, -2), (10, 1025, -2), (11, 64, -2), (12, 0, -2), (12, 1 << 28, -2), (13, 20, -2),
              (14, 0, -2), (14, 5000, -2), (15, 1023, -2), (15, 262145, -2), (16, 0, -2), (16, 4097, -2), (17, -1, -2),
              (18, -1, -2), (17, 449, -2), (18, 509, -2), (17, 2 ** 31 - 1, -2)])


# ------------------------------------------------------------------ overlapping buffers
def _overlaps_refused(call, sizes, outputs, alike=()):
    """Every output moved onto each other buffer's start and end is refused; `alike` pairs may be the same."""
    far = [(i + 1) * FAR for i in range(len(sizes))]
    for i in outputs:
        for j, n in enumerate(sizes):
            if j == i:
                continue
            for at in (far[j] - (sizes[i] - 1) // 256 * 256, far[j], far[j] + (n - 1) // 256 * 256):
                if at == far[j] and ((i, j) in alike or (j, i) in alike):
                    continue
                moved = list(far)
                moved[i] = at
                assert call(moved) == -1, (i, j, hex(at))


def test_chunk_attn_refuses_overlaps(lib):
    ws = B.spc_kv4_chunk_attn_workspace_size(100, 2, 32, 8, 128)
    # q, cache, table, len, cu, out, lse, workspace
    sizes = [(99 * 5120 + 4096) * 2, 50 * 64 * 8 * 144, 2 * 16 * 4, 8, 12, 100 * 32 * 256, 100 * 32 * 4, ws]
    _overlaps_refused(lambda a: lib.spc_kv4_chunk_attn(*a[:5], 100, 2, 32, 8, 128, 50, 64, 16, 5120, 0.1, *a[5:], ws, None),
                      sizes, (5, 6, 7))


def test_attn_mass_refuses_overlaps(lib):
    ws = B.spc_kv4_attn_mass_workspace_size(100, 2, 32, 8, 128)
    # q, cache, table, len, cu, lse, mass_prev, mass_next, workspace
    mass = 2 * 8 * 1024 * 4
    sizes = [(99 * 5120 + 4096) * 2, 50 * 64 * 8 * 144, 2 * 16 * 4, 8, 12, 100 * 32 * 4, mass, mass, ws]
    _overlaps_refused(lambda a: lib.spc_kv4_attn_mass(*a[:8], 100, 2, 32, 8, 128, 50, 64, 16, 1024, 5120, 0.1, 1.0, a[8], ws,
                                                      None), sizes, (7, 8), alike=((7, 6),))


def test_evict_refuses_overlaps(lib):
    # cache, table, table_next, len, len_next, mass, mass_next, kept, status
    mass = 2 * 8 * 1024 * 4
    sizes = [50 * 64 * 8 * 144, 128, 128, 8, 8, mass, mass, 2 * 8 * 512 * 4, 4]

    def call(a):
        return lib.spc_kv4_evict(*a, 2, 8, 128, 50, 64, 16, 1024, 512, 4, 64, None)
    _overlaps_refused(call, sizes, (0, 4, 6, 7, 8), alike=((6, 5),))
    far = [(i + 1) * FAR for i in range(9)]
    assert call(far[:2] + [far[1] + 64] + far[3:]) == -1               # tables that are neither one nor apart


# ------------------------------------------------------------------ binding refusals
def test_binding_refuses_wrong_tensors(lib):
    i32 = torch.zeros(64, dtype=torch.int32)
    q = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    cache = torch.zeros(2, 8, 16, 144, dtype=torch.uint8)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    sums = torch.zeros(1, 8, 32)

    def chunk(q=FAKE, cache=FAKE, table=FAKE, out=FAKE, lse=FAKE, ws=ws, cu=FAKE):
        B.spc_kv4_chunk_attn(q, cache, table, FAKE, cu, 4, 1, 8, 8, 128, 2, 16, 2, 0.1, out, lse, ws, stream=0)

    def mass(lse=FAKE, prev=FAKE, mass=FAKE):
        B.spc_kv4_attn_mass(FAKE, FAKE, FAKE, FAKE, FAKE, lse, prev, mass, 4, 1, 8, 8, 128, 2, 16, 2, 32, 0.1, 1.0, FAKE, 1 << 30,
                            stream=0)

    def evict(kept=FAKE, status=FAKE, mass=FAKE):
        B.spc_kv4_evict(FAKE, FAKE, FAKE, FAKE, FAKE, mass, FAKE, kept, status, 1, 8, 128, 2, 16, 2, 32, 8, 0, 0, stream=0)

    for fn, bad in ((chunk, dict(q=q.float())), (chunk, dict(q=q[:3])), (chunk, dict(q=q[:, :, ::2])), (chunk, dict(q=q)),
                    (chunk, dict(cache=cache[:1])), (chunk, dict(cache=cache.float())), (chunk, dict(table=i32[:1])),
                    (chunk, dict(out=q.float())), (chunk, dict(lse=q)), (chunk, dict(lse=sums[..., :2])), (chunk, dict(cu=i32[:1])),
                    (chunk, dict(ws=ws)), (mass, dict(lse=q)), (mass, dict(prev=sums.double())), (mass, dict(mass=sums[:, :7])),
                    (mass, dict(mass=sums)), (evict, dict(kept=sums)), (evict, dict(kept=i32[:63])), (evict, dict(status=sums)),
                    (evict, dict(mass=i32))):
        with pytest.raises(ValueError):
            fn(**bad)
    with pytest.raises(B.SpcError) as e:
        B.spc_kv4_evict(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, 1, 8, 64, 2, 16, 2, 32, 8, 0, 0, stream=0)
    assert e.value.status == -2
