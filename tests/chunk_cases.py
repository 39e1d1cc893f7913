"""Helpers of the tests of chunks of new tokens over the paged 4-bit cache:
calls on a paged_cases.Cache and their tolerances."""
import numpy as np
import torch

import oracle.paged_oracle as P
from sparse_kv_cache_retrieval_gb300 import binding as spc
from tests.paged_cases import DEV, SCALE, f64, i32


def cu_of(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


def workspace(size):
    return torch.zeros(size, dtype=torch.uint8, device=DEV)


def chunk(c, q, new, out=None, lse=True, ws=None, scale=SCALE, cache=None, table=None, lens=None, cu=None, stream=None):
    """spc_kv4_chunk_attn on a Cache: (out, lse, workspace); rows are 7 before the call."""
    T, n_q = q.shape[:2]
    B = len(c.lens)
    if ws is None:
        ws = workspace(spc.spc_kv4_chunk_attn_workspace_size(T, B, n_q, c.n_kv, 128))
    if out is None:
        out = torch.full((T, n_q, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    if lse is True:
        lse = torch.full((T, n_q), 7.0, device=DEV)
    spc.spc_kv4_chunk_attn(q, torch.from_numpy(c.rec).to(DEV) if cache is None else cache,
                           i32(c.table) if table is None else table, i32(c.lens) if lens is None else lens,
                           i32(cu_of(new)) if cu is None else cu, T, B, n_q, c.n_kv, 128, c.num_blocks, c.bs, c.max_blocks,
                           scale, out, lse, ws, stream=stream)
    return out, lse, ws


def mass(c, q, new, lse, prev, keep, out=None, ws=None, scale=SCALE, cache=None, table=None, lens=None, cu=None, cap=None,
         stream=None):
    """spc_kv4_attn_mass on a Cache: (mass, workspace); entries are 7 before the call."""
    T, n_q = q.shape[:2]
    B = len(c.lens)
    cap = cap or c.max_blocks * c.bs
    if ws is None:
        ws = workspace(spc.spc_kv4_attn_mass_workspace_size(T, B, n_q, c.n_kv, 128))
    if out is None:
        out = torch.full((B, c.n_kv, cap), 7.0, device=DEV)
    spc.spc_kv4_attn_mass(q, torch.from_numpy(c.rec).to(DEV) if cache is None else cache,
                          i32(c.table) if table is None else table, i32(c.lens) if lens is None else lens,
                          i32(cu_of(new)) if cu is None else cu, lse, prev, out, T, B, n_q, c.n_kv, 128, c.num_blocks, c.bs,
                          c.max_blocks, cap, scale, keep, ws, stream=stream)
    return out, ws


# A logit is a sum of 128 products, exact in fp32 each, added in any order: it
# is off by at most 128 * 2^-24 of err = sum |q k| scale. A weight is off by that,
# relatively, and the sum of the weights too, and by 2^-22 for the exponential.
# Sums of weights run over at most 2^10 in a row (a thread's columns of a tile,
# then the tiles), 2^-14 relatively. The weights that multiply V are rounded to
# fp16, 2^-11, and the result to bf16, 2^-8 of it. Below 2^-22 of the largest
# weight fp16 has steps of 2^-32 of it (they are kept 2^8 times as large, and the
# type's last step is 2^-24): such a weight is off by up to 2^-33 of the largest,
# which is at most 1, and a row's result by that times the sum of |v| over what it
# sees. That sum counts where the weights that count meet zeros in V.
def chunk_tol(want, mag, err, vsum):
    e = 128 * 2.0 ** -24 * err[..., None]
    return 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -14 + 2.0 ** -14 + 2 * e) * mag + 2.0 ** -33 * vsum


def lse_tol(want, err):
    return 128 * 2.0 ** -24 * err + 2.0 ** -14 + 2.0 ** -22 + 2.0 ** -23 * np.abs(want)


# A sum of weights: each off by 128 * 2^-24 of (sum |q k| scale + |lse|) and 2^-22, the
# sum by 2^-14, keep * prev and the addition by 2^-24 each.
def mass_tol(want, rel):
    return 128 * 2.0 ** -24 * rel + (2.0 ** -22 + 2.0 ** -14 + 2.0 ** -23) * np.abs(want) + 1e-37


def close(got, want, tol, name):
    """Within tol where want is finite; the same infinities and NaN elsewhere."""
    got = f64(got)
    if got.size == 0:
        return
    odd = ~np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{name}: NaN at {np.argwhere(np.isnan(got) != np.isnan(want))[:4]}"
    both = odd & ~np.isnan(want)
    assert np.array_equal(got[both], want[both]), f"{name}: infinities"
    over = np.where(odd, -1.0, np.abs(np.where(odd, 0, got) - np.where(odd, 0, want)) - np.where(odd, 0, tol))
    i = np.unravel_index(np.argmax(over), over.shape)
    assert over[i] <= 0, f"{name} at {i}: got {got[i]:.9g}, want {want[i]:.9g}, tolerance {np.broadcast_to(tol, got.shape)[i]:.3g}"


def check_chunk(c, q, new, out, lse, scale=SCALE, table=None, lens=None):
    """Both outputs of a call against the oracle; rows of no request are still 7."""
    cu = cu_of(new)
    with np.errstate(invalid="ignore", over="ignore"):
        want, mag, want_lse, err, vsum = P.chunk_attention(f64(q), c.rec, c.table if table is None else table,
                                                     c.lens if lens is None else lens, cu, scale)
    n = cu[-1]
    assert np.all(f64(out[n:]) == 7)
    close(out[:n], want[:n], chunk_tol(want, mag, err, vsum)[:n], "out")
    if lse is not None:
        assert np.all(f64(lse[n:]) == 7)
        close(lse[:n], want_lse[:n], lse_tol(want_lse, err)[:n], "lse")
    return want_lse
