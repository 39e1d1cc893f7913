"""Helpers of the paged 4-bit cache tests: seeded inputs on the GPU and the
oracle's view of the same bits."""
import math

import numpy as np
import torch

import oracle.paged_oracle as P
from sparse_kv_cache_retrieval_gb300 import binding as spc

DEV = "cuda"
SCALE = 1.0 / math.sqrt(128)


def i32(a):
    return torch.tensor(np.asarray(a, np.int32), device=DEV)


def bf16(rng, *shape, scale=1.0):
    """bf16 normals on the CPU."""
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


class Cache:
    """A pool of records with each request's blocks scattered over it; every
    byte that no request owns is 0xff (codes -6, scales NaN)."""

    def __init__(self, rng, lens, n_kv, bs, spare=3, max_blocks=None, amp=1.0):
        used = [-(-n // bs) for n in lens]
        self.bs, self.n_kv, self.lens = bs, n_kv, list(lens)
        self.num_blocks = sum(used) + spare
        self.max_blocks = max_blocks or max(used + [1])
        perm = rng.permutation(self.num_blocks)
        self.table = np.full((len(lens), self.max_blocks), -1, np.int32)
        self.rec = np.full((self.num_blocks, n_kv, bs, 144), 0xff, np.uint8)
        at = 0
        for b, n in enumerate(lens):
            mine = perm[at:at + used[b]]
            at += used[b]
            self.table[b, :used[b]] = mine
            kv = P.records(rng.standard_normal((n_kv, n, 128)) * amp, rng.standard_normal((n_kv, n, 128)) * amp)
            for i, blk in enumerate(mine):
                m = min(bs, n - i * bs)
                self.rec[blk, :, :m] = kv[:, i * bs:i * bs + m]


def decode(c, q, selected=None, out=None, ws=None, scale=SCALE, cache=None, table=None, lens=None, stream=None):
    """spc_kv4_decode_attn on a Cache: (out tensor, workspace)."""
    B, n_q = q.shape[:2]
    budget = 0 if selected is None else selected.shape[2]
    if ws is None:
        ws = torch.zeros(spc.spc_kv4_decode_attn_workspace_size(B, n_q, c.n_kv, 128, c.max_blocks, c.bs, budget),
                         dtype=torch.uint8, device=DEV)
    if out is None:
        out = torch.full((B, n_q, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    spc.spc_kv4_decode_attn(q, torch.from_numpy(c.rec).to(DEV) if cache is None else cache,
                            i32(c.table) if table is None else table, i32(c.lens) if lens is None else lens,
                            selected, B, n_q, c.n_kv, 128, c.num_blocks, c.bs, c.max_blocks, budget, scale, out, ws,
                            stream=stream)
    return out, ws


# The rounding of the result to bf16 is at most 2^-8 |out|. The weights w that
# multiply V are rounded too: in fp16 by at most 2^-11 w, in bf16 by 2^-8 w, so
# the sum moves by at most that times sum w |v|. What fp32 accumulation, the
# exponential and (for the 4-bit cache) queries scaled to fp16 add stays below
# 2^-10 sum w |v|: a logit is off by at most 128 * 2^-24 * sum |q k| scale, under
# 2^-13 at these inputs, twice (numerator and sum), and 2^-22 for the exponential.
def decode_tol(want, mag):
    return 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -10) * mag


def prompt_tol(want, mag):
    return 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -10) * mag


def check(got, want, tol):
    got = f64(got)
    assert np.all(np.isfinite(got)), "not finite"
    over = np.abs(got - want) - tol
    i = np.unravel_index(np.argmax(over), over.shape)
    assert over[i] <= 0, f"at {i}: got {got[i]:.6g}, want {want[i]:.6g}, tolerance {tol[i]:.3g}"
    # the same two half steps in the 2-norm
    n = np.linalg.norm(want)
    assert np.linalg.norm(got - want) <= 2.0 ** -7 * n + 1e-30, "2-norm"
