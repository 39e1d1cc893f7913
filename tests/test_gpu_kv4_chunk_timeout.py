"""Bounded waits of the chunk attention and of the accumulated weight that run
out: the call records SPC_ERR_TIMEOUT in its workspace's status word, ends by
itself and leaves the workspace ready, so that the next call matches again. No
GPU fault is involved: the library's test build can make a call issue none of
its copies and give up waiting after a few thousand cycles."""
import ctypes
import time

import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from sparse_kv_cache_retrieval_gb300 import _build
from sparse_kv_cache_retrieval_gb300 import binding as spc
from tests.chunk_cases import check_chunk, chunk, close, cu_of, mass, mass_tol
from tests.paged_cases import DEV, SCALE, Cache, bf16, f64

pytestmark = pytest.mark.gpu


@pytest.fixture
def hooks(monkeypatch):
    lib = ctypes.CDLL(_build.build(test_hooks=True))
    for name, (res, args) in spc.SIGNATURES.items():
        getattr(lib, name).restype, getattr(lib, name).argtypes = res, args
    lib.spc_test_starve_paged.restype = ctypes.c_int
    lib.spc_test_starve_paged.argtypes = [ctypes.c_int, ctypes.c_longlong]
    monkeypatch.setattr(spc, "_lib", lib)
    return lib


def starved(lib, call, status):
    assert lib.spc_test_starve_paged(1, 20000) == 0
    t0 = time.perf_counter()
    call()
    torch.cuda.synchronize()                        # it ends by itself
    assert time.perf_counter() - t0 < 10
    assert int(status.item()) == -4
    status.zero_()


# at most one tile of rows a request; two tiles side by side, and a request's third alone; one of a request that is cut
CASES = [(8, 2, [900, 40], [5, 1]), (8, 1, [2000, 300], [50, 20]), (4, 1, [20000], [3]), (8, 2, [4000], [200])]


@pytest.mark.parametrize("n_q,n_kv,lens,new", CASES)
def test_chunk_attention(hooks, n_q, n_kv, lens, new):
    rng = np.random.default_rng(sum(lens))
    c = Cache(rng, lens, n_kv, 64)
    q = bf16(rng, sum(new), n_q, 128).to(DEV)
    out, lse, ws = chunk(c, q, new)
    status = ws[:4].view(torch.int32)
    starved(hooks, lambda: chunk(c, q, new, ws=ws), status)
    out, lse, _ = chunk(c, q, new, ws=ws)
    check_chunk(c, q, new, out, lse)
    assert int(status.item()) == 0


@pytest.mark.parametrize("n_q,n_kv,lens,new", CASES)
def test_accumulated_weight(hooks, n_q, n_kv, lens, new):
    rng = np.random.default_rng(sum(lens))
    c = Cache(rng, lens, n_kv, 64)
    q = bf16(rng, sum(new), n_q, 128).to(DEV)
    _, lse, _ = chunk(c, q, new)
    prev = torch.from_numpy(rng.random((len(lens), n_kv, c.max_blocks * 64)).astype(np.float32)).to(DEV)
    _, ws = mass(c, q, new, lse, prev, 0.5)
    status = ws[:4].view(torch.int32)
    starved(hooks, lambda: mass(c, q, new, lse, prev, 0.5, ws=ws), status)
    got, _ = mass(c, q, new, lse, prev, 0.5, ws=ws)
    want, rel = P.attn_mass(f64(q), c.rec, c.table, c.lens, cu_of(new), f64(lse), f64(prev), 0.5, got.shape[2], SCALE)
    for b, n in enumerate(lens):
        close(got[b, :, :n], want[b, :, :n], mass_tol(want, rel)[b, :, :n], f"mass of request {b}")
    assert int(status.item()) == 0
