"""Bounded waits of the paged path's attention kernels that run out: the call
records SPC_ERR_TIMEOUT in its workspace's status word, ends by itself and
leaves the workspace ready, so that the next call matches again. No GPU fault
is involved: the library's test build (libspc_testhooks.so) can make a launch
issue none of its copies and give up waiting after a few thousand cycles."""
import ctypes
import time

import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from sparse_kv_cache_retrieval_gb300 import _build
from sparse_kv_cache_retrieval_gb300 import binding as spc
from tests.paged_cases import DEV, SCALE, Cache, bf16, check, decode, decode_tol, f64, i32, prompt_tol

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


@pytest.mark.parametrize("n_q,lens,budget", [(8, [5000, 40], 0), (64, [5000, 40], 0), (8, [5000, 40], 700)])
def test_decode_attention(hooks, n_q, lens, budget):
    rng = np.random.default_rng(n_q + budget)
    c = Cache(rng, lens, 1, 64)
    q = bf16(rng, 2, n_q, 128)
    sel = None if budget == 0 else rng.integers(0, 5000, (2, 1, budget)).astype(np.int32)
    out, ws = decode(c, q.to(DEV), None if sel is None else i32(sel))
    status = ws[:4].view(torch.int32)

    def call():
        decode(c, q.to(DEV), None if sel is None else i32(sel), out=out, ws=ws)
    starved(hooks, call, status)
    call()
    want, mag = P.decode_attention(f64(q), c.rec, c.table, c.lens, sel, SCALE)
    check(out, want, decode_tol(want, mag))
    assert int(status.item()) == 0


def test_prompt_attention(hooks):
    rng = np.random.default_rng(3)
    q, k, v = (bf16(rng, 900, n, 128).to(DEV) for n in (8, 2, 2))
    cu, out = i32([0, 300, 900]), torch.zeros(900, 8, 128, dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(spc.spc_prompt_attn_workspace_size(900, 2, 8, 2, 128), dtype=torch.uint8, device=DEV)
    status = ws[:4].view(torch.int32)

    def call():
        spc.spc_prompt_attn(q, k, v, cu, 900, 2, 8, 2, 128, SCALE, out, ws)
    call()
    starved(hooks, call, status)
    call()
    want, mag = P.prompt_attention(f64(q), f64(k), f64(v), [0, 300, 900], SCALE)
    check(out, want, prompt_tol(want, mag))
    assert int(status.item()) == 0
