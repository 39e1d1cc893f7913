"""The attention calls at the ends of their limits: the most requests, heads and
positions at once, and the most rows. Contexts whose table names one block over
and over have the result of that block alone; prompts are checked on rows drawn
from the whole."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from sparse_kv_cache_retrieval_gb300 import binding as spc
from tests.paged_cases import DEV, SCALE, bf16, check, decode_tol, f64, prompt_tol

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,n_kv,G,bs,full", [(64, 128, 1, 64, 262144), (64, 16, 16, 16, 262144), (64, 128, 64, 128, 262144),
                                              (64, 128, 32, 64, 2048), (1, 1, 8, 128, 262144)])
def test_decode_attention(B, n_kv, G, bs, full):
    rng = np.random.default_rng(120 + G)
    rec = P.records(rng.standard_normal((1, n_kv, bs, 128)), rng.standard_normal((1, n_kv, bs, 128)))
    cache = torch.from_numpy(rec).to(DEV)
    max_blocks = full // bs
    table = torch.zeros(B, max_blocks, dtype=torch.int32, device=DEV)
    lens = torch.full((B,), full, dtype=torch.int32, device=DEV)
    if B > 3:
        lens[1], lens[B - 1] = bs, 0                        # a short and an empty one among them
    q = bf16(rng, B, n_kv * G, 128)
    out = torch.full((B, n_kv * G, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(spc.spc_kv4_decode_attn_workspace_size(B, n_kv * G, n_kv, 128, max_blocks, bs, 0), dtype=torch.uint8,
                     device=DEV)
    spc.spc_kv4_decode_attn(q.to(DEV), cache, table, lens, None, B, n_kv * G, n_kv, 128, 1, bs, max_blocks, 0, SCALE, out, ws)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32).item()) == 0
    rows = [0, 1, B // 2, B - 1] if B > 3 else [0]
    want, mag = P.decode_attention(f64(q[rows]), rec, np.zeros((len(rows), 1), np.int32), [bs] * len(rows), None, SCALE)
    if B > 3:
        want[-1] = mag[-1] = 0
    # up to 2^13 equal blocks: an fp32 sum of that many is off by 2^-24 for each at most
    check(out[rows], want, decode_tol(want, mag) + 2.0 ** -11 * mag)


def test_prompt_attention_of_the_most_rows():
    # 2^24 rows: 61 sequences of 262144, three of other lengths, and rows behind the last
    T, n = 1 << 24, 262144
    rng = np.random.default_rng(121)
    lens = [n] * 61 + [1, n // 2 + 3, n - 5]
    lens = [lens[i] for i in rng.permutation(64)]
    cu = np.concatenate([[0], np.cumsum(lens)])
    assert cu[-1] <= T and max(lens) <= n
    g = torch.Generator(device=DEV).manual_seed(121)
    q, k, v = (torch.randn(T, 1, 128, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(3))
    out = torch.full((T, 1, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(spc.spc_prompt_attn_workspace_size(T, 64, 1, 1, 128), dtype=torch.uint8, device=DEV)
    spc.spc_prompt_attn(q, k, v, torch.tensor(cu, dtype=torch.int32, device=DEV), T, 64, 1, 1, 128, SCALE, out, ws)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32).item()) == 0
    for b in sorted({0, 33, 63, *np.argsort(lens)[:3].tolist()}):
        a, e = int(cu[b]), int(cu[b + 1])
        kb, vb = k[a:e, 0].double(), v[a:e, 0].double()
        for i in sorted({a, e - 1, int(rng.integers(a, e)), int(rng.integers(a, e))}):
            w = torch.softmax(kb[:i + 1 - a] @ q[i, 0].double() * SCALE, 0)
            want, mag = (w @ vb[:i + 1 - a]).cpu().numpy(), (w @ vb[:i + 1 - a].abs()).cpu().numpy()
            # long contexts of random values average to little: the rounding of the weights, in mag, is what is left
            assert np.all(np.abs(f64(out[i, 0]) - want) <= prompt_tol(want, mag)), (b, i - a)
    assert torch.all(out[int(cu[-1]):] == 7)


def test_rows_computed_again_over_the_longest_sequence():
    # an infinity in the last row's V: the rows of its block of keys that do not see it are computed again, which
    # takes a second or so, and no wait gives up meanwhile
    n = 262144
    g = torch.Generator(device=DEV).manual_seed(122)
    q, k, v = (torch.randn(n, m, 128, generator=g, device=DEV, dtype=torch.bfloat16) for m in (8, 1, 1))
    v[n - 1, 0, 5] = float("inf")
    out = torch.full((n, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(spc.spc_prompt_attn_workspace_size(n, 1, 8, 1, 128), dtype=torch.uint8, device=DEV)
    spc.spc_prompt_attn(q, k, v, torch.tensor([0, n], dtype=torch.int32, device=DEV), n, 1, 8, 1, 128, SCALE, out, ws)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32).item()) == 0
    odd = (~torch.isfinite(out[n - 300:].float())).nonzero()
    assert odd[:, 0].unique().tolist() == [299] and odd[:, 2].unique().tolist() == [5] and len(odd) == 8
    kd, vd = k[:, 0].double(), v[:, 0].double()
    for i in (n - 2, n - 77, n - 128, n - 129):
        w = torch.softmax(kd[:i + 1] @ q[i].double().T * SCALE, 0)
        want, mag = (w.T @ vd[:i + 1]).cpu().numpy(), (w.T @ vd[:i + 1].abs()).cpu().numpy()
        assert np.all(np.abs(f64(out[i]) - want) <= prompt_tol(want, mag)), i
