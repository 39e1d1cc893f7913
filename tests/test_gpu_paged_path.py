"""The paged 4-bit path as a serving loop runs it: prompts are admitted from
their lengths alone, attended over and written into the cache in 4 bits; then
decode steps append one token a request and attend over the cache; one request
ends and its blocks serve another. Checked against the oracle at every step."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from sparse_kv_cache_retrieval_gb300 import binding as spc
from tests.paged_cases import DEV, SCALE, Cache, bf16, check, decode, decode_tol, f64, i32, prompt_tol

pytestmark = pytest.mark.gpu
B, N_Q, N_KV, BS, MB, NUM = 3, 16, 2, 16, 12, 30


class Requests:
    def __init__(self):
        self.rng = np.random.default_rng(40)
        self.table, self.free = np.full((B, MB), -1, np.int32), self.rng.permutation(NUM).astype(np.int32)
        self.n_free, self.lens = NUM, [0] * B
        self.rec = np.zeros((NUM, N_KV, BS, 144), np.uint8)          # the oracle's cache
        self.d = dict(table=i32(self.table), free=i32(self.free), n=[i32([NUM]), i32([0])], status=i32([0]),
                      len=i32([0] * B), cache=torch.full((NUM, N_KV, BS, 144), 0xff, dtype=torch.uint8, device=DEV),
                      ws=torch.zeros(spc.spc_kv4_decode_attn_workspace_size(B, N_Q, N_KV, 128, MB, BS, 0),
                                     dtype=torch.uint8, device=DEV))
        self.turn = 0

    def grow(self, nxt):
        """Lengths -> slots and cu_seqlens; rows for the new positions stored in 4 bits."""
        d, i = self.d, self.turn % 2
        self.turn += 1
        n = max(1, sum(max(0, b - a) for a, b in zip(self.lens, nxt)))
        slots, cu, lens_next = torch.empty(n, dtype=torch.int32, device=DEV), torch.empty(B + 1, dtype=torch.int32, device=DEV), i32(nxt)
        spc.spc_block_map(d["len"], lens_next, d["table"], d["free"], d["n"][i], d["n"][1 - i], cu, slots, d["status"],
                          B, MB, BS, NUM, n)
        d["len"] = lens_next
        x = bf16(self.rng, n, N_Q + 2 * N_KV, 128).to(DEV)
        q, k, v = x[:, :N_Q], x[:, N_Q:N_Q + N_KV], x[:, N_Q + N_KV:]
        spc.spc_kv4_store(k, v, slots, d["cache"], n, N_KV, 128, NUM, BS)
        self.table, self.free, self.n_free, wcu, wslots, ok = P.block_map(self.lens, nxt, self.table, self.free,
                                                                          self.n_free, BS, n)
        assert ok
        self.lens = list(nxt)
        for t, s in enumerate(wslots):
            if s >= 0:
                self.rec[s // BS, :, s % BS] = P.records(f64(k[t]), f64(v[t]))
        torch.cuda.synchronize()
        assert int(d["status"].item()) == 0
        assert np.array_equal(slots.cpu().numpy(), wslots) and np.array_equal(cu.cpu().numpy(), wcu)
        assert int(d["n"][1 - i].item()) == self.n_free
        return q, k, v, cu, wcu

    def prompt(self, nxt):
        q, k, v, cu, wcu = self.grow(nxt)
        out = torch.zeros(q.shape[0], N_Q, 128, dtype=torch.bfloat16, device=DEV)
        ws = torch.zeros(spc.spc_prompt_attn_workspace_size(q.shape[0], B, N_Q, N_KV, 128), dtype=torch.uint8, device=DEV)
        spc.spc_prompt_attn(q, k, v, cu, q.shape[0], B, N_Q, N_KV, 128, SCALE, out, ws)
        want, mag = P.prompt_attention(f64(q), f64(k), f64(v), wcu, SCALE)
        check(out, want, prompt_tol(want, mag))

    def step(self, nxt):
        self.grow(nxt)
        d = self.d
        q = bf16(self.rng, B, N_Q, 128)
        out = torch.zeros(B, N_Q, 128, dtype=torch.bfloat16, device=DEV)
        spc.spc_kv4_decode_attn(q.to(DEV), d["cache"], d["table"], d["len"], None, B, N_Q, N_KV, 128, NUM, BS, MB, 0,
                                SCALE, out, d["ws"])
        want, mag = P.decode_attention(f64(q), self.rec, self.table, self.lens, None, SCALE)
        check(out, want, decode_tol(want, mag))


def test_prompts_decode_steps_and_a_new_request():
    r = Requests()
    r.prompt([100, 47, 0])
    for _ in range(3):
        r.step([n + (n > 0) for n in r.lens])
    r.prompt([0, r.lens[1], 170])               # the first request ends, a third comes in, the second waits
    for _ in range(4):
        r.step([n + (n > 0) for n in r.lens])
    # what the cache holds, read back as rows
    n = r.lens[2]
    slots = np.array([r.table[2, p // BS] * BS + p % BS for p in range(n)], np.int32)
    k, v = (torch.zeros(n, N_KV, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    spc.spc_kv4_load(r.d["cache"], i32(slots), k, v, n, N_KV, 128, NUM, BS)
    wk, wv = P.values(r.rec[slots // BS, :, slots % BS])
    assert np.array_equal(f64(k), wk) and np.array_equal(f64(v), wv)


def test_calls_on_three_streams_at_once():
    # each with a workspace of its own; every result the same as alone
    rng = np.random.default_rng(41)
    c = Cache(rng, [3000, 900, 5000], 1, 64)
    lens = [700, 1300]
    q, k, v = (bf16(rng, sum(lens), n, 128).to(DEV) for n in (16, 2, 2))
    cu = i32([0, 700, 2000])
    cache, table, ln = torch.from_numpy(c.rec).to(DEV), i32(c.table), i32(c.lens)

    def prompt(stream, out, ws):
        spc.spc_prompt_attn(q, k, v, cu, 2000, 2, 16, 2, 128, SCALE, out, ws, stream=stream)

    def attend(n_q):
        qd = bf16(rng, 3, n_q, 128).to(DEV)
        return lambda stream, out, ws: decode(c, qd, out=out, ws=ws, cache=cache, table=table, lens=ln, stream=stream)

    calls = [(prompt, (2000, 16, 128), spc.spc_prompt_attn_workspace_size(2000, 2, 16, 2, 128))]
    for n_q in (8, 64):
        calls.append((attend(n_q), (3, n_q, 128), spc.spc_kv4_decode_attn_workspace_size(3, n_q, 1, 128, c.max_blocks, 64, 0)))
    runs = []
    for f, shape, size in calls:
        s, ws = torch.cuda.Stream(), torch.zeros(size, dtype=torch.uint8, device=DEV)
        alone = torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
        s.wait_stream(torch.cuda.current_stream())
        f(s, alone, ws)
        s.synchronize()
        runs.append((f, s, ws, alone, [torch.zeros_like(alone) for _ in range(20)]))
    torch.cuda.synchronize()
    for i in range(20):
        for f, s, ws, _, outs in runs:
            f(s, outs[i], ws)
    torch.cuda.synchronize()
    for _, _, ws, alone, outs in runs:
        assert int(ws[:4].view(torch.int32).item()) == 0
        assert all(torch.equal(alone, o) for o in outs)
