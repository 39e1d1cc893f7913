"""The calls over the paged 4-bit cache as a server makes them, one after the
other: a prompt's rows stored and attended in chunks, the weights of its last
tokens summed, the cache cut to its budget, the blocks given back, a next turn
and decode steps over what was kept."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from sparse_kv_cache_retrieval_gb300 import binding as spc
from tests.chunk_cases import chunk_tol, close, cu_of, lse_tol, mass_tol, workspace
from tests.paged_cases import DEV, SCALE, bf16, decode_tol, f64, i32

pytestmark = pytest.mark.gpu

B, N_Q, N_KV, BS, BLOCKS, TABLE, BUDGET, SINK, RECENT = 3, 8, 2, 16, 260, 80, 128, 4, 32
CAP = TABLE * BS


class Server:
    def __init__(self):
        self.table, self.free = i32(np.full((B, TABLE), -1)), i32(np.arange(BLOCKS)[::-1].copy())
        self.n_free, self.n_free_next, self.status = i32([BLOCKS]), i32([0]), i32([0])
        self.cache = torch.zeros(BLOCKS, N_KV, BS, 144, dtype=torch.uint8, device=DEV)
        self.len, self.len_next, self.cu = i32([0] * B), i32([0] * B), i32([0] * (B + 1))
        self.mass = torch.zeros(B, N_KV, CAP, device=DEV)
        self.kept = i32(np.zeros((B, N_KV, BUDGET)))
        # fewest rows a call: one workspace of each kind serves them all in turn
        self.ws = workspace(spc.spc_kv4_chunk_attn_workspace_size(700, B, N_Q, N_KV, 128))
        self.ws_mass = workspace(spc.spc_kv4_attn_mass_workspace_size(700, B, N_Q, N_KV, 128))
        self.ws_dec = workspace(spc.spc_kv4_decode_attn_workspace_size(B, N_Q, N_KV, 128, TABLE, BS, 0))

    def map(self, n_slots):
        slots = torch.zeros(max(1, n_slots), dtype=torch.int32, device=DEV)
        spc.spc_block_map(self.len, self.len_next, self.table, self.free, self.n_free, self.n_free_next, self.cu, slots,
                          self.status, B, TABLE, BS, BLOCKS, max(1, n_slots))
        self.n_free.copy_(self.n_free_next)
        self.len.copy_(self.len_next)
        return slots

    def turn(self, q, k, v):
        """The new tokens' rows stored, attended and weighed: (out, lse)."""
        T = q.shape[0]
        slots = self.map(T)
        spc.spc_kv4_store(k, v, slots, self.cache, T, N_KV, 128, BLOCKS, BS)
        out, lse = torch.zeros(T, N_Q, 128, dtype=torch.bfloat16, device=DEV), torch.zeros(T, N_Q, device=DEV)
        shape = (T, B, N_Q, N_KV, 128, BLOCKS, BS, TABLE)
        spc.spc_kv4_chunk_attn(q, self.cache, self.table, self.len, self.cu, *shape, SCALE, out, lse, self.ws)
        spc.spc_kv4_attn_mass(q, self.cache, self.table, self.len, self.cu, lse, self.mass, self.mass, *shape, CAP, SCALE, 1.0,
                              self.ws_mass)
        return out, lse

    def evict(self):
        spc.spc_kv4_evict(self.cache, self.table, self.table, self.len, self.len_next, self.mass, self.mass, self.kept,
                          self.status, B, N_KV, 128, BLOCKS, BS, TABLE, CAP, BUDGET, SINK, RECENT)


def test_turns_with_evictions():
    rng = np.random.default_rng(0)
    s = Server()
    k_all, v_all = [[[] for _ in range(N_KV)] for _ in range(B)], [[[] for _ in range(N_KV)] for _ in range(B)]
    mass = np.zeros((B, N_KV, CAP))
    grown, lens = [[400, 90, 0], [150, 1, 130], [1, 1, 1], [1, 0, 1], [64, 200, 30]], np.zeros(B, int)
    for turn, new in enumerate(grown):
        T = sum(new)
        q, k, v = (bf16(rng, T, n, 128).to(DEV) for n in (N_Q, N_KV, N_KV))
        before = lens.copy()
        lens = lens + new
        s.len_next.copy_(i32(lens))
        out, lse = s.turn(q, k, v)
        # the oracle's own cache of what this step sees
        rec, table, cu = s.cache.cpu().numpy(), s.table.cpu().numpy(), cu_of(new)
        for b in range(B):
            for g in range(N_KV):
                rows = P.records(f64(k[cu[b]:cu[b + 1], g]), f64(v[cu[b]:cu[b + 1], g]))
                at = np.arange(before[b], lens[b])
                assert np.array_equal(rec[table[b, at // BS], g, at % BS], rows)
                k_all[b][g].extend(rows)
                at = np.arange(lens[b])
                assert np.array_equal(rec[table[b, at // BS], g, at % BS], np.array(k_all[b][g]).reshape(-1, 144))
        want, mag, want_lse, err, vsum = P.chunk_attention(f64(q), rec, table, lens, cu, SCALE)
        close(out, want, chunk_tol(want, mag, err, vsum), "out")
        close(lse, want_lse, lse_tol(want_lse, err), "lse")
        if turn in (2, 3):                                  # a single token a request: the decode attention's result
            dec = torch.zeros(B, N_Q, 128, dtype=torch.bfloat16, device=DEV)
            qd = torch.zeros(B, N_Q, 128, dtype=torch.bfloat16, device=DEV)
            for b in range(B):
                if new[b]:
                    qd[b] = q[cu[b]]
            spc.spc_kv4_decode_attn(qd, s.cache, s.table, s.len, None, B, N_Q, N_KV, 128, BLOCKS, BS, TABLE, 0, SCALE, dec,
                                    s.ws_dec)
            for b in range(B):
                if new[b]:
                    close(dec[b], want[cu[b]], decode_tol(want[cu[b]], mag[cu[b]]), "decode")
        got = s.mass.cpu().numpy()
        for b in range(B):
            w, rel = P.attn_mass(f64(q), rec, table, lens, cu, f64(lse), mass, 1.0, CAP, SCALE)
            n = lens[b]
            close(s.mass[b, :, :n], w[b, :, :n], mass_tol(w, rel)[b, :, :n], "mass")
        mass = got.astype(np.float64)
        # the eviction goes by the sums that are there, so that its sets are the oracle's to the last position
        after = P.evict(rec, table, table, lens, got, BUDGET, SINK, RECENT)
        s.evict()
        assert np.array_equal(s.kept.cpu().numpy(), after[1]) and np.array_equal(s.len_next.cpu().numpy(), after[2])
        assert np.array_equal(s.mass.cpu().numpy(), after[3]) and np.array_equal(s.cache.cpu().numpy(), after[0])
        for b in range(B):
            for g in range(N_KV):
                k_all[b][g] = [k_all[b][g][p] for p in after[1][b, g] if p >= 0]
        s.map(0)                                            # the blocks behind the kept ones go back
        lens, mass = after[2].astype(int), after[3].astype(np.float64)
        assert int(s.n_free.item()) == BLOCKS - sum(-(-int(n) // BS) for n in lens)
        assert int(s.status.item()) == 0 and not s.ws[:4].any() and not s.ws_mass[:4].any()


def test_a_captured_step_with_eviction():
    """Decode steps in one graph: map, store, attention, weights, eviction and the blocks given back."""
    rng = np.random.default_rng(1)
    eager, graphed = Server(), Server()
    n0 = [200, 128, 40]
    q, k, v = (bf16(rng, sum(n0), n, 128).to(DEV) for n in (N_Q, N_KV, N_KV))
    for s in (eager, graphed):
        s.len_next.copy_(i32(n0))
        s.turn(q, k, v)
        s.evict()
        s.map(0)
    q, k, v = (torch.zeros(B, n, 128, dtype=torch.bfloat16, device=DEV) for n in (N_Q, N_KV, N_KV))

    def step(s):
        s.len_next.copy_(s.len + 1)
        out, lse = s.turn(q, k, v)
        s.evict()
        s.map(0)
        return out, lse
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            captured = step(graphed)
    for i in range(6):
        for t in (q, k, v):
            t.copy_(bf16(rng, *t.shape))
        want = step(eager)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(captured, want):
            assert torch.equal(x, y), i
        for name in ("cache", "mass", "len", "table", "kept", "n_free"):
            assert torch.equal(getattr(eager, name), getattr(graphed, name)), (i, name)
    assert eager.len.tolist() == [128, 128, 46]
