"""Float64 oracle of the paged 4-bit cache path -- TEST INFRASTRUCTURE ONLY.

Plain numpy from the definitions: block tables and slot maps, the e2m1 / e4m3
rounding of K and V rows, decode attention over a paged cache, causal
attention over packed prompts, and for chunks of new tokens over the cache their
attention, the weights that its positions receive, and the eviction by those.
Shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

RECORD = 144
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def _e4m3_table():
    v = np.zeros(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if b & 127 == 127:
            x = np.nan
        v[b] = -x if b & 128 else x
    return v


E4M3 = _e4m3_table()


def _nearest_even(x, table):
    """Index of the nearest entry of an ascending table, ties to the even index."""
    hi = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = x - table[lo], table[hi] - x
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(x >= table[-1], len(table) - 1, np.where(up, hi, lo))


def quantise(rows):
    """(codes uint8 [..., 128], scale bytes uint8 [..., 8]) of float64 rows."""
    x = np.asarray(rows, np.float64).reshape(rows.shape[:-1] + (8, 16))
    a = np.abs(x).max(-1)                                  # NaN stays NaN
    sb = _nearest_even(np.where(np.isnan(a), 0, np.minimum(a / 6, 448)), E4M3[:127]).astype(np.uint8)
    s = E4M3[sb]
    sb = np.where(np.isnan(a), 127, sb).astype(np.uint8)
    with np.errstate(invalid="ignore", divide="ignore"):
        y = np.where(s[..., None] > 0, np.abs(x) / s[..., None], 0.0)
    code = _nearest_even(np.minimum(np.nan_to_num(y, nan=0, posinf=6), 6), E2M1[:8])
    code = code + 8 * np.signbit(x)
    return code.reshape(rows.shape).astype(np.uint8), sb


def records(k, v):
    kc, ks = quantise(k)
    vc, vs = quantise(v)
    return np.concatenate([kc[..., ::2] | kc[..., 1::2] << 4, vc[..., ::2] | vc[..., 1::2] << 4, ks, vs], -1)


def values(rec):
    """Float64 K and V rows of records [..., 144]."""
    out = []
    for c0, s0 in ((0, 128), (64, 136)):
        c = rec[..., c0:c0 + 64]
        x = np.stack([E2M1[c & 15], E2M1[c >> 4]], -1).reshape(rec.shape[:-1] + (8, 16))
        out.append((x * E4M3[rec[..., s0:s0 + 8]][..., None]).reshape(rec.shape[:-1] + (128,)))
    return out


def block_map(lens, lens_next, table, free, n_free, bs, n_slots):
    """(table, free, n_free, cu, slots, ok) after the call, on copies."""
    B, max_blocks = table.shape
    nb = lambda n: -(-int(n) // bs)  # noqa: E731
    fail = (table.copy(), free.copy(), n_free, np.zeros(B + 1, np.int32), np.full(n_slots, -1, np.int32), False)
    if not 0 <= n_free <= len(free) or any(not 0 <= n <= max_blocks * bs for n in list(lens) + list(lens_next)):
        return fail
    t, f = table.copy(), free.copy()
    given = [int(table[b, i]) for b in range(B) for i in range(nb(lens_next[b]), nb(lens[b]))]
    if n_free + len(given) > len(free):
        return fail
    f[n_free:n_free + len(given)] = given
    top = n_free + len(given)
    cu, slots = [0], []
    for b in range(B):
        for i in range(nb(lens[b]), nb(lens_next[b])):
            if top == 0:
                return fail
            top -= 1
            t[b, i] = f[top]
        slots += [int(t[b, p // bs]) * bs + p % bs for p in range(int(lens[b]), int(lens_next[b]))]
        cu.append(len(slots))
    if len(slots) > n_slots:
        return fail
    slots = np.array(slots + [-1] * (n_slots - len(slots)), np.int32)
    return t, f, top, np.array(cu, np.int32), slots, True


def softmax_rows(q, k, v, scale):
    """[m][d] queries over [n][d] keys: (out [m][d], sum of |weights| |v|)."""
    if len(k) == 0:
        return np.zeros_like(q), np.zeros_like(q)
    x = (q @ k.T) * scale
    w = np.exp(x - x.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    return w @ v, w @ np.abs(v)


def decode_attention(q, cache, table, lens, selected, scale):
    """q [B][n_q][d] float64, cache uint8 [num_blocks][n_kv][bs][144], selected
    [B][n_kv][budget] or None. Returns (out, bound) with bound = sum w |v|."""
    num_blocks, n_kv, bs, _ = cache.shape
    B, n_q, d = q.shape
    out, mag = np.zeros((B, n_q, d)), np.zeros((B, n_q, d))
    G = n_q // n_kv
    for b in range(B):
        L = max(0, min(int(lens[b]), table.shape[1] * bs))
        for g in range(n_kv):
            pos = np.arange(L) if selected is None else selected[b, g].astype(np.int64)
            pos = pos[(pos >= 0) & (pos < L)]
            blk = table[b, pos // bs].astype(np.int64)
            ok = (blk >= 0) & (blk < num_blocks)
            k, v = values(cache[blk[ok], g, (pos % bs)[ok]])
            hs = slice(g * G, (g + 1) * G)
            out[b, hs], mag[b, hs] = softmax_rows(q[b, hs], k, v, scale)
    return out, mag


def prompt_attention(q, k, v, cu, scale):
    """q [T][n_q][d], k, v [T][n_kv][d] float64. Returns (out, bound); rows
    outside every sequence are NaN in `bound`."""
    T, n_q, d = q.shape
    G = n_q // k.shape[1]
    out, mag = np.zeros((T, n_q, d)), np.full((T, n_q, d), np.nan)
    for s, e in zip(cu[:-1], cu[1:]):
        n = e - s
        if n == 0:
            continue
        later = np.arange(n)[None, :] > np.arange(n)[:, None]
        for h in range(n_q):
            x = (q[s:e, h] @ k[s:e, h // G].T) * scale
            x[later] = -np.inf
            w = np.exp(x - x.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            out[s:e, h] = w @ v[s:e, h // G]
            mag[s:e, h] = w @ np.abs(v[s:e, h // G])
    return out, mag


def _seen(cache, table_row, L, P):
    """The positions 0 .. P of a request of L whose block is in the pool, with their blocks."""
    pos = np.arange(max(0, min(L, P + 1)))
    blk = table_row[pos // cache.shape[2]].astype(np.int64)
    ok = (blk >= 0) & (blk < cache.shape[0])
    return pos[ok], blk[ok]


def chunk_attention(q, cache, table, lens, cu, scale):
    """New tokens q [T][n_q][d] (float64), request b's last cu[b + 1] - cu[b]
    positions. Returns (out, bound, lse, err, vsum): bound = sum w |v|, err = the
    largest sum |q k| scale of a row's logits, vsum = sum |v| of what a row sees;
    NaN in rows of no request."""
    num_blocks, n_kv, bs, _ = cache.shape
    T, n_q, d = q.shape
    G = n_q // n_kv
    out, mag = np.full((T, n_q, d), np.nan), np.full((T, n_q, d), np.nan)
    lse, err, vsum = np.full((T, n_q), np.nan), np.full((T, n_q), np.nan), np.full((T, n_q, d), np.nan)
    for b in range(len(lens)):
        L, n = max(0, min(int(lens[b]), table.shape[1] * bs)), cu[b + 1] - cu[b]
        for g in range(n_kv):
            pos, blk = _seen(cache, table[b], L, L)
            k, v = values(cache[blk, g, pos % bs])
            for i in range(n):
                m = int(np.searchsorted(pos, L - n + i, side="right"))
                t, hs = cu[b] + i, slice(g * G, (g + 1) * G)
                out[t, hs], mag[t, hs] = softmax_rows(q[t, hs], k[:m], v[:m], scale)
                err[t, hs], lse[t, hs], vsum[t, hs] = 0, -np.inf, np.abs(v[:m]).sum(0)
                if m:
                    x = (q[t, hs] @ k[:m].T) * scale
                    lse[t, hs] = x.max(-1) + np.log(np.exp(x - x.max(-1, keepdims=True)).sum(-1))
                    err[t, hs] = (np.abs(q[t, hs]) @ np.abs(k[:m]).T).max(-1) * scale
    return out, mag, lse, err, vsum


def attn_mass(q, cache, table, lens, cu, lse, prev, keep, cap, scale):
    """(mass [B][n_kv][cap], rel): what spc_kv4_attn_mass writes, NaN where it
    writes nothing, and rel = the sum of weight * (sum |q k| scale + |lse|)."""
    num_blocks, n_kv, bs, _ = cache.shape
    G, B = q.shape[1] // n_kv, len(lens)
    mass, rel = np.full((B, n_kv, cap), np.nan), np.zeros((B, n_kv, cap))
    for b in range(B):
        L, n = max(0, min(int(lens[b]), table.shape[1] * bs)), cu[b + 1] - cu[b]
        for g in range(n_kv):
            mass[b, g, :L] = keep * prev[b, g, :L] if keep else 0
            for i in range(n):
                pos, blk = _seen(cache, table[b], L, L - n + i)
                k, _ = values(cache[blk, g, pos % bs])
                for h in range(g * G, (g + 1) * G):
                    y = lse[cu[b] + i, h]
                    if len(pos) == 0 or y == -np.inf:
                        continue
                    row = q[cu[b] + i, h]
                    w = np.exp((k @ row) * scale - y)
                    mass[b, g, pos] += w
                    rel[b, g, pos] += w * ((np.abs(k) @ np.abs(row)) * scale + abs(y))
    return mass, rel


def evict(cache, table, table_next, lens, mass, budget, n_sink, n_recent):
    """(cache, kept, len_next, mass_next, ok) after the call, on copies."""
    num_blocks, n_kv, bs, _ = cache.shape
    new, B = cache.copy(), len(lens)
    kept, after, len_next, ok = np.full((B, n_kv, budget), -1, np.int32), mass.copy(), np.zeros(B, np.int32), True
    for b in range(B):
        L = max(0, min(int(lens[b]), table.shape[1] * bs))
        K = min(L, budget)
        used = np.concatenate([table[b, :-(-L // bs)], table_next[b, :-(-K // bs)]])
        if np.any((used < 0) | (used >= num_blocks)):
            len_next[b], ok = L, False
            continue
        len_next[b] = K
        for g in range(n_kv):
            s = np.nan_to_num(np.maximum(mass[b, g, :L].astype(np.float64), 0), nan=0.0, posinf=np.inf)
            s[:n_sink] = s[max(0, L - n_recent):] = np.inf
            forced = np.zeros(L, bool)
            forced[:n_sink] = forced[max(0, L - n_recent):] = True
            order = np.lexsort((np.arange(L), -s, ~forced))
            pos = np.sort(order[:K])
            kept[b, g, :K] = pos
            i = np.arange(K)
            new[table_next[b, i // bs], g, i % bs] = cache[table[b, pos // bs], g, pos % bs]
            after[b, g, :K], after[b, g, K:L] = mass[b, g, pos], 0
    return new, kept, len_next, after, ok


__all__ = ["RECORD", "E2M1", "E4M3", "quantise", "records", "values", "block_map", "decode_attention",
           "prompt_attention", "softmax_rows", "chunk_attention", "attn_mass", "evict"]
