"""Measured cases of serving over the paged 4-bit cache beyond one new token a
request: attention of a chunk of new tokens, the attention weight that every
cached position has received, and the eviction of the positions that received
the least.

``own`` is set by whoever imports the module: with it ``run`` calls the
library, without it the same operators in elementary torch operations.

A 4-bit record holds one position of one KV head: 64 bytes of K codes (two
e2m1 values a byte, the lower index in the low nibble), 64 bytes of V codes,
8 e4m3 scales for K and 8 for V, one for each 16 values. A cache is
[num_blocks][n_kv][block_size][144] bytes. len[b] positions of request b are in
the cache, the last of them its new tokens' own, so that new token i of n sits
at position len[b] - n + i and sees the positions up to its own.
"""
import math

import torch

own = False

DEV = "cuda"
D = 128
REC = 144
GROUPS = (1, 2, 4, 8, 16, 32, 64)
MOST = 64 * 2048 * 65536            # (head, new token, position) triples of the largest case


def _spc():
    from sparse_kv_cache_retrieval_gb300 import binding
    return binding


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a short second turn behind a short first one: latency counts
        {"name": "chunk_turn", "op": "chunk", "B": 1, "n_q": 32, "n_kv": 8, "lo": 1017, "hi": 1017, "nlo": 17, "nhi": 17,
         "block": 64, "pad": 0, "tail": 0},
        # drafts of 4 tokens checked for 8 requests of 64K, 64 heads on 8: the cache's bytes count
        {"name": "chunk_draft", "op": "chunk", "B": 8, "n_q": 64, "n_kv": 8, "lo": 65536, "hi": 65536, "nlo": 4, "nhi": 4,
         "block": 64, "pad": 0, "tail": 0},
        # prefill chunks and single tokens of 16 requests of different lengths in one batch, queries in fused rows
        {"name": "chunk_ragged", "op": "chunk", "B": 16, "n_q": 32, "n_kv": 8, "lo": 100, "hi": 20000, "nlo": 1, "nhi": 700,
         "block": 16, "pad": 2048, "tail": 37},
        # a question of 512 tokens about a document of 32K
        {"name": "chunk_32k", "op": "chunk", "B": 1, "n_q": 32, "n_kv": 8, "lo": 32768, "hi": 32768, "nlo": 512, "nhi": 512,
         "block": 64, "pad": 0, "tail": 0},
        # the last chunk of 2048 tokens of a prompt of 64K, 64 heads on 8
        {"name": "chunk_64k", "op": "chunk", "B": 1, "n_q": 64, "n_kv": 8, "lo": 65536, "hi": 65536, "nlo": 2048, "nhi": 2048,
         "block": 64, "pad": 0, "tail": 0},
        # a decode step at the start of its context, the sums of earlier steps kept: latency
        {"name": "mass_short", "op": "mass", "B": 1, "n_q": 32, "n_kv": 8, "lo": 1000, "hi": 1000, "nlo": 1, "nhi": 1,
         "block": 64, "pad": 0, "tail": 0, "keep": 1.0},
        # a decode step of 8 requests of 64K, older steps fading
        {"name": "mass_decode", "op": "mass", "B": 8, "n_q": 64, "n_kv": 8, "lo": 65536, "hi": 65536, "nlo": 1, "nhi": 1,
         "block": 64, "pad": 0, "tail": 0, "keep": 0.96875},
        # the last 64 tokens of prompts of different lengths looking back over them
        {"name": "mass_window", "op": "mass", "B": 5, "n_q": 32, "n_kv": 8, "lo": 777, "hi": 32768, "nlo": 64, "nhi": 64,
         "block": 32, "pad": 2048, "tail": 5, "keep": 0.0},
        # every token of a prompt of 16K
        {"name": "mass_prompt", "op": "mass", "B": 1, "n_q": 32, "n_kv": 8, "lo": 16384, "hi": 16384, "nlo": 16384,
         "nhi": 16384, "block": 64, "pad": 0, "tail": 0, "keep": 0.0},
        # one request back to its budget after 64 decode steps
        {"name": "evict_step", "op": "evict", "B": 1, "n_kv": 8, "lo": 1088, "hi": 1088, "budget": 1024, "block": 64},
        # requests of different lengths, some shorter than the budget
        {"name": "evict_ragged", "op": "evict", "B": 16, "n_kv": 8, "lo": 1, "hi": 20001, "budget": 2047, "block": 16},
        # 8 prompts of 64K cut to 4096 positions a head
        {"name": "evict_64k", "op": "evict", "B": 8, "n_kv": 8, "lo": 65536, "hi": 65536, "budget": 4096, "block": 64},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("chunk", "chunk", "mass", "mass", "evict"))
    block = rng.choice((16, 32, 64, 128))
    n_kv = rng.choice((1, 2, 4, 8))
    B = _log_int(rng, 1, 32)
    if op == "evict":
        hi = _log_int(rng, 64, min(131072, 8 * 8 * 65536 // (B * n_kv)))
        return {"op": op, "B": B, "n_kv": n_kv, "lo": _log_int(rng, 1, hi), "hi": hi, "budget": _log_int(rng, 16, 4096),
                "block": block}
    n_q = n_kv * rng.choice([g for g in GROUPS if g * n_kv <= 64])
    hi = _log_int(rng, 16, min(131072, 8 * 8 * 65536 // (B * n_kv)))
    nhi = _log_int(rng, 1, max(1, min(hi, 16384, MOST // (B * n_q * hi))))
    case = {"op": op, "B": B, "n_q": n_q, "n_kv": n_kv, "lo": _log_int(rng, 1, hi), "hi": hi, "nlo": _log_int(rng, 1, nhi),
            "nhi": nhi, "block": block, "pad": rng.choice((0, 8, 2048)), "tail": rng.choice((0, 0, 37))}
    if op == "mass":
        case["keep"] = rng.choice((0.0, 0.5, 1.0))
    return case


def _lens(case):
    """Lengths and new tokens of the requests: both spread evenly over their ranges, in different orders."""
    B = case["B"]
    at = [i * 7 % B if B % 7 else i for i in range(B)]
    lens = [case["hi"] if B == 1 else case["lo"] + (case["hi"] - case["lo"]) * i // (B - 1) for i in range(B)]
    if case["op"] == "evict":
        return [(n, 0) for n in lens]
    new = [case["nhi"] if B == 1 else case["nlo"] + (case["nhi"] - case["nlo"]) * i // (B - 1) for i in at]
    return [(n, min(n, m)) for n, m in zip(lens, new)]


def _lens_of(case, seed):
    """The same in an order of the seed."""
    pairs = _lens(case)
    return [pairs[i] for i in torch.randperm(case["B"], generator=torch.Generator().manual_seed(seed)).tolist()]


# ------------------------------------------------------------------ inputs
def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _quant(x):
    """Codes (uint8 0..15) and e4m3 scales of rows [..., 128]."""
    x = x.unflatten(-1, (8, 16))
    s = (x.abs().amax(-1) / 6).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = s.float()[..., None]
    y = torch.where(sf > 0, x.abs() / sf, 0.0)
    code = ((y > 0.25).byte() + (y >= 0.75).byte() + (y > 1.25).byte() + (y >= 1.75).byte() + (y > 2.5).byte()
            + (y >= 3.5).byte() + (y > 5).byte())
    return (code + torch.signbit(x).byte() * 8).flatten(-2), s


def _records(k, v):
    kc, ks = _quant(k)
    vc, vs = _quant(v)
    return torch.cat([kc[..., 0::2] + kc[..., 1::2] * 16, vc[..., 0::2] + vc[..., 1::2] * 16,
                      ks.view(torch.uint8), vs.view(torch.uint8)], -1)


def _values(rec):
    """K and V rows in fp32 of records [..., 144]."""
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=rec.device)
    codes = rec[..., :128]
    x = lut[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    s = rec[..., 128:].contiguous().view(torch.float8_e4m3fn).float()
    x = (x.unflatten(-1, (16, 16)) * s[..., None]).flatten(-2)
    return x[..., :D], x[..., D:]


def _prepare_cache(case, seed, g, room):
    """Requests with their blocks scattered over a pool; `room` more blocks at its end."""
    B, n_kv, bs = case["B"], case["n_kv"], case["block"]
    pairs = _lens_of(case, seed)
    used = [-(-n // bs) for n, _ in pairs]
    max_blocks, n_used = max(used), sum(used) + 3
    perm = torch.randperm(n_used, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, max_blocks), -1, dtype=torch.int32, device=DEV)
    cache = torch.zeros(n_used + room, n_kv, bs, REC, dtype=torch.uint8, device=DEV)
    at = 0
    for b in range(B):
        mine = perm[at:at + used[b]]
        at += used[b]
        table[b, :used[b]] = mine
        cache[mine.long()] = _records(*torch.randn(2, used[b], n_kv, bs, D, generator=g, device=DEV))
    return {"op": case["op"], "B": B, "n_kv": n_kv, "bs": bs, "max_blocks": max_blocks, "num_blocks": n_used + room,
            "n_used": n_used, "cache": cache, "table": table, "len": _i32([n for n, _ in pairs]), "pairs": pairs}


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return _prepare_evict(case, seed, g) if case["op"] == "evict" else _prepare_attn(case, seed, g)


def _prepare_attn(case, seed, g):
    s = _prepare_cache(case, seed, g, 0)
    n_q, n_kv, B = case["n_q"], case["n_kv"], case["B"]
    cu = [0]
    for _, n in s["pairs"]:
        cu.append(cu[-1] + n)
    T = cu[-1] + case["tail"]
    # rows of their own, or at the start of wider rows (a fused projection's output); logits of a deviation of 2
    x = (2 * torch.randn(T, n_q * D + case["pad"], generator=g, device=DEV)).to(torch.bfloat16)
    s.update({"n_q": n_q, "T": T, "q": x[:, :n_q * D].unflatten(1, (n_q, D)), "cu": _i32(cu), "scale": 1.0 / math.sqrt(D),
              "max_new": max(n for _, n in s["pairs"]), "cap": s["max_blocks"] * s["bs"]})
    if case["op"] == "chunk":
        s["out"] = torch.zeros(T, n_q, D, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.zeros(T, n_q, device=DEV)
    else:
        s["keep"] = case["keep"]
        s["lse"] = _lse_of(s)
        s["prev"] = torch.rand(B, n_kv, s["cap"], generator=g, device=DEV).pow_(4)
        s["mass"] = torch.zeros(B, n_kv, s["cap"], device=DEV)
    return s


def _prepare_evict(case, seed, g):
    bs, budget, B, n_kv = case["block"], case["budget"], case["B"], case["n_kv"]
    kept_blocks = -(-min(budget, case["hi"]) // bs)
    s = _prepare_cache(case, seed, g, B * kept_blocks)
    # the kept positions go to blocks of their own (the prompt's may be shared with other requests)
    s["first"] = s["n_used"]
    table_next = torch.full_like(s["table"], -1)
    table_next[:, :kept_blocks] = (s["first"] + torch.randperm(B * kept_blocks, generator=g, device=DEV).to(torch.int32)
                                   ).view(B, kept_blocks)
    cap = s["max_blocks"] * bs
    # sums of attention weights: a few large, most small, a tenth nothing at all
    mass = torch.randn(B, n_kv, cap, generator=g, device=DEV).mul_(3).exp_()
    mass *= torch.rand(B, n_kv, cap, generator=g, device=DEV) > 0.1
    s.update({"table_next": table_next, "cap": cap, "budget": budget, "n_sink": min(4, budget // 4),
              "n_recent": min(64, budget // 4), "mass": mass, "mass_next": torch.zeros(B, n_kv, cap, device=DEV),
              "kept": torch.zeros(B, n_kv, budget, dtype=torch.int32, device=DEV), "len_next": _i32([0] * B),
              "status": _i32([0])})
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return {"chunk": _run_chunk, "mass": _run_mass, "evict": _run_evict}[s["op"]](s)


def _padded(s, dtype=torch.float32):
    """Queries [B][n_kv][G n][D] with the new tokens of each request side by side, K and V [B][n_kv][cap][D], and which
    position [B][n][cap] each new token sees."""
    B, n_kv, n, cu = s["B"], s["n_kv"], s["max_new"], s["cu"].long()
    i = torch.arange(n, device=DEV)
    q = s["q"][(cu[:-1, None] + i).clamp(max=s["T"] - 1)].to(dtype)
    q = q.unflatten(2, (n_kv, s["n_q"] // n_kv)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    rec = s["cache"][s["table"].long().clamp(min=0)].transpose(1, 2).flatten(2, 3)
    new = cu[1:] - cu[:-1]
    at = torch.where(i < new[:, None], s["len"][:, None] - new[:, None] + i, -1)
    return q, *_values(rec), torch.arange(s["cap"], device=DEV) <= at[:, :, None]


def _packed(s, x):
    """[B][n_kv][G][n]... back to the packed rows [T][n_q]..., zeros behind the last request."""
    cu = s["cu"].long()
    t = torch.arange(s["T"], device=DEV)
    b = torch.searchsorted(cu, t, right=True) - 1
    inside = b < s["B"]
    b = b.clamp(max=s["B"] - 1)
    x = x.movedim(3, 1)[b, (t - cu[b]).clamp(max=s["max_new"] - 1)].flatten(1, 2)
    return torch.where(inside.view(-1, *[1] * (x.dim() - 1)), x, 0.0)


def _logits(s, q, k, sees):
    x = torch.matmul(q.mul_(s["scale"]), k.transpose(2, 3)).unflatten(2, (-1, s["max_new"]))
    return x.masked_fill_(~sees[:, None, None], -math.inf)


def _lse_of(s):
    q, k, _, sees = _padded(s)
    x = _logits(s, q, k, sees)
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    return _packed(s, m[..., 0] + x.sub_(m).exp_().sum(-1).log_())


def _run_chunk(s):
    if own:
        spc = _spc()
        if "workspace" not in s:
            n = spc.spc_kv4_chunk_attn_workspace_size(s["T"], s["B"], s["n_q"], s["n_kv"], D)
            s["workspace"] = torch.zeros(n, dtype=torch.uint8, device=DEV)
        spc.spc_kv4_chunk_attn(s["q"], s["cache"], s["table"], s["len"], s["cu"], s["T"], s["B"], s["n_q"], s["n_kv"], D,
                               s["num_blocks"], s["bs"], s["max_blocks"], s["scale"], s["out"], s["lse"], s["workspace"])
        return s["out"], s["lse"]
    q, k, v, sees = _padded(s)
    x = _logits(s, q, k, sees)
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    z = x.sub_(m).exp_().sum(-1, keepdim=True)
    o = torch.matmul(x.flatten(2, 3), v).unflatten(2, (-1, s["max_new"])).div_(z)
    return _packed(s, o).to(torch.bfloat16), _packed(s, (m + z.log_())[..., 0])


def _run_mass(s):
    if own:
        spc = _spc()
        if "workspace" not in s:
            n = spc.spc_kv4_attn_mass_workspace_size(s["T"], s["B"], s["n_q"], s["n_kv"], D)
            s["workspace"] = torch.zeros(n, dtype=torch.uint8, device=DEV)
        spc.spc_kv4_attn_mass(s["q"], s["cache"], s["table"], s["len"], s["cu"], s["lse"], s["prev"], s["mass"], s["T"],
                              s["B"], s["n_q"], s["n_kv"], D, s["num_blocks"], s["bs"], s["max_blocks"], s["cap"],
                              s["scale"], s["keep"], s["workspace"])
        return s["mass"]
    q, k, _, sees = _padded(s)
    x = _logits(s, q, k, sees)
    cu, n = s["cu"].long(), s["max_new"]
    lse = s["lse"][(cu[:-1, None] + torch.arange(n, device=DEV)).clamp(max=s["T"] - 1)]
    lse = lse.unflatten(2, (s["n_kv"], -1)).permute(0, 2, 3, 1)
    total = x.sub_(lse[..., None]).exp_().flatten(2, 3).sum(2)
    inside = torch.arange(s["cap"], device=DEV) < s["len"][:, None]
    return torch.where(inside[:, None], total + s["keep"] * s["prev"], 0.0)


def _run_evict(s):
    if own:
        _spc().spc_kv4_evict(s["cache"], s["table"], s["table_next"], s["len"], s["len_next"], s["mass"], s["mass_next"],
                             s["kept"], s["status"], s["B"], s["n_kv"], D, s["num_blocks"], s["bs"], s["max_blocks"],
                             s["cap"], s["budget"], s["n_sink"], s["n_recent"])
        return s["cache"][s["first"]:], s["kept"], s["len_next"], s["mass_next"]
    B, n_kv, bs, cap, budget = s["B"], s["n_kv"], s["bs"], s["cap"], s["budget"]
    p = torch.arange(cap, device=DEV)
    n = s["len"].long()[:, None]
    # what is always kept comes first, what is not there last; equal sums in the order of their positions
    rank = torch.where((p < s["n_sink"]) | (p >= n - s["n_recent"]), math.inf, 0.0)
    rank = torch.where(p < n, rank, -math.inf)[:, None] + s["mass"]
    order = rank.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    order = torch.nn.functional.pad(order, (0, budget - order.shape[-1]), value=cap)
    keeps = torch.minimum(n, torch.full_like(n, budget))                # [B][1]
    i = torch.arange(budget, device=DEV)
    there = (i < keeps)[:, None]                                        # [B][1][budget]
    kept = torch.where(there, order, cap).sort(dim=-1).values
    src = kept.clamp(max=cap - 1)
    b = torch.arange(B, device=DEV)[:, None, None]
    g = torch.arange(n_kv, device=DEV)[:, None]
    rec = s["cache"][s["table"].long()[b, src // bs].clamp(min=0), g, src % bs]
    at, room = i.clamp(max=cap - 1), there & (i < cap)
    dst = s["table_next"].long()[b, (at // bs)].clamp(min=0).expand(B, n_kv, budget)
    to = (dst * n_kv + g) * bs + at % bs
    flat = s["cache"].view(-1, REC)
    flat[to[room.expand_as(to)]] = rec[room.expand_as(to)]
    mass = torch.zeros_like(s["mass"])
    m = min(budget, cap)
    mass[..., :m] = torch.where(there, s["mass"].gather(-1, src), 0.0)[..., :m]
    return (s["cache"][s["first"]:], torch.where(there, kept, -1).to(torch.int32), keeps[:, 0].to(torch.int32), mass)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    pairs, n_kv, B = _lens(case), case["n_kv"], case["B"]
    total = sum(n for n, _ in pairs)
    entries = 4 * sum(-(-n // case["block"]) for n, _ in pairs)
    if case["op"] == "evict":
        kept = sum(min(n, case["budget"]) for n, _ in pairs)
        return {"bytes": n_kv * (8 * total + kept * (2 * REC + 4)) + entries + 4 * -(-kept // case["block"]) + 8 * B, "flops": 0}
    T, n_q = sum(m for _, m in pairs), case["n_q"]
    seen = sum(m * (n - m) + m * (m + 1) // 2 for n, m in pairs)
    small = entries + 4 * (2 * B + 1) + T * n_q * (2 * D + 4)
    if case["op"] == "chunk":
        return {"bytes": total * n_kv * REC + small + T * n_q * 2 * D, "flops": 4 * D * n_q * seen}
    return {"bytes": total * n_kv * (REC // 2 + (8 if case["keep"] else 4)) + small, "flops": 2 * D * n_q * seen}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "evict":
        return None, None, None, _exact_evict(s)
    cu, bs, n_kv, G = s["cu"].tolist(), s["bs"], s["n_kv"], s["n_q"] // s["n_kv"]
    out = torch.zeros(s["T"], s["n_q"], D, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["T"], s["n_q"], dtype=torch.float64, device=DEV)
    mass = torch.zeros(s["B"], n_kv, s["cap"], dtype=torch.float64, device=DEV)
    for b, (n, m) in enumerate(s["pairs"]):
        rows = s["cache"][s["table"][b, :-(-n // bs)].long()].transpose(0, 1).flatten(1, 2)[:, :n]
        for g in range(n_kv):
            k = _exact_rows(rows[g, :, :64], rows[g, :, 128:136])
            v = _exact_rows(rows[g, :, 64:128], rows[g, :, 136:])
            if s["op"] == "mass" and s["keep"]:
                mass[b, g, :n] = s["keep"] * s["prev"][b, g, :n].double()
            for h in range(g * G, g * G + G):
                for i in range(0, m, 2048):
                    j = min(m, i + 2048)
                    at, e = slice(cu[b] + i, cu[b] + j), n - m + j
                    x = (s["q"][at, h].double() @ k[:e].T) * s["scale"]
                    later = torch.arange(e, device=DEV) > torch.arange(n - m + i, e, device=DEV)[:, None]
                    x.masked_fill_(later, -math.inf)
                    if s["op"] == "mass":
                        mass[b, g, :e] += torch.exp(x - s["lse"][at, h, None].double()).sum(0)
                        continue
                    lse[at, h] = torch.logsumexp(x, -1)
                    out[at, h] = torch.softmax(x, -1) @ v[:e]
    return mass if s["op"] == "mass" else (out, lse)


def _exact_rows(codes, scales):
    n = torch.stack([codes % 16, codes // 16], -1).flatten(-2).long()
    e, m = (n // 2) % 4, (n % 2).double()
    x = torch.where(e == 0, m / 2, torch.exp2((e - 1).double()) * (1 + m / 2)) * (1 - 2 * (n // 8).double())
    b = scales.long()
    e, m = (b // 8) % 16, (b % 8).double()
    f = torch.where(e == 0, m / 8 * 2.0 ** -6, torch.exp2((e - 7).double()) * (1 + m / 8))
    return (x.unflatten(-1, (8, 16)) * f[..., None]).flatten(-2)


def _exact_evict(s):
    """The sums behind the eviction, head by head: positions by falling sum, the lower one first."""
    after = torch.zeros(s["B"], s["n_kv"], s["cap"], dtype=torch.float64)
    mass = s["mass"].double().cpu()
    for b, (n, _) in enumerate(s["pairs"]):
        for g in range(s["n_kv"]):
            x = mass[b, g, :n]
            if n <= s["budget"]:
                after[b, g, :n] = x
                continue
            free = x[s["n_sink"]:n - s["n_recent"]]
            picked = torch.sort(-free, stable=True).indices[:s["budget"] - s["n_sink"] - s["n_recent"]]
            all_ = torch.cat([x[:s["n_sink"]], free[picked.sort().values], x[n - s["n_recent"]:]])
            after[b, g, :s["budget"]] = all_
    return after
