"""Cases and plain forms of the 8-bit cache operators: the step plan, the insert and the attention.

A serving step of a grouped-query layer beside the compressed layers: the step's
requests get their cache blocks and their rows' slots (csa.step_plan), the new keys
and values go into an e4m3 cache with one scale for each block of tokens and head
(csa.kv8_store), and the queries attend to that cache (csa.kv8_attn), with capped
scores, a bias by distance, a window, documents or a prefix.

`run` computes a case in its plain form (elementary torch operations, in 32 bits), or
with the library's calls where `own` is true.  A case's lengths come from the case
alone (so `work` knows them); every other input comes from the seed.
"""

import numpy as np
import torch

own = False

TINY = 2.0 ** -100  # the smallest scale of a block


# ------------------------------------------------------------------ cases


def listed():
    return [
        # One decode step of 64 sequences at the contexts of the c4a decode workload: a
        # plan is a few microseconds of latency before the step's first kernel.
        plan("plan_decode_b64", 64, 32768, 65536, 1, 1, 256, 11),
        # A large ragged batch, prompts and single tokens together, some requests with
        # nothing to do in this step; blocks of 64 tokens.
        plan("plan_ragged_b2000", 2000, 0, 20000, 0, 97, 64, 12),
        # The insert of one decode step: 64 sequences, 8 key heads of 128, blocks of 256
        # tokens (the library's logical block).
        store("store_decode_b64", 64, 32768, 65536, 1, 1, 8, 128, 256, "bf16", 21),
        # Eight prompt chunks of 2048 tokens at unaligned starts.
        store("store_chunks_8x2048", 8, 4096, 131072, 2048, 2048, 8, 128, 256, "bf16", 22),
        # fp32 rows of an odd layout: 3 heads of 80, blocks of 16 tokens, ragged prompts.
        store("store_ragged_f32", 37, 0, 900, 1, 300, 3, 80, 16, "f32", 23),
        # The smallest call: one sequence, a short context, 4 query heads a key head.
        attn("attn_decode_b1_500", 1, 517, 517, 1, 1, 32, 8, 128, 64, "bf16", 31),
        # The decode workload's batch: 32 sequences, contexts in [32768, 65536], 64 query
        # heads over 8 key heads.
        attn("attn_decode_b32_64k", 32, 32768, 65536, 1, 1, 64, 8, 128, 256, "bf16", 32),
        # One long sequence (the context of the c128a decode workload) with capped scores:
        # the cache is split over the whole GPU.
        attn("attn_decode_b1_128k_cap", 1, 131071, 131071, 1, 1, 64, 8, 128, 256, "bf16", 33, softcap=50.0),
        # Many ragged sequences of a windowed layer with a bias by distance, the first
        # tokens always visible; 64 dims, blocks of 16, up to 3 new tokens a sequence.
        attn("attn_window_bias_b128", 128, 0, 8192, 1, 3, 24, 3, 64, 16, "bf16", 34, window=1024, bias=True, prefix=8),
        # Two prompt chunks of 2048 tokens behind 4k and 16k of context, capped scores.
        attn("attn_chunks_2x2048_cap", 2, 4096, 16384, 2048, 2048, 64, 8, 128, 256, "bf16", 35, softcap=30.0),
        # Packed documents: ragged prompts whose rows see their own document alone, some
        # rows nothing at all, a prefix seen in both directions; single tokens among them.
        attn("attn_docs_ragged_b12", 12, 0, 3000, 1, 700, 32, 4, 128, 32, "bf16", 36, docs=True, prefix=64),
        # fp32 queries of an odd layout (heads of 96, 3 query heads a key head).
        attn("attn_ragged_f32", 5, 0, 700, 1, 40, 12, 4, 96, 32, "f32", 37, bias=True),
    ]


def plan(name, reqs, cached_lo, cached_hi, new_lo, new_hi, block, lens):
    return _named(name, {"op": "plan", "reqs": reqs, "cached_lo": cached_lo, "cached_hi": cached_hi, "new_lo": new_lo,
                         "new_hi": new_hi, "block": block, "lens": lens})


def store(name, reqs, cached_lo, cached_hi, new_lo, new_hi, kv_heads, dim, block, dtype, lens):
    return _named(name, {"op": "store", "reqs": reqs, "cached_lo": cached_lo, "cached_hi": cached_hi, "new_lo": new_lo,
                         "new_hi": new_hi, "kv_heads": kv_heads, "dim": dim, "block": block, "dtype": dtype, "lens": lens})


def attn(name, reqs, cached_lo, cached_hi, new_lo, new_hi, heads, kv_heads, dim, block, dtype, lens, softcap=0.0, window=0,
         bias=False, docs=False, prefix=0):
    return _named(name, {"op": "attn", "reqs": reqs, "cached_lo": cached_lo, "cached_hi": cached_hi, "new_lo": new_lo,
                         "new_hi": new_hi, "heads": heads, "kv_heads": kv_heads, "dim": dim, "block": block, "dtype": dtype,
                         "lens": lens, "softcap": softcap, "window": window, "bias": bias, "docs": docs, "prefix": prefix})


def _named(name, case):
    return case if name is None else dict(case, name=name)


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(np.exp(rng.uniform(np.log(lo), np.log(hi + 1)))))))


def draw(rng):
    lens = rng.randrange(1 << 30)
    op = rng.choice(["plan", "store", "store", "attn", "attn", "attn"])
    block = rng.choice([16, 32, 64, 128, 256])
    if op == "plan":
        reqs = _log(rng, 1, 2000)
        return plan(None, reqs, 0, _log(rng, 1, 20000), 0, _log(rng, 1, max(1, 190000 // reqs)), block, lens)
    if op == "store":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        reqs, kv_heads, dim = _log(rng, 1, 128), rng.choice([1, 2, 3, 4, 5, 8]), 16 * rng.randint(2, 12)
        most = min(2048, (1 << 27) // (reqs * kv_heads * dim * 4 * (2 if dtype == "f32" else 1)))
        return store(None, reqs, 0, _log(rng, 1, 20000), 1, _log(rng, 1, max(1, most)), kv_heads, dim, block, dtype, lens)
    extra = {"softcap": rng.choice([0.0, 0.0, 30.0]), "window": rng.choice([0, 0, _log(rng, 1, 4096)]), "bias": rng.random() < 0.3,
             "docs": rng.random() < 0.2, "prefix": rng.choice([0, 0, _log(rng, 1, 200)])}
    kv_heads, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8, 16])
    if rng.random() < 0.15:  # fp32, or head sizes that are not a power of two
        return attn(None, _log(rng, 1, 8), 0, _log(rng, 1, 1000), 1, _log(rng, 1, 32), kv_heads * min(group, 8), kv_heads,
                    rng.choice([32, 48, 80, 96, 112, 160, 192]), block, rng.choice(["f32", "bf16"]), lens, **extra)
    dim = rng.choice([64, 128, 128, 256])
    if rng.random() < 0.5:  # single tokens, or a few
        reqs = _log(rng, 1, 128)
        hi = _log(rng, 16, min(131072, (1 << 21) // reqs))
        return attn(None, reqs, hi // 2, hi, 1, rng.choice([1, 1, 1, 2, 4]), kv_heads * group, kv_heads, dim, block, "bf16", lens, **extra)
    reqs, hi = _log(rng, 1, 12), _log(rng, 16, 8192)
    most = max(1, (1 << 28) // (reqs * kv_heads * group * (hi + 1024)))
    return attn(None, reqs, 0, hi, 1, _log(rng, 1, min(1024, most)), kv_heads * group, kv_heads, dim, block, "bf16", lens, **extra)


# ------------------------------------------------------------------ inputs


def _lengths(case):
    """(tokens stored, tokens of the step) of every request."""
    r = np.random.RandomState(case["lens"])
    cached = r.randint(case["cached_lo"], case["cached_hi"] + 1, size=case["reqs"])
    new = r.randint(case["new_lo"], case["new_hi"] + 1, size=case["reqs"])
    if not new.sum():
        new[0] = 1
    return cached, new


def _firsts(case):
    """First visible position of every row: its document's first token; one row in fifty sees nothing."""
    cached, new = _lengths(case)
    r = np.random.RandomState(case["lens"] + 1)
    out = []
    for c, n in zip(cached, new):
        pos = c + np.arange(n)
        cuts = np.unique(np.concatenate([[0], r.randint(0, c + n, size=1 + (c + n) // 400)]))
        first = cuts[np.searchsorted(cuts, pos, side="right") - 1]
        out.append(np.where(r.random_sample(n) < 0.02, c + n, first))
    return np.concatenate(out)


def _starts(new):
    return np.concatenate([[0], np.cumsum(new)])


def _dev(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x)).to(device="cuda", dtype=dtype)


def _type(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    cached, new = _lengths(case)
    P, B = case["block"], case["reqs"]
    held, need = -(-cached // P), -(-(cached + new) // P)
    s = {"case": case, "reqs": B, "block": P, "rows": int(new.sum()), "max_new": int(new.max()), "max_blocks": int(max(need.max(), 1)),
         "cached": _dev(cached), "n_new": _dev(new), "err": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if case["op"] == "plan":
        blocks, taken = int(need.sum()) + 100, int((need - held).sum())
        ids = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
        s["blocks"] = blocks
        s["held"] = torch.full((B, s["max_blocks"] + 3), -1, dtype=torch.int32, device="cuda")
        _fill(s["held"], held, ids[: blocks - taken - 50])
        s["free"] = ids[blocks - taken - 50:].contiguous()
        s["table"] = s["held"].clone()
        s["capacity"] = -(-s["rows"] // 64) * 64  # a captured step has room for more rows than it uses
        s["row_start"] = torch.empty(B + 1, dtype=torch.int32, device="cuda")
        s["seq_id"] = torch.empty(s["capacity"], dtype=torch.int32, device="cuda")
        s["pos"] = torch.empty(s["capacity"], dtype=torch.int32, device="cuda")
        s["slot"] = torch.empty(s["capacity"], dtype=torch.int64, device="cuda")
        s["used"] = torch.empty(1, dtype=torch.int32, device="cuda")
        return s
    s["row_start"] = _dev(_starts(new))
    Hk, D, dt = case["kv_heads"], case["dim"], _type(case)
    if case["op"] == "store":  # the cache holds the blocks that the call touches, and some that it does not
        lo = cached // P
        blocks = int((need - lo).sum()) + 3
        table = np.full((B, s["max_blocks"]), -1, dtype=np.int32)
        ids = torch.randperm(blocks, generator=g, device="cuda").cpu().numpy()
        k = 0
        for b in range(B):
            table[b, lo[b]:need[b]] = ids[k:k + need[b] - lo[b]]
            k += need[b] - lo[b]
        s["table"] = _dev(table)
        # rows as a projection makes them: key and value side by side in one row, some tokens louder
        loud = 1.0 + 2.0 * (torch.rand(s["rows"], 1, 1, 1, generator=g, device="cuda") < 0.02)
        s["kv"] = (torch.randn(s["rows"], 2, Hk, D, generator=g, device="cuda") * loud).to(dt)
    else:
        blocks = int(need.sum()) + 3
        s["table"] = torch.full((B, s["max_blocks"]), -1, dtype=torch.int32, device="cuda")
        _fill(s["table"], need, torch.randperm(blocks, generator=g, device="cuda").to(torch.int32))
    for n in ("k", "v"):
        x = torch.empty(blocks, Hk, P, D, dtype=torch.uint8, device="cuda")
        for at in range(0, blocks, 4096):  # normal values, 4.48 standard deviations at the largest code
            part = torch.randn(x[at:at + 4096].shape, generator=g, device="cuda", dtype=torch.bfloat16)
            x[at:at + 4096] = (part * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s[n] = x
        s[n + "_scale"] = (0.7 + 0.6 * torch.rand(blocks, Hk, generator=g, device="cuda")) / 100
    if case["op"] == "attn":
        H, T = case["heads"], s["rows"]
        s["q"] = (1.5 * torch.randn(T, H, D, generator=g, device="cuda")).to(dt)
        s["out"] = torch.empty(T, H, D, dtype=dt, device="cuda")
        s["lse"] = torch.empty(T, H, dtype=torch.float32, device="cuda")
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, H + 1, device="cuda") / H) if case["bias"] else None
        s["first"] = _dev(_firsts(case)) if case["docs"] else None
        # at most the tokens that are stored after the step
        s["prefix"] = _dev(np.minimum(case["prefix"], cached + new)) if case["prefix"] else None
    return s


def _fill(table, counts, ids):
    """Row b of the table gets the next counts[b] of the ids."""
    n = torch.as_tensor(counts, device="cuda")
    at = torch.arange(table.shape[1], device="cuda")[None] < n[:, None]
    table[at] = ids[: int(n.sum())]


# ------------------------------------------------------------------ one pass


def run(s):
    op = s["case"]["op"]
    if own:
        return {"plan": _own_plan, "store": _own_store, "attn": _own_attn}[op](s)
    return {"plan": _plain_plan, "store": _plain_store, "attn": _plain_attn}[op](s)


def _own_cache(s):
    """The cache handle, which a program makes once, when it allocates the cache."""
    if "cache" not in s:
        import compressed_sparse_long_c128a_gb300 as csa

        s["csa"], s["cache"] = csa, csa.Kv8Cache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    return s["csa"], s["cache"]


def _own_plan(s):
    import compressed_sparse_long_c128a_gb300 as csa

    csa.step_plan(s["cached"], s["n_new"], s["free"], s["table"], s["block"], s["blocks"], s["row_start"], s["seq_id"], s["pos"],
                  s["slot"], s["used"], s["err"])
    return [s[k] for k in ("table", "row_start", "seq_id", "pos", "slot", "used")]


def _own_store(s):
    csa, cache = _own_cache(s)
    csa.kv8_store(s["kv"][:, 0], s["kv"][:, 1], s["row_start"], s["cached"], cache, s["table"], s["err"])
    return _stored(s)


def _own_attn(s):
    csa, cache = _own_cache(s)
    c = s["case"]
    if "ws" not in s:  # the workspace, allocated once like the caches
        n = csa.kv8_attn_workspace_size(s["rows"], s["reqs"], c["heads"], cache, s["max_new"])
        s["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    csa.kv8_attn(s["q"], s["row_start"], s["cached"], cache, s["table"], s["max_new"], s["out"], s["ws"], s["err"],
                 softcap=c["softcap"], window=c["window"], slopes=s["slopes"], first=s["first"], prefix=s["prefix"], lse=s["lse"])
    return [s["out"], s["lse"]]


def _stored(s):
    """The cache after an insert: codes as the values they stand for, and the scales."""
    f8 = torch.float8_e4m3fn
    return [s["k"].view(f8), s["v"].view(f8), s["k_scale"], s["v_scale"]]


def _plain_plan(s):
    P, T = s["block"], s["capacity"]
    cached, new = s["cached"].long(), s["n_new"].long()
    end = torch.cumsum(new, 0)
    start = end - new
    held, need = (cached + P - 1) // P, (cached + new + P - 1) // P
    took = torch.cumsum(need - held, 0)
    # blocks: those held stay, the new ones are the next free ids, the rest of the row is unmapped
    j = torch.arange(s["table"].shape[1], device="cuda")[None]
    at = (took - (need - held))[:, None] + j - held[:, None]
    fresh = s["free"][at.clamp(0, s["free"].numel() - 1)]
    table = torch.where(j < held[:, None], s["held"], torch.where(j < need[:, None], fresh, -1))
    # rows: request and position of each, and the slot its token has in the cache
    i = torch.arange(T, device="cuda")
    b = torch.searchsorted(end, i, right=True)
    real = i < end[-1]
    b = b.clamp(max=s["reqs"] - 1)
    pos = cached[b] + i - start[b]
    block = table[b, (pos // P).clamp(0, table.shape[1] - 1)].long()
    slot = torch.where(real, block * P + pos % P, -1)
    row_start = torch.cat([torch.zeros_like(end[:1]), end])
    return [table, row_start.int(), torch.where(real, b, -1).int(), torch.where(real, pos, -1).int(), slot, took[-1:].int()]


def _rows(s):
    """Request, position and place in the request of every row."""
    i = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(s["row_start"][1:].long(), i, right=True)
    off = i - s["row_start"][b]
    return b, s["cached"][b].long() + off, off


def _plain_store(s):
    P, B, f8 = s["block"], s["reqs"], torch.float8_e4m3fn
    b, pos, _ = _rows(s)
    block, row = s["table"][b, pos // P].long(), pos % P
    cached, new = s["cached"].long(), s["n_new"].long()
    # the block that a request was in the middle of: its first rows are older than the step
    old_block = s["table"].gather(1, (cached // P).clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0].long()
    partly = ((cached % P > 0) & (new > 0))[:, None]
    old_rows = (torch.arange(P, device="cuda")[None] < (cached % P)[:, None]) & partly  # [B, P]
    old_block = torch.where(partly[:, 0], old_block, 0)
    _insert(s, "k", s["kv"][:, 0], block, row, old_block, old_rows, f8)
    _insert(s, "v", s["kv"][:, 1], block, row, old_block, old_rows, f8)
    return _stored(s)


def _insert(s, name, x, block, row, old_block, old_rows, f8):
    x, codes, scale = x.float(), s[name], s[name + "_scale"]
    nb, Hk = scale.shape
    top = torch.zeros(nb, Hk, device="cuda").index_reduce_(0, block, x.abs().amax(-1), "amax")
    touched = torch.zeros(nb, 1, dtype=torch.bool, device="cuda").index_fill_(0, block, True)
    # a block whose first row is written starts anew, another one keeps its scale or raises it
    begun = torch.zeros(nb, 1, dtype=torch.int32, device="cuda").index_reduce_(0, block, (row == 0).int()[:, None], "amax") > 0
    before = torch.where(begun, 0.0, scale)
    after = torch.where(touched, torch.maximum(before, top * (1.0 / 448.0)).clamp(min=TINY), scale)
    inv = 1.0 / after
    # the older rows of a block whose scale rose are rounded again
    ratio = (before * inv)[old_block]  # [B, Hk]
    old = codes[old_block]  # [B, Hk, P, D]
    again = (old.view(f8).float() * ratio[:, :, None, None]).clamp(-448, 448).to(f8).view(torch.uint8)
    rose = (after > before)[old_block]
    at = old_rows[:, None, :] & rose[:, :, None]
    bi, hi, ri = at.nonzero(as_tuple=True)
    codes[old_block[bi], hi, ri] = again[bi, hi, ri]
    codes[block, :, row] = (x * inv[block][..., None]).clamp(-448, 448).to(f8).view(torch.uint8)
    scale.copy_(after)


def _plain_attn(s):
    c, P, f8 = s["case"], s["block"], torch.float8_e4m3fn
    B, N, H, Hk, D = s["reqs"], s["max_new"], c["heads"], c["kv_heads"], c["dim"]
    G, S = H // Hk, s["max_blocks"] * P
    table = s["table"].clamp(min=0).long()

    def gathered(n):  # [B, Hk, S, D]
        x = s[n][table].view(f8).float() * s[n + "_scale"][table][..., None, None]
        return x.transpose(1, 2).reshape(B, Hk, S, D)

    cached, new = s["cached"].long(), (s["row_start"][1:] - s["row_start"][:-1]).long()
    i = torch.arange(N, device="cuda")[None]
    row = (s["row_start"][:-1].long()[:, None] + i).clamp(max=s["rows"] - 1)  # [B, N]
    q = s["q"][row].float().view(B, N, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * N, D)
    x = torch.matmul(q, gathered("k").transpose(-1, -2)) * D ** -0.5  # [B, Hk, G * N, S]
    x = x.view(B, Hk, G, N, S)
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    p, t = (cached[:, None] + i)[:, :, None], torch.arange(S, device="cuda")[None, None]  # [B, N, 1], [1, 1, S]
    if s["slopes"] is not None:
        x = x - s["slopes"].view(1, Hk, G, 1, 1) * (p - t).abs()[:, None, None].float()
    see = t <= p
    if c["window"]:
        see = see & (p - t < c["window"])
    if s["prefix"] is not None:
        see = see | (t < s["prefix"].long()[:, None, None])
    if s["first"] is not None:
        see = see & (t >= s["first"].long()[row][:, :, None])
    see = see & (t < (cached + new)[:, None, None])
    x = torch.where(see[:, None, None], x, -torch.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -torch.inf, 0.0, m)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, Hk, G * N, S), gathered("v")).view(B, Hk, G, N, D) / torch.where(total > 0, total, 1.0)
    lse = (m + torch.log(total))[..., 0]  # -inf where a row sees nothing
    b, _, off = _rows(s)
    out = o.permute(0, 3, 1, 2, 4)[b, off].reshape(s["rows"], H, D)
    return [out.to(_type(c)), lse.permute(0, 3, 1, 2)[b, off].reshape(s["rows"], H)]


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    cached, new = _lengths(case)
    P, B, T = case["block"], case["reqs"], int(new.sum())
    held, need = -(-cached // P), -(-(cached + new) // P)
    if case["op"] == "plan":
        # lengths in, free ids in, tables written once, four values a row out
        width = int(max(need.max(), 1)) + 3
        return {"bytes": 8 * B + 4 * int((need - held).sum()) + 4 * B * width + 4 * (B + 1) + 16 * (-(-T // 64) * 64), "flops": 0}
    Hk, D = case["kv_heads"], case["dim"]
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "store":
        touched = int((need - cached // P)[new > 0].sum())
        return {"bytes": 2 * T * Hk * D * (size + 1) + 2 * 8 * touched * Hk, "flops": 0}
    # attention: pairs of a row and a key that it sees, and the keys that some row of the request sees
    H, pairs, keys = case["heads"], 0, 0
    first = _firsts(case) if case["docs"] else None
    at = _starts(new)
    for b in range(B):
        n = int(cached[b] + new[b])
        if not new[b]:
            continue
        pos = cached[b] + np.arange(new[b])
        f = np.zeros_like(pos) if first is None else first[at[b]:at[b + 1]]
        pre = min(case["prefix"], n)
        lo = np.maximum(f, pos - case["window"] + 1 if case["window"] else 0)
        near = np.maximum(pos + 1 - lo, 0)  # keys by causality and window
        far = np.maximum(pre - f, 0)  # keys of the prefix
        both = np.maximum(np.minimum(pre, pos + 1) - np.maximum(f, lo), 0)
        pairs += int((near + far - both).sum())
        edge = np.zeros(n + 1, dtype=np.int64)
        for a, e in ((lo, np.maximum(pos + 1, lo)), (f, np.maximum(pre, f))):
            np.add.at(edge, np.minimum(a, n), 1)
            np.add.at(edge, np.minimum(e, n), -1)
        keys += int((np.cumsum(edge)[:-1] > 0).sum())
    return {"bytes": keys * Hk * D * 2 + T * H * (2 * D * size + 4), "flops": 4 * pairs * H * D}


# ------------------------------------------------------------------ the definition, in 64 bits


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    cached, new = _lengths(case)
    return _exact_store(case, s, cached, new) if case["op"] == "store" else _exact_attn(case, s, cached, new)


def _e4m3(x):
    """x rounded to the nearest e4m3 value (ties to even), at most 448, in 64 bits."""
    mant, exp = torch.frexp(x)
    step = torch.exp2((exp.clamp(min=-5) - 4).double())  # 4 significant bits, 2^-9 at the smallest
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_store(case, s, cached, new):
    P, f8 = case["block"], torch.float8_e4m3fn
    table, at = s["table"].cpu().numpy(), _starts(new)
    got = []
    for which, n in enumerate(("k", "v")):
        val, scale = s[n].view(f8).double(), s[n + "_scale"].double()
        for b in range(case["reqs"]):
            lo, hi = int(cached[b]), int(cached[b] + new[b])
            for j in range(lo // P, -(-hi // P) if new[b] else 0):
                p0, p1 = max(lo, j * P), min(hi, (j + 1) * P)
                x = s["kv"][at[b] + p0 - lo:at[b] + p1 - lo, which].double().transpose(0, 1)  # [Hk, rows, D]
                blk, old = int(table[b, j]), p0 - j * P
                was = scale[blk] if old else torch.zeros_like(scale[blk])
                to = torch.maximum(was, x.abs().amax((1, 2)) / 448).clamp(min=TINY)
                if old:
                    val[blk, :, :old] = _e4m3(val[blk, :, :old] * (was / to)[:, None, None])
                val[blk, :, old:old + p1 - p0] = _e4m3(x / to[:, None, None])
                scale[blk] = to
        got.append((val, scale))
    return [got[0][0], got[1][0], got[0][1], got[1][1]]


def _exact_attn(case, s, cached, new):
    H, Hk, D, P, f8 = case["heads"], case["kv_heads"], case["dim"], case["block"], torch.float8_e4m3fn
    G, at, table = H // Hk, _starts(new), s["table"].cpu().numpy()
    out = torch.zeros(s["rows"], H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((s["rows"], H), -torch.inf, dtype=torch.float64, device="cuda")
    for b in range(case["reqs"]):
        n, r0, r1 = int(cached[b] + new[b]), int(at[b]), int(at[b + 1])
        if r0 == r1:
            continue
        ids = torch.as_tensor(table[b, : -(-n // P)].astype(np.int64), device="cuda")
        t = torch.arange(n, device="cuda")[None]
        p = int(cached[b]) + torch.arange(r1 - r0, device="cuda")[:, None]
        hidden = t > p
        if case["window"]:
            hidden |= t <= p - case["window"]
        if s["prefix"] is not None:
            hidden &= t >= int(s["prefix"][b])
        if s["first"] is not None:
            hidden |= t < s["first"][r0:r1, None]
        for h in range(Hk):
            k = (s["k"][ids, h].view(f8).double() * s["k_scale"][ids, h].double()[:, None, None]).reshape(-1, D)[:n]
            v = (s["v"][ids, h].view(f8).double() * s["v_scale"][ids, h].double()[:, None, None]).reshape(-1, D)[:n]
            for g in range(h * G, (h + 1) * G):
                a = s["q"][r0:r1, g].double() @ k.T / D ** 0.5
                if case["softcap"]:
                    a = torch.tanh(a / case["softcap"]) * case["softcap"]
                if s["slopes"] is not None:
                    a = a - float(s["slopes"][g]) * (t - p).abs()
                a = a.masked_fill(hidden, -torch.inf)
                z = torch.logsumexp(a, 1)
                w = torch.exp(a - torch.where(torch.isinf(z), 0.0, z)[:, None])
                out[r0:r1, g], lse[r0:r1, g] = w @ v, z
    return [out, lse]
