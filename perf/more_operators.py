"""What the operators of a decoding step with a 4-bit cache and the requests' own adapters
are measured on.

Four operators beside the quantized linear layers of a served model:

* ``kv4_cache_write``: new keys and values into a paged cache of 4-bit codes,
* ``kv4_cache_read``: tokens of that cache as 16-bit rows,
* ``kv4_attention``: attention of drafted tokens (or single tokens) over that cache, with an
  optional sliding window whose first tokens stay visible,
* ``lora_add``: low-rank adapters of many requests at once, added to a shared projection.

``own`` false: plain torch in 32 bits.  ``own`` true: the calls a user makes.

The 4-bit cache.  A token's head row x[0 .. D) is held as b + s c: b = fp16(min x),
s = fp16((max x - min x) / 15) (binary32 before the last rounding),
c = clamp(rint((x - b) / s), 0, 15), and c = 0 where s = 0.  Layouts (last index contiguous), r = slot % 16:

* key codes    int32 [pages][kv heads][page / 16][16][D / 8]: dword (r, o) holds the codes of
  d = 8 o + c at bits 4 (c / 2) + 16 (c % 2)
* value codes  int32 [pages][kv heads][page / 16][2][D / 2][2]: dword (r / 8, p, r % 8 / 4) holds
  d = 2 p and 2 p + 1 of four tokens, token r % 4 in byte 0, 2, 1, 3 (even d low)
* scales       fp16 [pages][kv heads][page / 16][4][16]: s and b of the keys, of the values
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}

# The heads, hidden sizes and layers are those of the LLaMA-2 shapes the benchmark
# runs (7B: 32 / 32 heads, 13B: 40 / 40, 70B: 64 / 8, all 128 wide).


def listed():
    return [
        # a decoding step's new keys and values, one token a request: latency only
        {"name": "store 16 decode", "op": "store", "B": 16, "ctx_lo": 33, "ctx_hi": 4095,
         "new_lo": 1, "new_hi": 1, "Hkv": 8, "D": 128, "page": 16, "dtype": "fp16"},
        # prompts written, and taken back as the cache holds them, for the prompts' own
        # attention to see what later steps will see; ragged, some start inside a page
        {"name": "store prompts", "op": "store", "B": 24, "ctx_lo": 0, "ctx_hi": 100, "new_lo": 1,
         "new_hi": 2047, "Hkv": 8, "D": 128, "page": 32, "dtype": "bf16"},
        # a short shared prefix taken from the cache, every head with keys of its own
        {"name": "read 57", "op": "read", "B": 1, "ctx_lo": 0, "ctx_hi": 0, "new_lo": 57,
         "new_hi": 57, "Hkv": 32, "D": 128, "page": 16, "dtype": "fp16"},
        # the prefixes of twelve prompts
        {"name": "read prefixes", "op": "read", "B": 12, "ctx_lo": 0, "ctx_hi": 0, "new_lo": 129,
         "new_hi": 4095, "Hkv": 8, "D": 128, "page": 64, "dtype": "bf16"},
        # one request, one token, a short context: the smallest call
        {"name": "attn 1x1 ctx 37", "op": "attn", "B": 1, "ctx_lo": 37, "ctx_hi": 37, "new_lo": 1,
         "new_hi": 1, "H": 32, "Hkv": 32, "D": 128, "page": 16, "tree": False, "window": 0,
         "sinks": 0, "dtype": "fp16"},
        # ordinary decoding, single tokens, grouped heads, ragged contexts
        {"name": "attn 32x1 ctx 4k", "op": "attn", "B": 32, "ctx_lo": 129, "ctx_hi": 4095,
         "new_lo": 1, "new_hi": 1, "H": 64, "Hkv": 8, "D": 128, "page": 16, "tree": False,
         "window": 0, "sinks": 0, "dtype": "fp16"},
        # checking trees of up to seven drafted tokens, bfloat16
        {"name": "attn 24x7 ctx 8k", "op": "attn", "B": 24, "ctx_lo": 1001, "ctx_hi": 8191,
         "new_lo": 3, "new_hi": 7, "H": 64, "Hkv": 8, "D": 128, "page": 32, "tree": True,
         "window": 0, "sinks": 0, "dtype": "bf16"},
        # long conversations under a window of 4096 with four sinks, one head per key head
        {"name": "attn 8x1 window 4k", "op": "attn", "B": 8, "ctx_lo": 3001, "ctx_hi": 30011,
         "new_lo": 1, "new_hi": 1, "H": 40, "Hkv": 40, "D": 128, "page": 32, "tree": False,
         "window": 4096, "sinks": 4, "dtype": "bf16"},
        # two very long contexts: the work has to be split along the cache
        {"name": "attn 2x1 ctx 128k", "op": "attn", "B": 2, "ctx_lo": 100003, "ctx_hi": 131063,
         "new_lo": 1, "new_hi": 1, "H": 64, "Hkv": 8, "D": 128, "page": 64, "tree": False,
         "window": 0, "sinks": 0, "dtype": "fp16"},
        # one token with one small adapter on an output projection: the smallest call
        {"name": "lora 1x4096x4096 r16", "op": "lora", "B": 1, "len_lo": 1, "len_hi": 1, "L": 4,
         "R": 16, "N": 4096, "K": 4096, "dtype": "fp16"},
        # a decoding step of 64 requests with forty adapters loaded, ragged ranks
        {"name": "lora 64x10240x8192 r64", "op": "lora", "B": 64, "len_lo": 1, "len_hi": 1,
         "L": 40, "R": 64, "N": 10240, "K": 8192, "dtype": "bf16"},
        # prompts of a few adapters through the same projection
        {"name": "lora prompts", "op": "lora", "B": 9, "len_lo": 37, "len_hi": 797, "L": 6, "R": 64,
         "N": 10240, "K": 8192, "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "read", "attn", "attn", "attn", "lora", "lora"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "lora":
        # odd numbers of k-blocks and row tiles: the listed ones are even
        R = rng.choice([8, 16, 32, 64, 128])
        K = 128 * (_log(rng, 4, 90) | 1)
        N = 16 * (_log(rng, 16, 640) | 1)
        most = 4096 * 6 * 64 * 18432 // (R * (K + N))     # tokens times adapters
        L = _log(rng, 1, 64)
        T = _log(rng, 1, max(1, min(3600, most // L)))
        B = _log(rng, 1, min(T, 64))
        hi = max(1, T // B)
        return {"op": op, "B": B, "len_lo": rng.randint(1, hi), "len_hi": hi, "L": L, "R": R,
                "N": N, "K": K, "dtype": dtype}
    page = rng.choice([16, 32, 64, 128])
    Hkv, group = rng.choice([(8, 8), (8, 4), (32, 1), (40, 1), (1, 16), (4, 7)])
    D = rng.choice([64, 96, 128, 128, 256])
    if op in ("store", "read"):
        T = _log(rng, 8, 24 * 1024 * 8 * 128 // (Hkv * D))
        B = _log(rng, 1, min(T, 64))
        hi = max(1, T // B)
        return {"op": op, "B": B, "ctx_lo": 0, "ctx_hi": rng.randint(0, 300),
                "new_lo": rng.randint(1, hi), "new_hi": hi, "Hkv": Hkv, "D": D, "page": page,
                "dtype": dtype}
    new = _log(rng, 1, 24)
    # keys read, and scores of the plain form, at most those of the largest listed cases
    most = min(230000 * 1024 // (Hkv * D), 4600 * 24 * 64 * 7 * 128 // (Hkv * group * new * D))
    keys = _log(rng, 16, max(17, most))
    B = _log(rng, 1, max(1, min(64, keys // 8)))
    hi = max(1, min(131000, keys // B))
    window = rng.random() < 0.4
    return {"op": op, "B": B, "ctx_lo": rng.randint(hi // 2, hi), "ctx_hi": hi,
            "new_lo": rng.randint(1, new), "new_hi": new, "H": Hkv * group, "Hkv": Hkv, "D": D,
            "page": page, "tree": rng.random() < 0.6,
            "window": _log(rng, 8, max(9, hi)) if window else 0,
            "sinks": rng.randint(0, 40) if window else 0, "dtype": dtype}


# ---- the requests of a case --------------------------------------------------------


def _spread(lo, hi, n, step):
    """n whole numbers in lo .. hi, spread evenly but not in order."""
    return [lo + int((hi - lo + 1) * (((i + 1) * step) % 1.0)) for i in range(n)]


def _lengths(case):
    """(context lengths, new lengths) of the case's requests."""
    ctx = _spread(case["ctx_lo"], case["ctx_hi"], case["B"], 0.6180339887498949)
    new = _spread(case["new_lo"], case["new_hi"], case["B"], 0.7548776662466927)
    new[0] = case["new_hi"]
    return ctx, new


def _adapters(case):
    """(lengths of the requests, their adapters, the adapters' ranks): some adapters are
    asked for often, some never, and one request in eight has none (-1)."""
    B, L = case["B"], case["L"]
    lens = _spread(case["len_lo"], case["len_hi"], B, 0.7548776662466927)
    lens[0] = case["len_hi"]
    ids = [-1 if i % 8 == 5 else int(L * (((i + 1) * 0.6180339887498949) % 1.0) ** 1.5)
           for i in range(B)]
    ranks = [r // 4 * 4 if r > 4 else r
             for r in _spread(max(1, case["R"] // 4), case["R"], L, 0.5698402909980532)]
    ranks[ids[0]] = case["R"]
    return lens, ids, ranks


def _pages(n, page):
    return (n + page - 1) // page


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


# ---- inputs ------------------------------------------------------------------------


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) % (1 << 62))


def _normal(shape, g, dtype, by=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * by).to(dtype)


def _pool(case):
    """Pages of the case's cache: what its requests need, and a sixteenth more."""
    ctx, new = _lengths(case)
    need = sum(_pages(c + n, case["page"]) for c, n in zip(ctx, new))
    return need + need // 16 + 1


def _full_tables(case, g):
    """Block tables with every page of the requests, the new tokens' included."""
    ctx, new = _lengths(case)
    need = torch.tensor([_pages(c + n, case["page"]) for c, n in zip(ctx, new)], device=DEV)
    order = torch.randperm(_pool(case), generator=g, device=DEV).to(torch.int32)
    col = torch.arange(max(1, int(need.max())), device=DEV)
    at = (need.cumsum(0) - need)[:, None] + col
    return torch.where(col < need[:, None], order[at.clamp(max=order.numel() - 1)],
                       -1).contiguous()


def _slots(table, ctx, new, page):
    """The slot of every new token, request after request."""
    b = torch.repeat_interleave(torch.arange(len(new), device=DEV), torch.tensor(new, device=DEV))
    start = torch.tensor(np.cumsum([0] + new[:-1]), device=DEV)
    pos = torch.tensor(ctx, device=DEV)[b] + torch.arange(len(b), device=DEV) - start[b]
    return (table[b, pos // page].long() * page + pos % page).to(torch.int32)


def _cache(case, g):
    """A cache of codes spread as those of normal rows are, with such rows' scales."""
    lead = (_pool(case), case["Hkv"], case["page"] // 16)
    D = case["D"]

    def codes(shape):
        words = torch.zeros(shape, dtype=torch.int32, device=DEV)
        for c in range(8):
            u = torch.randn(shape, generator=g, device=DEV).mul_(2.9).add_(7.5).round_()
            words |= u.clamp_(0, 15).to(torch.int32) << (4 * c)
        return words

    s = torch.rand(lead + (2, 1, 16), generator=g, device=DEV) * 0.15 + 0.27
    b = s * (torch.randn(lead + (2, 1, 16), generator=g, device=DEV) * 0.7 - 7.5)
    scales = torch.cat((s, b), -2).reshape(lead + (4, 16)).to(torch.float16)
    return codes(lead + (16, D // 8)), codes(lead + (2, D // 2, 2)), scales


def _trees(new, words, seed):
    """Ancestor bits of random trees: token t's parent is an earlier token of its
    request or the context's end; a token attends itself and its ancestors."""
    rng = np.random.RandomState(seed % (1 << 31))
    mask = np.zeros((sum(new), words), np.uint32)
    at = 0
    for n in new:
        for t in range(n):
            parent = rng.randint(-1, t)
            if parent >= 0:
                mask[at + t] = mask[at + parent]
            mask[at + t, t // 32] |= np.uint32(1 << (t % 32))
        at += n
    return torch.from_numpy(mask.view(np.int32)).to(DEV)


def prepare(case, seed):
    g = _generator(seed)
    state = {"case": case}
    dt = DTYPES[case["dtype"]]
    if case["op"] == "lora":
        L, R, N, K = case["L"], case["R"], case["N"], case["K"]
        lens, ids, ranks = _adapters(case)
        state["ids"] = _i32([i for i, n in zip(ids, lens) for _ in range(n)])
        state["x"] = _normal((sum(lens), K), g, dt)
        state["y"] = _normal((sum(lens), N), g, dt)
        state["a"] = _normal((L, R, K), g, dt, K ** -0.5)
        state["b"] = _normal((L, N, R), g, dt, 0.1)
        state["ranks"] = _i32(ranks)
        state["by"] = torch.rand(L, generator=g, device=DEV) + 0.5
        return state
    ctx, new = _lengths(case)
    state["ctx"], state["new"] = _i32(ctx), _i32(new)
    state["cu"] = _i32([0] + np.cumsum(new).tolist())
    state["table"] = _full_tables(case, g)
    state["kc"], state["vc"], state["sc"] = _cache(case, g)
    if case["op"] != "attn":
        state["slots"] = _slots(state["table"], ctx, new, case["page"])
        if case["op"] == "store":
            # keys and values as a fused projection leaves them: [token][k heads, v heads];
            # some key channels are larger than the others
            kv = torch.randn((sum(new), 2 * case["Hkv"], case["D"]), generator=g, device=DEV)
            kv[:, :case["Hkv"], 5::48] *= 3
            kv = kv.to(dt)
            state["k"], state["v"] = kv[:, :case["Hkv"]], kv[:, case["Hkv"]:]
        return state
    state["q"] = _normal((sum(new), case["H"], case["D"]), g, dt, 1.5)
    words = (max(new) + 31) // 32
    state["mask"] = _trees(new, words, seed) if case["tree"] else None
    state["max_new"], state["max_len"] = max(new), max(c + n for c, n in zip(ctx, new))
    return state


# ---- the plain forms ---------------------------------------------------------------


def _plain_values(s, page, row):
    """Keys and values [..][kv heads][D] in 32 bits of the tokens at `row` of the pages."""
    block, r = row // 16, row % 16
    at = torch.arange(8, device=row.device)
    words = s["kc"][page, :, block, r]                             # [..][kv heads][D / 8]
    k = (words[..., None] >> (4 * (at // 2) + 16 * (at % 2)).int()) & 15
    words = s["vc"][page, :, block, r // 8, :, r % 8 // 4]         # [..][kv heads][D / 2]
    byte = r % 4 // 2 + r % 2 * 2
    words = words >> (8 * byte).int()[..., None, None]
    v = torch.stack((words & 15, (words >> 4) & 15), -1)
    by = s["sc"][page, :, block, :, r].float()[..., None]          # [..][kv heads][4][1]
    return (k.flatten(-2).float() * by[..., 0, :] + by[..., 1, :],
            v.flatten(-2).float() * by[..., 2, :] + by[..., 3, :])


def _plain_read(s):
    slots, page = s["slots"].long(), s["case"]["page"]
    k, v = _plain_values(s, slots // page, slots % page)
    dt = DTYPES[s["case"]["dtype"]]
    return k.to(dt), v.to(dt)


def _plain_quantize(x):
    """(codes int32 [T][kv heads][D], scales, offsets fp16) of rows."""
    x = x.float()
    low = x.amin(-1, keepdim=True)
    b = low.half()
    step = ((x.amax(-1, keepdim=True) - low) / 15).half()
    c = torch.where(step > 0, ((x - b.float()) / step.float()).round().clamp(0, 15), 0.0)
    return c.to(torch.int32), step[..., 0], b[..., 0]


def _plain_store(s):
    c = s["case"]
    page, D, Hkv = c["page"], c["D"], c["Hkv"]
    slots = s["slots"].long()
    at, block, r = slots // page, slots % page // 16, slots % 16
    codes, s["sc"][at, :, block, 0, r], s["sc"][at, :, block, 1, r] = _plain_quantize(s["k"])
    bit = torch.arange(8, dtype=torch.int32, device=r.device)
    words = codes.view(-1, Hkv, D // 8, 8) << (4 * (bit // 2) + 16 * (bit % 2))
    s["kc"][at, :, block, r] = words.sum(-1).to(torch.int32)
    codes, s["sc"][at, :, block, 2, r], s["sc"][at, :, block, 3, r] = _plain_quantize(s["v"])
    as_bytes = s["vc"].view(torch.uint8).view(*s["vc"].shape, 4)
    pair = codes[..., ::2] | codes[..., 1::2] << 4
    as_bytes[at, :, block, r // 8, :, r % 8 // 4, r % 4 // 2 + r % 2 * 2] = pair.to(torch.uint8)
    return _plain_read(s)


def _plain_attention(s):
    c = s["case"]
    B, H, Hkv, D, page, T = c["B"], c["H"], c["Hkv"], c["D"], c["page"], s["max_new"]
    dev = s["q"].device
    ctx, new, start = s["ctx"].long(), s["new"].long(), s["cu"][:-1].long()
    # the positions that some token may attend: the sinks, then the window's
    window = c["window"] or 1 << 30
    sinks = c["sinks"] if c["window"] else 0
    first = (ctx + 1 - window).clamp(min=sinks)                     # [B]
    col = torch.arange(sinks + min(s["max_len"], c["window"] + T if c["window"] else 1 << 30),
                       device=dev)
    pos = torch.where(col < sinks, col, first[:, None] + col - sinks)   # [B][L]
    L = pos.shape[1]
    end = (ctx + new)[:, None]
    at = pos.clamp(max=page * s["table"].shape[1] - 1)
    k, v = _plain_values(s, s["table"].long().gather(1, at // page).clamp(min=0), at % page)
    k, v = k.transpose(1, 2), v.transpose(1, 2).contiguous()        # [B][kv heads][L][D]
    t = torch.arange(T, device=dev)
    row = (start[:, None] + t).clamp(max=s["q"].shape[0] - 1)       # [B][T]
    q = s["q"][row].float().view(B, T, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4)
    j = pos - ctx[:, None]                                          # [B][L]
    inside = (pos[:, None] > (ctx[:, None] + t - window)[..., None]) | (pos < sinks)[:, None]
    if s["mask"] is None:
        seen = (j[:, None] <= t[:, None]) & inside                  # [B][T][L]
    else:
        words = s["mask"].shape[1]
        word = (j // 32).clamp(0, words - 1)[:, None].expand(B, T, L)
        bit = (s["mask"][row].gather(2, word) >> (j % 32).int()[:, None]) & 1
        drafted = (j[:, None] >= 0) & (bit == 1) & (j[:, None] < new[:, None, None])
        # the attended drafted tokens are the last positions of a token's window
        bits = (s["mask"][row][..., None] >> torch.arange(32, device=dev).int()) & 1
        count = bits.sum((-2, -1))                                  # [B][T]
        inside = pos[:, None] >= (ctx[:, None] + count - window)[..., None]
        seen = drafted | ((j[:, None] < 0) & (inside | (pos < sinks)[:, None]))
    seen &= (pos < end)[:, None]
    score = (q.reshape(B, Hkv, -1, D) @ k.transpose(2, 3)).view(B, Hkv, H // Hkv, T, L)
    score = (score / math.sqrt(D)).masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(B, Hkv, -1, L) @ v).view(B, Hkv, H // Hkv, T, D)
    out = torch.where(total > 0, out / total, 0.0)
    lse = (top + total.log())[..., 0]
    tok = torch.arange(s["q"].shape[0], device=dev)
    b = torch.searchsorted(s["cu"][1:].long(), tok, right=True)
    i = tok - start[b]
    out = out[b, :, :, i].reshape(-1, H, D)
    return out.to(s["q"].dtype), lse[b, :, :, i].reshape(-1, H)


def _plain_lora(s):
    c = s["case"]
    L, R, N, K, T = c["L"], c["R"], c["N"], c["K"], s["x"].shape[0]
    h = (s["x"].float() @ s["a"].float().view(L * R, K).t()).view(T, L, R)
    # everything but a token's own adapter, and what is past that one's rank, is out
    mine = s["ids"][:, None] == torch.arange(L, device=DEV)         # [T][L]
    rank = torch.arange(R, device=DEV) < s["ranks"][:, None]        # [L][R]
    h = torch.where(mine[..., None] & rank, h * s["by"][:, None], 0.0)
    b = s["b"].float().transpose(1, 2).reshape(L * R, N)
    return (s["y"].float() + h.view(T, L * R) @ b).to(s["y"].dtype)


def run(state):
    op, case = state["case"]["op"], state["case"]
    if not own:
        return {"store": _plain_store, "read": _plain_read, "attn": _plain_attention,
                "lora": _plain_lora}[op](state)
    import w6a6_w6a8_integer_amd as fq
    s = state
    if op == "lora":
        return fq.lora_add(s["x"], s["y"], s["ids"], s["a"], s["b"], ranks=s["ranks"],
                           scales=s["by"], out=torch.empty_like(s["y"]))
    if op == "attn":
        return fq.kv4_attention(s["q"], s["kc"], s["vc"], s["sc"], s["table"], s["ctx"], s["cu"],
                                tree_mask=s["mask"], max_new=s["max_new"],
                                window=case["window"] or None, sinks=case["sinks"],
                                return_lse=True)
    if op == "store":
        fq.kv4_cache_write(s["k"], s["v"], s["slots"], s["kc"], s["vc"], s["sc"])
    return fq.kv4_cache_read(s["slots"], s["kc"], s["vc"], s["sc"], dtype=DTYPES[case["dtype"]])


def work(case):
    if case["op"] == "lora":
        lens, ids, ranks = _adapters(case)
        size = case["K"] + case["N"]
        used = sum(ranks[i] for i in set(ids) if i >= 0)
        tokens = sum(n for n, i in zip(lens, ids) if i >= 0)
        return {"bytes": 2 * used * size + 2 * tokens * case["K"] + 4 * sum(lens) * case["N"]
                + 4 * sum(lens) + 8 * case["L"],
                "flops": 2 * size * sum(n * ranks[i] for n, i in zip(lens, ids) if i >= 0)}
    ctx, new = _lengths(case)
    held = case["Hkv"] * (case["D"] + 8)            # bytes of a token in the cache
    rows = 4 * case["Hkv"] * case["D"]              # and as 16-bit keys and values
    if case["op"] == "read":
        return {"bytes": sum(new) * (held + rows + 4), "flops": 0}
    if case["op"] == "store":
        return {"bytes": sum(new) * 2 * (held + rows + 4), "flops": 0}
    # context keys that the first token attends, in a window the last ones and the sinks
    seen = [min(c, case["window"] - 1 + case["sinks"]) if case["window"] else c for c in ctx]
    tokens = sum(new) * case["H"]
    return {"bytes": held * sum(c + n for c, n in zip(seen, new))
            + tokens * (4 * case["D"] + 4),
            "flops": 4 * case["D"] * case["H"] * sum(n * (c + 1) for c, n in zip(seen, new))}


# ---- the definitions in 64 bits ----------------------------------------------------


def _exact_token(s, slot):
    """Keys and values [n][kv heads][D] of the tokens at `slot`, by flat element indexes."""
    c = s["case"]
    Hkv, D, page = c["Hkv"], c["D"], c["page"]
    h = torch.arange(Hkv, device=DEV)[:, None]
    d = torch.arange(D, device=DEV)
    slot = slot.long()[:, None, None]
    block = (slot // page * Hkv + h) * (page // 16) + slot % page // 16    # [n][kv heads][1]
    r = slot % 16
    word = s["kc"].view(-1)[block * (2 * D) + r * (D // 8) + d // 8].long()
    k = (word >> (d % 8 // 2 * 4 + d % 2 * 16)) & 15
    word = s["vc"].view(-1)[block * (2 * D) + r // 8 * D + d // 2 * 2 + r % 8 // 4].long()
    byte = torch.tensor([0, 2, 1, 3], device=DEV)[r % 4]
    v = (word >> (8 * byte + d % 2 * 4)) & 15
    sc = s["sc"].view(-1).double()
    at = block * 64 + r
    return k * sc[at] + sc[at + 16], v * sc[at + 32] + sc[at + 48]


def _exact_read(s):
    parts = [_exact_token(s, p) for p in s["slots"].split(2048)]
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])


def _exact_store(s):
    out = []
    for x in (s["k"].double(), s["v"].double()):
        low = x.min(-1, keepdim=True).values
        step = ((x.max(-1, keepdim=True).values - low) / 15).half().double()
        low = low.half().double()
        code = torch.where(step == 0, 0.0, torch.clamp(torch.round((x - low) / step), 0, 15))
        out.append(low + code * step)
    return out


def _exact_attention(s):
    c = s["case"]
    H, Hkv, D, page = c["H"], c["Hkv"], c["D"], c["page"]
    window, sinks = c["window"], c["sinks"]
    outs, lses = [], []
    at = 0
    for b, (ctx, n) in enumerate(zip(s["ctx"].tolist(), s["new"].tolist())):
        low = max(0, ctx + 1 - window) if window else 0
        pos = torch.cat((torch.arange(min(sinks, low)), torch.arange(low, ctx + n)))
        seen = torch.zeros((n, pos.numel()), dtype=torch.bool)
        for t in range(n):
            mine = list(range(t + 1)) if s["mask"] is None else [
                j for j in range(n) if (int(s["mask"][at + t, j // 32]) >> (j % 32)) & 1]
            since = ctx + len(mine) - window if window else 0
            seen[t] = (pos < ctx) & ((pos >= since) | (pos < sinks))
            for j in mine:
                if s["mask"] is not None or ctx + j >= since or ctx + j < sinks:
                    seen[t] |= pos == ctx + j
        seen, pos = seen.to(DEV), pos.to(DEV)
        slot = s["table"][b].long()[pos // page] * page + pos % page
        q = s["q"][at:at + n].double()
        out = torch.zeros((n, H, D), dtype=torch.float64, device=DEV)
        x = torch.empty((n, H, pos.numel()), dtype=torch.float64, device=DEV)
        group = H // Hkv
        step = max(1, (1 << 25) // (Hkv * D))
        for i in range(0, pos.numel(), step):
            k = _exact_token(s, slot[i:i + step])[0].permute(1, 2, 0).contiguous()
            y = q.view(n, Hkv, group, D).transpose(0, 1).reshape(Hkv, n * group, D) @ k
            x[:, :, i:i + step] = y.view(Hkv, n, group, -1).transpose(0, 1).flatten(1, 2) * D ** -.5
        x = torch.where(seen[:, None], x, -math.inf)
        lses.append(torch.logsumexp(x, 2))
        x = torch.softmax(x, 2)
        for i in range(0, pos.numel(), step):
            v = _exact_token(s, slot[i:i + step])[1].transpose(0, 1).contiguous()
            w = x[:, :, i:i + step].reshape(n, Hkv, group, -1).transpose(0, 1).flatten(1, 2)
            out += (w @ v).view(Hkv, n, group, D).transpose(0, 1).reshape(n, H, D)
        outs.append(out)
        at += n
    return torch.cat(outs), torch.cat(lses)


def _exact_lora(s):
    out = s["y"].double()
    for i in range(s["case"]["L"]):
        rows = torch.nonzero(s["ids"] == i)[:, 0]
        r = int(s["ranks"][i])
        h = s["x"][rows].double() @ s["a"][i, :r].double().t()
        out[rows] += float(s["by"][i]) * (h @ s["b"][i, :, :r].double().t())
    return out


def exact(case, seed):
    state = prepare(case, seed)
    return {"store": _exact_store, "read": _exact_read, "attn": _exact_attention,
            "lora": _exact_lora}[case["op"]](state)
