"""What the operators of a decoding step with drafted tokens are measured on.

Four operators that surround the quantized linear layers of a served model:

* ``gemv_w4``: products of a few activation rows with 4-bit group-scaled weights,
* ``block_tables``: the paged cache's block tables and slot maps from request lengths,
* ``kv_cache_write``: new keys and values into the paged cache,
* ``tree_attention``: attention of drafted tokens (or single tokens) over the cache.

``own`` false: plain torch in 32 bits.  ``own`` true: the calls a user makes.

Layouts (element [..] order, last one contiguous):

* 4-bit weights, int32[N * K / 8]: 16-row tiles, then 128-deep k-blocks; in a tile and
  k-block, lane l = 0 .. 63 holds four dwords, dword j the codes of row l % 16 at
  k = 32 j + 8 (l / 16) + 0 .. 7; code c of these eight sits at bits
  4 (c / 2) + 16 (c % 2), as q + 8 with q in [-8, 7].  Scales fp16[K / group][N].
* keys  [pages][kv heads][page / 16][D / 32][16 keys][32], values
  [pages][kv heads][page / 16][D][16 keys].
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
        # one token of a drafting model through a 4096-wide output projection: the
        # smallest weight, where the launch counts
        {"name": "gemv 1x4096x4096", "op": "gemv", "M": 1, "N": 4096, "K": 4096, "group": 128,
         "dtype": "fp16"},
        # thirteen drafted tokens through a down projection, finer groups, bfloat16
        {"name": "gemv 13x5120x13824 g64", "op": "gemv", "M": 13, "N": 5120, "K": 13824,
         "group": 64, "dtype": "bf16"},
        # one token through the widest layer (gate and up in one): all HBM
        {"name": "gemv 1x57344x8192", "op": "gemv", "M": 1, "N": 57344, "K": 8192, "group": 128,
         "dtype": "fp16"},
        # sixteen requests decoding a token each: the step's bookkeeping, latency only
        {"name": "tables 16 decode", "op": "tables", "B": 16, "ctx_lo": 1, "ctx_hi": 4096,
         "new_lo": 1, "new_hi": 1, "page": 16},
        # a queue of prompts admitted at once, odd lengths, whole tables built
        {"name": "tables 512 prompts", "op": "tables", "B": 512, "ctx_lo": 0, "ctx_hi": 0,
         "new_lo": 17, "new_hi": 8191, "page": 64},
        # keys and values of sixteen requests with a tree of five tokens each
        {"name": "kv write 80", "op": "write", "B": 16, "ctx_lo": 33, "ctx_hi": 4095,
         "new_lo": 5, "new_hi": 5, "Hkv": 8, "D": 128, "page": 16, "dtype": "fp16"},
        # a prefill's keys and values, ragged prompts that start inside a page
        {"name": "kv write prompts", "op": "write", "B": 24, "ctx_lo": 0, "ctx_hi": 100,
         "new_lo": 1, "new_hi": 2047, "Hkv": 8, "D": 128, "page": 32, "dtype": "bf16"},
        # one request, one token, a short context: the smallest call
        {"name": "attn 1x1 ctx 37", "op": "attn", "B": 1, "ctx_lo": 37, "ctx_hi": 37, "new_lo": 1,
         "new_hi": 1, "H": 32, "Hkv": 32, "D": 128, "page": 16, "tree": False, "dtype": "fp16"},
        # ordinary decoding, single tokens, grouped heads, ragged contexts
        {"name": "attn 32x1 ctx 4k", "op": "attn", "B": 32, "ctx_lo": 129, "ctx_hi": 4095,
         "new_lo": 1, "new_hi": 1, "H": 64, "Hkv": 8, "D": 128, "page": 16, "tree": False,
         "dtype": "fp16"},
        # checking trees of up to thirteen drafted tokens, bfloat16
        {"name": "attn 24x13 ctx 8k", "op": "attn", "B": 24, "ctx_lo": 1001, "ctx_hi": 8191,
         "new_lo": 3, "new_hi": 13, "H": 64, "Hkv": 8, "D": 128, "page": 32, "tree": True,
         "dtype": "bf16"},
        # one head per key head and a wide tree, narrower heads
        {"name": "attn 8x48 mha d64", "op": "attn", "B": 8, "ctx_lo": 5, "ctx_hi": 2050,
         "new_lo": 21, "new_hi": 48, "H": 40, "Hkv": 40, "D": 64, "page": 16, "tree": True,
         "dtype": "fp16"},
        # two very long contexts: the work has to be split along the cache
        {"name": "attn 2x9 ctx 128k", "op": "attn", "B": 2, "ctx_lo": 100003, "ctx_hi": 131063,
         "new_lo": 6, "new_hi": 9, "H": 64, "Hkv": 8, "D": 128, "page": 64, "tree": True,
         "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemv", "gemv", "tables", "write", "attn", "attn", "attn"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "gemv":
        # odd numbers of k-blocks and row tiles: the listed ones are even
        K = 128 * (_log(rng, 4, 222) | 1)
        N = 16 * (_log(rng, 16, min(3582, 57344 * 8192 // K // 16 - 1)) | 1)
        return {"op": op, "M": _log(rng, 1, 64), "N": N, "K": K, "group": rng.choice([32, 64, 128]),
                "dtype": dtype}
    page = rng.choice([16, 32, 64, 128])
    if op == "tables":
        B = _log(rng, 1, 512)
        hi = _log(rng, 1, 8191)
        ctx = _log(rng, 1, 8191) - 1
        return {"op": op, "B": B, "ctx_lo": rng.randint(0, ctx), "ctx_hi": ctx,
                "new_lo": rng.randint(0, hi), "new_hi": hi, "page": page}
    Hkv, group = rng.choice([(8, 8), (8, 4), (32, 1), (40, 1), (1, 16), (4, 7)])
    D = rng.choice([64, 96, 128, 128, 256])
    if op == "write":
        T = _log(rng, 8, 24 * 1024 * 8 * 128 // (Hkv * D))
        B = _log(rng, 1, min(T, 64))
        hi = max(1, T // B)
        return {"op": op, "B": B, "ctx_lo": 0, "ctx_hi": rng.randint(0, 300),
                "new_lo": rng.randint(1, hi), "new_hi": hi, "Hkv": Hkv, "D": D, "page": page,
                "dtype": dtype}
    new = _log(rng, 1, 64)
    # keys read, and scores of the plain form, at most those of the largest listed case
    most = min(230000 * 1024 // (Hkv * D), 131072 * 2 * 64 * 9 // (Hkv * group * new))
    keys = _log(rng, 16, max(17, most))
    B = _log(rng, 1, max(1, min(64, keys // 8)))
    hi = max(1, min(131000, keys // B))
    return {"op": op, "B": B, "ctx_lo": rng.randint(hi // 2, hi), "ctx_hi": hi,
            "new_lo": rng.randint(1, new), "new_hi": new, "H": Hkv * group, "Hkv": Hkv, "D": D,
            "page": page, "tree": rng.random() < 0.7, "dtype": dtype}


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


def _pages(n, page):
    return (n + page - 1) // page


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


# ---- inputs ------------------------------------------------------------------------


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) % (1 << 62))


def _normal(shape, g, dtype, by=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * by).to(dtype)


def _quantized(N, K, group, g):
    """4-bit codes of normal weights in the packed layout, and their scales."""
    packed = torch.empty(N // 16, K // 128, 64, 4, dtype=torch.int32, device=DEV)
    scales = torch.empty(K // group, N, dtype=torch.float16, device=DEV)
    step = max(16, min(N, (1 << 26) // K // 16 * 16))
    for n0 in range(0, N, step):
        n1 = min(N, n0 + step)
        w = torch.randn((n1 - n0, K // group, group), generator=g, device=DEV) * 0.02
        s = (w.abs().amax(2) / 7).to(torch.float16)
        q = torch.round(w / s.float()[..., None]).clamp_(-7, 7).to(torch.int32).view(n1 - n0, K)
        scales[:, n0:n1] = s.t()
        # [tile][row][k-block][j][lane / 16][pair][half] -> [tile][k-block][lane / 16][row][j]
        u = (q + 8).view(-1, 16, K // 128, 4, 4, 4, 2).permute(0, 2, 4, 1, 3, 5, 6)
        at = torch.arange(4, dtype=torch.int32, device=DEV)
        d = ((u[..., 0] | (u[..., 1] << 16)) << (4 * at)).sum(-1).to(torch.int32)
        packed[n0 // 16:n1 // 16] = d.reshape(-1, K // 128, 64, 4)
    return packed.view(-1), scales


def _tables(case, g, pool):
    """(block tables with the pages the requests hold, the pool's other pages in a
    random order)."""
    ctx, new = _lengths(case)
    page = case["page"]
    most = max(1, max(_pages(c + n, page) for c, n in zip(ctx, new)))
    order = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    held = torch.tensor([_pages(c, page) for c in ctx], device=DEV)
    first = held.cumsum(0) - held
    col = torch.arange(most, device=DEV)
    at = (first[:, None] + col).clamp(max=pool - 1)
    table = torch.where(col < held[:, None], order[at], -1).contiguous()
    return table, order[sum(_pages(c, page) for c in ctx):].contiguous()


def _pool(case):
    """Pages of the case's cache: what its requests need, and a sixteenth more."""
    ctx, new = _lengths(case)
    need = sum(_pages(c + n, case["page"]) for c, n in zip(ctx, new))
    return need + need // 16 + 1


def _full_tables(case, g):
    """Block tables with every page of the requests, the new tokens' included."""
    ctx, new = _lengths(case)
    full = dict(case, ctx_lo=0, ctx_hi=0)
    table = torch.full((case["B"], max(1, max(_pages(c + n, case["page"])
                                              for c, n in zip(ctx, new)))), -1,
                       dtype=torch.int32, device=DEV)
    need = torch.tensor([_pages(c + n, full["page"]) for c, n in zip(ctx, new)], device=DEV)
    order = torch.randperm(_pool(case), generator=g, device=DEV).to(torch.int32)
    col = torch.arange(table.shape[1], device=DEV)
    at = (need.cumsum(0) - need)[:, None] + col
    return torch.where(col < need[:, None], order[at.clamp(max=order.numel() - 1)], table)


def _slots(table, ctx, new, page):
    """The slot of every new token, request after request."""
    b = torch.repeat_interleave(torch.arange(len(new), device=DEV), torch.tensor(new, device=DEV))
    start = torch.tensor(np.cumsum([0] + new[:-1]), device=DEV)
    pos = torch.tensor(ctx, device=DEV)[b] + torch.arange(len(b), device=DEV) - start[b]
    return (table[b, pos // page].long() * page + pos % page).to(torch.int32)


def _cache(case, g):
    pages, D, page = _pool(case), case["D"], case["page"]
    dt = DTYPES[case["dtype"]]
    k = _normal((pages, case["Hkv"], page // 16, D // 32, 16, 32), g, dt)
    v = _normal((pages, case["Hkv"], page // 16, D, 16), g, dt)
    return k, v


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
    if case["op"] == "gemv":
        state["w"], state["s"] = _quantized(case["N"], case["K"], case["group"], g)
        state["x"] = _normal((case["M"], case["K"]), g, DTYPES[case["dtype"]])
        return state
    ctx, new = _lengths(case)
    state["ctx"], state["new"] = _i32(ctx), _i32(new)
    state["cu"] = _i32([0] + np.cumsum(new).tolist())
    if case["op"] == "tables":
        state["table"], state["free"] = _tables(case, g, _pool(case))
        state["head"] = _i32([0])
        # a program's slot map has room for its largest step
        state["most"] = max(256, (sum(new) + 255) // 256 * 256)
        return state
    state["table"] = _full_tables(case, g)
    state["kc"], state["vc"] = _cache(case, g)
    dt = DTYPES[case["dtype"]]
    if case["op"] == "write":
        # keys and values as a fused projection leaves them: [token][k heads, v heads]
        kv = _normal((sum(new), 2 * case["Hkv"], case["D"]), g, dt)
        state["k"], state["v"] = kv[:, :case["Hkv"]], kv[:, case["Hkv"]:]
        state["slots"] = _slots(state["table"], ctx, new, case["page"])
        return state
    state["q"] = _normal((sum(new), case["H"], case["D"]), g, dt, 1.5)
    words = (max(new) + 31) // 32
    state["mask"] = _trees(new, words, seed) if case["tree"] else None
    state["max_new"], state["max_len"] = max(new), max(c + n for c, n in zip(ctx, new))
    return state


# ---- the plain forms ---------------------------------------------------------------


def _plain_gemv(s):
    c = s["case"]
    N, K = c["N"], c["K"]
    d = s["w"].view(N // 16, K // 128, 4, 16, 4, 1)
    at = 4 * torch.arange(4, dtype=torch.int32, device=d.device)
    pair = (d >> at) & 0x000F000F                                  # [...][j][pair]
    u = torch.stack((pair & 15, pair >> 16), -1)                   # [...][j][pair][half]
    q = u.permute(0, 3, 1, 4, 2, 5, 6).reshape(N, K // c["group"], c["group"]).float() - 8
    w = q * s["s"].t().float()[..., None]
    return (s["x"].float() @ w.view(N, K).t()).to(s["x"].dtype)


def _plain_tables(s):
    page, most = s["case"]["page"], s["most"]
    ctx, new, table, free = s["ctx"], s["new"], s["table"], s["free"]
    B, cols = table.shape
    have = (ctx + page - 1) // page
    add = (ctx + new + page - 1) // page - have
    end = add.cumsum(0)
    col = torch.arange(cols, device=ctx.device)
    j = col - have[:, None]
    at = s["head"] + (end - add)[:, None] + j
    inside = (at >= 0) & (at < free.numel())
    fresh = torch.where(inside, free[at.clamp(0, max(0, free.numel() - 1))], -1)
    table = torch.where((j >= 0) & (j < add[:, None]), fresh, table)
    cu = torch.cat((new.new_zeros(1), new.cumsum(0).to(torch.int32)))
    t = torch.arange(most, device=ctx.device, dtype=torch.int32)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=B - 1)
    pos = ctx[b] + t - cu[b]
    at = pos // page
    got = table[b, at.clamp(0, cols - 1)]
    slot = torch.where((t < cu[-1]) & (at < cols) & (got >= 0), got * page + pos % page, -1)
    counts = torch.stack((cu[-1], end[-1], s["head"][0] + end[-1])).to(torch.int32)
    return table, slot.to(torch.int32), cu, counts


def _plain_write(s):
    c = s["case"]
    page, D = c["page"], c["D"]
    slots = s["slots"].long()
    at, block, row = slots // page, slots % page // 16, slots % 16
    T = slots.numel()
    s["kc"][at, :, block, :, row] = s["k"].reshape(T, c["Hkv"], D // 32, 32)
    s["vc"][at, :, block, :, row] = s["v"]
    return s["kc"], s["vc"]


def _plain_attention(s):
    c = s["case"]
    B, H, Hkv, D, page, T = c["B"], c["H"], c["Hkv"], c["D"], c["page"], s["max_new"]
    dev = s["q"].device
    nblk = _pages(s["max_len"], page)
    L = nblk * page
    at = s["table"][:, :nblk].clamp(min=0).long()
    k = s["kc"][at].permute(0, 2, 1, 3, 5, 4, 6).reshape(B, Hkv, L, D).float()
    v = s["vc"][at].permute(0, 2, 1, 3, 5, 4).reshape(B, Hkv, L, D).float()
    ctx, new, start = s["ctx"].long(), s["new"].long(), s["cu"][:-1].long()
    t = torch.arange(T, device=dev)
    row = (start[:, None] + t).clamp(max=s["q"].shape[0] - 1)      # [B][T]
    q = s["q"][row].float().view(B, T, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4)
    j = torch.arange(L, device=dev) - ctx[:, None]                 # [B][L]
    if s["mask"] is None:
        seen = j[:, None] <= t[:, None]                            # [B][T][L]
    else:
        words = s["mask"].shape[1]
        word = (j // 32).clamp(0, words - 1)[:, None].expand(B, T, L)
        bit = (s["mask"][row].gather(2, word) >> (j % 32).int()[:, None]) & 1
        seen = (j[:, None] < 0) | ((bit == 1) & (j[:, None] < new[:, None, None]))
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


def run(state):
    op, case = state["case"]["op"], state["case"]
    if not own:
        return {"gemv": _plain_gemv, "tables": _plain_tables, "write": _plain_write,
                "attn": _plain_attention}[op](state)
    import w6a6_w6a8_integer_amd as fq
    s = state
    if op == "gemv":
        return fq.gemv_w4(s["x"], s["w"], s["s"], case["N"])
    if op == "tables":
        slots, cu, counts = fq.block_tables(s["ctx"], s["new"], s["free"], s["table"],
                                            page_size=case["page"], max_tokens=s["most"],
                                            free_head=s["head"])
        return s["table"], slots, cu, counts
    if op == "write":
        fq.kv_cache_write(s["k"], s["v"], s["slots"], s["kc"], s["vc"])
        return s["kc"], s["vc"]
    return fq.tree_attention(s["q"], s["kc"], s["vc"], s["table"], s["ctx"], s["cu"],
                             tree_mask=s["mask"], max_new=s["max_new"], return_lse=True)


def work(case):
    if case["op"] == "gemv":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": N * K // 2 + 2 * N * K // case["group"] + 2 * M * (N + K),
                "flops": 2 * M * N * K}
    ctx, new = _lengths(case)
    page = case["page"]
    if case["op"] == "tables":
        added = sum(_pages(c + n, page) - _pages(c, page) for c, n in zip(ctx, new))
        return {"bytes": 12 * case["B"] + 8 * added + 4 * sum(new), "flops": 0}
    width = case["Hkv"] * case["D"]
    if case["op"] == "write":
        return {"bytes": 8 * sum(new) * width + 4 * sum(new), "flops": 0}
    keys = sum(c + n for c, n in zip(ctx, new))
    rows = sum(new) * case["H"]
    return {"bytes": 4 * keys * width + rows * (4 * case["D"] + 4),
            "flops": 4 * case["D"] * case["H"] * sum(n * (c + 1) for c, n in zip(ctx, new))}


# ---- the definitions in 64 bits ----------------------------------------------------


def _exact_gemv(s):
    c = s["case"]
    N, K, group = c["N"], c["K"], c["group"]
    d = s["w"].cpu().numpy().view(np.uint32).reshape(-1, K // 128, 64, 4)
    y = torch.empty((c["M"], N), dtype=torch.float64, device=DEV)
    x = s["x"].double()
    scale = s["s"].double().repeat_interleave(group, 0)            # [K][N]
    step = max(1, (1 << 26) // K // 16)
    for a in range(0, N // 16, step):
        part = torch.from_numpy(d[a:a + step].view(np.int32)).to(DEV)
        w = torch.empty((part.shape[0], 16, K), dtype=torch.float64, device=DEV)
        by_k = w.view(part.shape[0], 16, K // 128, 4, 4, 8)        # k = 128 kb + 32 j + 8 p + c
        lanes = part.view(part.shape[0], K // 128, 4, 16, 4)       # lane = 16 p + row
        for code in range(8):
            v = (lanes >> (4 * (code // 2) + 16 * (code % 2))) & 15
            by_k[..., code] = (v - 8).permute(0, 3, 1, 4, 2).double()
        n0 = 16 * a
        w = w.view(-1, K)
        y[:, n0:n0 + w.shape[0]] = x @ (w.t() * scale[:, n0:n0 + w.shape[0]])
    return y


def _exact_tables(s):
    page = s["case"]["page"]
    table = s["table"].cpu().numpy().copy()
    free = s["free"].cpu().numpy()
    head = taken = int(s["head"][0])
    slot = np.full(s["most"], -1, np.int32)
    cu = [0]
    for b, (c, n) in enumerate(zip(s["ctx"].tolist(), s["new"].tolist())):
        for i in range(-(-c // page), -(-(c + n) // page)):
            table[b, i] = free[taken]
            taken += 1
        pos = np.arange(c, c + n)
        slot[cu[-1]:cu[-1] + n] = table[b, pos // page] * page + pos % page
        cu.append(cu[-1] + n)
    return table, slot, np.array(cu, np.int32), np.array([cu[-1], taken - head, taken], np.int32)


def _exact_write(s):
    c = s["case"]
    Hkv, D, page = c["Hkv"], c["D"], c["page"]
    kc, vc = s["kc"].double().view(-1), s["vc"].double().view(-1)
    slot = s["slots"].long()[:, None, None]
    h = torch.arange(Hkv, device=DEV)[:, None]
    d = torch.arange(D, device=DEV)
    block = (slot // page * Hkv + h) * (page // 16) + slot % page // 16
    kc[block * 16 * D + d // 32 * 512 + slot % 16 * 32 + d % 32] = s["k"].double()
    vc[block * 16 * D + d * 16 + slot % 16] = s["v"].double()
    return kc.view_as(s["kc"]), vc.view_as(s["vc"])


def _exact_attention(s):
    c = s["case"]
    H, Hkv, D, page = c["H"], c["Hkv"], c["D"], c["page"]
    outs, lses = [], []
    at = 0
    for b, (ctx, n) in enumerate(zip(s["ctx"].tolist(), s["new"].tolist())):
        pos = torch.arange(ctx + n, device=DEV)
        p = s["table"][b].long()[pos // page]
        blk, r = pos % page // 16, pos % 16
        seen = torch.ones((n, ctx + n), dtype=torch.bool)
        for t in range(n):
            for j in range(n):
                seen[t, ctx + j] = (j <= t if s["mask"] is None
                                    else bool((int(s["mask"][at + t, j // 32]) >> (j % 32)) & 1))
        seen = seen.to(DEV)
        q = s["q"][at:at + n].double()
        out = torch.zeros((n, H, D), dtype=torch.float64, device=DEV)
        lse = torch.full((n, H), -math.inf, dtype=torch.float64, device=DEV)
        for hk in range(Hkv):
            k = s["kc"][p, hk, blk, :, r].reshape(-1, D).double()
            v = s["vc"][p, hk, blk, :, r].double()
            for h in range(hk * (H // Hkv), (hk + 1) * (H // Hkv)):
                x = (q[:, h] @ k.t()) * D ** -0.5
                x = torch.where(seen, x, -math.inf)
                lse[:, h] = torch.logsumexp(x, 1)
                out[:, h] = torch.softmax(x, 1) @ v
        outs.append(out)
        lses.append(lse)
        at += n
    return torch.cat(outs), torch.cat(lses)


def exact(case, seed):
    state = prepare(case, seed)
    return {"gemv": _exact_gemv, "tables": _exact_tables, "write": _exact_write,
            "attn": _exact_attention}[case["op"]](state)
