"""Decoding with drafted token trees on a small random model, one GPU.

The served model's layers are 6-bit (W6AxLinear), the drafting model's 4-bit copies of
them (W4Linear).  A step, for a batch of requests of different lengths:

1. the drafting model grows a tree of likely continuations of every request;
2. the served model takes all of the trees in one pass: block_tables gives their tokens
   slots, and in each layer kv_cache_write puts their keys and values there and
   tree_attention lets each token attend its request and its ancestors;
3. along each tree the tokens that the served model would itself have chosen are kept,
   their keys and values moved together behind the request's, and spare pages given back.

The tokens are those that decoding one by one gives (--check runs both).

    python examples/drafted_decoding.py [--tokens 24] [--check]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import w6a6_w6a8_integer_amd as fq  # noqa: E402

DEV = "cuda"
VOCAB, HIDDEN, HEADS, KV_HEADS, WIDTH, INNER, LAYERS = 512, 512, 8, 2, 64, 1024, 2
PAGE, PAGES, COLUMNS = 16, 256, 16


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-5)).half()


def rotate(x, pos):
    """Rotary positions on [tokens][heads][WIDTH]."""
    inv = 10000.0 ** (-torch.arange(0, WIDTH, 2, device=x.device) / WIDTH)
    angle = (pos[:, None].float() * inv)[:, None]
    a, b = x.float().chunk(2, -1)
    return torch.cat((a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()),
                     -1).half()


class Cache:
    """A model's paged keys and values, and the pages of its requests."""

    def __init__(self, requests):
        self.layers = [fq.kv_cache(PAGES, KV_HEADS, WIDTH, PAGE) for _ in range(LAYERS)]
        self.table = torch.full((requests, COLUMNS), -1, dtype=torch.int32, device=DEV)
        self.free = torch.arange(PAGES, dtype=torch.int32, device=DEV)
        self.ctx = [0] * requests       # tokens kept

    def open(self, new):
        """Slots for new[b] more tokens of every request."""
        self.new = new
        total = sum(new)
        self.ctx_d, new_d = i32(self.ctx), i32(new)
        self.slots, self.cu, self.counts = fq.block_tables(self.ctx_d, new_d, self.free,
                                                           self.table, PAGE, total)
        self.start = [sum(new[:b]) for b in range(len(new))]

    def keep(self, rows):
        """Keeps rows[b] (indexes of the step's tokens of request b, in order), moved
        together behind the request's others, and gives the other pages back."""
        at = torch.tensor([self.start[b] + r for b, rs in enumerate(rows) for r in rs],
                          device=DEV)
        to = torch.tensor([self.start[b] + i for b, rs in enumerate(rows)
                           for i in range(len(rs))], device=DEV)
        if at.numel():
            for (k, v), (kc, vc) in zip(self.kv, self.layers):
                fq.kv_cache_write(k[at], v[at], self.slots[to], kc, vc)
        spare = []
        for b, rs in enumerate(rows):
            need = -(-(self.ctx[b] + self.new[b]) // PAGE)
            self.ctx[b] += len(rs)
            spare.append(self.table[b, -(-self.ctx[b] // PAGE):need])
        taken = int(self.counts[1])
        assert taken <= self.free.numel(), "the cache is full"
        self.free = torch.cat((self.free[taken:], *spare))


class Model:
    def __init__(self, weights, linear):
        self.embed, self.head = weights["embed"], weights["head"].float()
        self.layers = [{k: linear(w) for k, w in layer.items()} for layer in weights["layers"]]

    def __call__(self, cache, tokens, new, depth, masks):
        """Logits of the step's tokens: tokens and depths (behind the kept ones) of all
        requests in turn, masks int32[tokens][words] of the drafted ancestors or None."""
        cache.open(new)
        ctx = torch.cat([torch.full((n,), c) for c, n in zip(cache.ctx, new)]).to(DEV)
        pos = ctx + torch.tensor(depth, device=DEV)
        x = self.embed[torch.tensor(tokens, device=DEV)]
        cache.kv = []
        for layer, (kc, vc) in zip(self.layers, cache.layers):
            qkv = layer["qkv"](norm(x)).view(len(tokens), HEADS + 2 * KV_HEADS, WIDTH)
            q = rotate(qkv[:, :HEADS], pos)
            k = rotate(qkv[:, HEADS:HEADS + KV_HEADS], pos)
            v = qkv[:, HEADS + KV_HEADS:]
            fq.kv_cache_write(k, v, cache.slots, kc, vc)
            cache.kv.append((k, v))
            y = fq.tree_attention(q, kc, vc, cache.table, cache.ctx_d, cache.cu, tree_mask=masks,
                                  max_new=max(new))
            x = x + layer["o"](y.view(len(tokens), HIDDEN))
            gate, up = layer["gate_up"](norm(x)).chunk(2, -1)
            x = x + layer["down"]((torch.nn.functional.silu(gate.float()) * up).half())
        return norm(x).float() @ self.head.t()


def random_weights(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def w(n, k):
        return (torch.randn(n, k, generator=g, device=DEV) * k ** -0.5).half()

    return {"embed": w(VOCAB, HIDDEN) * 8, "head": w(VOCAB, HIDDEN),
            "layers": [{"qkv": w((HEADS + 2 * KV_HEADS) * WIDTH, HIDDEN), "o": w(HIDDEN, HIDDEN),
                        "gate_up": w(2 * INNER, HIDDEN), "down": w(HIDDEN, INNER)}
                       for _ in range(LAYERS)]}


class Tree:
    """Drafted tokens of one request: node 0 is its last token, not yet in the cache."""

    def __init__(self, token):
        self.tokens, self.parents, self.depth = [token], [-1], [0]

    def add(self, parent, token):
        self.tokens.append(token)
        self.parents.append(parent)
        self.depth.append(self.depth[parent] + 1)

    def masks(self):
        bits = []
        for t, p in enumerate(self.parents):
            bits.append((bits[p] if p >= 0 else 0) | 1 << t)
        return [[b - (1 << 32) if b >= 1 << 31 else b] for b in bits]


def run_trees(model, cache, trees):
    new = [len(t.tokens) for t in trees]
    return model(cache, sum((t.tokens for t in trees), []), new,
                 sum((t.depth for t in trees), []), i32(sum((t.masks() for t in trees), [])))


def draft(model, cache, trees, levels=3, width=2):
    """Grows every tree by `levels` levels: the best `width` followers of the first node,
    then of the likeliest path."""
    tips = [0] * len(trees)
    for _ in range(levels):
        best = run_trees(model, cache, trees).topk(width).indices.tolist()
        start = cache.start
        cache.keep([[] for _ in trees])          # the tree is run again with its new leaves
        for b, t in enumerate(trees):
            first = len(t.tokens)
            for token in best[start[b] + tips[b]]:
                t.add(tips[b], token)
            tips[b] = first


def generate(served, prompts, tokens, drafter=None):
    """Greedy continuations of the prompts, and the steps of the served model they took."""
    cache = Cache(len(prompts))
    new = [len(p) for p in prompts]
    logits = served(cache, sum(prompts, []), new, [i for n in new for i in range(n)], None)
    cache.keep([list(range(n)) for n in new])
    out = [[int(logits[s + n - 1].argmax())] for s, n in zip(cache.start, new)]
    drafts = None
    if drafter:
        drafts = Cache(len(prompts))
        drafter(drafts, sum(prompts, []), new, [i for n in new for i in range(n)], None)
        drafts.keep([list(range(n)) for n in new])
    steps = 1
    while min(len(o) for o in out) < tokens:
        trees = [Tree(o[-1]) for o in out]
        if drafter:
            draft(drafter, drafts, trees)
            run_trees(drafter, drafts, trees)    # keys and values of the last level too
        choice = run_trees(served, cache, trees).argmax(-1).tolist()
        kept = []
        for b, t in enumerate(trees):
            path, node = [0], 0
            while True:
                token = choice[cache.start[b] + node]
                out[b].append(token)
                follow = [n for n, p in enumerate(t.parents) if p == node and t.tokens[n] == token]
                if not follow:
                    break
                node = follow[0]
                path.append(node)
            kept.append(path)
        cache.keep(kept)
        if drafter:
            drafts.keep(kept)
        steps += 1
    return [o[:tokens] for o in out], steps


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--tokens", type=int, default=24)
    p.add_argument("--check", action="store_true", help="also decode one by one and compare")
    a = p.parse_args()
    weights = random_weights(1)
    served = Model(weights, lambda w: fq.W6AxLinear(w, abits=8))
    drafter = Model(weights, lambda w: fq.W4Linear(w, group=64))
    g = torch.Generator().manual_seed(2)
    prompts = [torch.randint(VOCAB, (n,), generator=g).tolist() for n in (5, 37, 16, 1)]
    out, steps = generate(served, prompts, a.tokens, drafter)
    for o in out:
        print(*o)
    print(f"{a.tokens} tokens of {len(prompts)} requests in {steps} steps of the served model")
    if a.check:
        plain, plain_steps = generate(served, prompts, a.tokens)
        print(f"one by one: {plain_steps} steps, the tokens are "
              f"{'the same' if plain == out else 'DIFFERENT'}")
        return 0 if plain == out else 1
    return 0


if __name__ == "__main__":
    sys.exit(main())
