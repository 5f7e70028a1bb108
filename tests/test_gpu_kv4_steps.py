"""A model's serving steps over the 4-bit cache on the GPU, as they are used: 6-bit layers with the
requests' own adapters, slots from the block tables, keys and values into the cache, attention
with a window; prompts first, then single tokens, the same steps eager and as a captured graph.
Each operator's results are held to its definition in 64 bits on what it was given."""
import math

import numpy as np
import pytest

import kv4_reference as ref

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DEV = "cuda:0"
F16 = torch.float16
HIDDEN, H, HKV, D, PAGE, PAGES, R, L = 512, 8, 2, 64, 16, 64, 16, 3
WINDOW, SINKS = 40, 4
PROMPTS, IDS, STEPS = [70, 5, 33, 130], [1, -1, 0, 2], 20


@pytest.fixture(scope="module")
def fq():
    import w6a6_w6a8_integer_amd as fq
    fq.lib()
    return fq


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


class Model:
    """One attention layer: a fused projection with adapters, the cache, an output projection."""

    def __init__(self, fq, r):
        self.fq = fq

        def normal(*shape):
            return torch.from_numpy((r.standard_normal(shape) * shape[-1] ** -0.5).astype(np.float32)).half().to(DEV)

        wide = (H + 2 * HKV) * D
        self.qkv, self.o = fq.W6AxLinear(normal(wide, HIDDEN), 8), fq.W6AxLinear(normal(HIDDEN, H * D), 8)
        self.ranks, self.by = i32([R, 5, 11]), torch.tensor([1.0, -0.5, 2.0], device=DEV)
        self.a1, self.b1 = normal(L, R, HIDDEN), normal(L, wide, R)
        self.a2, self.b2 = normal(L, R, H * D), normal(L, HIDDEN, R)
        self.cache = fq.kv4_cache(PAGES, HKV, D, PAGE, device=DEV)
        for t in self.cache:
            t.zero_()
        self.table = torch.full((len(IDS), 12), -1, dtype=torch.int32, device=DEV)
        self.free = torch.randperm(PAGES, generator=torch.Generator().manual_seed(7)).int().to(DEV)
        self.head, self.ctx = i32([0]), i32([0] * len(IDS))

    def step(self, x, new, ids, max_new, seen=None):
        """Everything from the hidden states x [T][HIDDEN] to the layer's output; `seen` gets the
        operators' arguments and results."""
        fq, T = self.fq, x.shape[0]
        slots, cu, counts = fq.block_tables(self.ctx, new, self.free, self.table, PAGE, T,
                                            free_head=self.head)
        base = self.qkv(x)
        qkv = fq.lora_add(x, base, ids, self.a1, self.b1, self.ranks, self.by,
                          out=torch.empty_like(base))
        heads = qkv.view(T, H + 2 * HKV, D)
        q, k, v = heads.split([H, HKV, HKV], 1)
        fq.kv4_cache_write(k, v, slots, *self.cache)
        out, lse = fq.kv4_attention(q, *self.cache, self.table, self.ctx, cu, max_new=max_new,
                                    window=WINDOW, sinks=SINKS, return_lse=True)
        flat = out.view(T, H * D)
        base2 = self.o(flat)
        y = fq.lora_add(flat, base2, ids, self.a2, self.b2, self.ranks, self.by,
                        out=torch.empty_like(base2))
        if seen is not None:
            seen.update(x=x, base=base, qkv=qkv, q=q, k=k, v=v, slots=slots, out=out, lse=lse,
                        flat=flat, base2=base2, y=y, ids=ids, ctx=self.ctx.clone())
        self.head.copy_(counts[2:])
        self.ctx.add_(new)
        return y


def check_adapters(x, y, out, ids, a, b, m):
    x, y, out, a, b = (t.double().cpu().numpy() for t in (x, y, out, a, b))
    want, tol = ref.lora(x, y, ids.cpu().numpy(), a, b, m.ranks.cpu().numpy(), m.by.cpu().numpy(), F16)
    assert (np.abs(out - want) <= tol).all()


def check_step(m, s, new):
    check_adapters(s["x"], s["base"], s["qkv"], s["ids"], m.a1, m.b1, m)
    check_adapters(s["flat"], s["base2"], s["y"], s["ids"], m.a2, m.b2, m)
    kc, vc, sc = (t.cpu().numpy().ravel() for t in m.cache)
    arrays = kc.view(np.uint32), vc.view(np.uint32), sc
    slots = s["slots"].cpu().numpy()
    # the new tokens' codes, scales and offsets
    for x, (c, by, b) in zip((s["k"], s["v"]), ref.read(*arrays, slots, HKV, D, PAGE)):
        want = ref.quantize(x.float().cpu().numpy())
        assert np.array_equal(c, want[0])
        assert np.array_equal(by, want[1].astype(float)) and np.array_equal(b, want[2].astype(float))
    table, ctx = m.table.cpu().numpy(), s["ctx"].cpu().numpy()
    q, out, lse = (s[n].double().cpu().numpy() for n in ("q", "out", "lse"))
    at = 0
    for i, n in enumerate(new):
        rows = slice(at, at + n)
        at += n
        pos = np.arange(ctx[i] + n)
        every = table[i][pos // PAGE] * PAGE + pos % PAGE
        assert np.array_equal(every[ctx[i]:], slots[rows])
        key, value = ref.read(*arrays, every, HKV, D, PAGE)
        want, want_lse, tol, tol_lse = ref.attention(
            q[rows], key, value, ref.attended(ctx[i], n, None, WINDOW, SINKS), D ** -0.5)
        tol = tol + ref.OUT_EPS[F16] * np.abs(want) * (1 + 2.0 ** -7) + ref.OUT_ABS[F16]
        assert (np.abs(out[rows] - want) <= tol).all(), i
        assert (np.abs(lse[rows] - want_lse) <= tol_lse).all(), i


def test_prompts_and_steps(fq):
    r = np.random.default_rng(51)
    m, twin = Model(fq, np.random.default_rng(50)), Model(fq, np.random.default_rng(50))

    def hidden(T):
        return torch.from_numpy(r.standard_normal((T, HIDDEN)).astype(np.float32)).half().to(DEV)

    # the prompts, whole, then 20 single tokens each
    T, B = sum(PROMPTS), len(IDS)
    x, seen = hidden(T), {}
    ids = i32(np.repeat(IDS, PROMPTS))
    y = m.step(x, i32(PROMPTS), ids, max(PROMPTS), seen)
    check_step(m, seen, PROMPTS)
    assert torch.equal(y, twin.step(x, i32(PROMPTS), ids, max(PROMPTS)))

    x, new, ids = torch.zeros(B, HIDDEN, dtype=F16, device=DEV), i32([1] * B), i32(IDS)
    spare = Model(fq, np.random.default_rng(50))
    spare.step(x, new, ids, 1)                       # loads the kernels
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = twin.step(x, new, ids, 1)
    for i in range(STEPS):
        x.copy_(hidden(B))
        if i == 9:                                   # another request takes a place's adapter
            ids.copy_(i32([0, 2, -1, 1]))
        torch.cuda.synchronize()
        graph.replay()
        seen = {}
        want = m.step(x, new, ids, 1, seen)
        torch.cuda.synchronize()
        check_step(m, seen, [1] * B)
        assert torch.equal(got, want), i
        for a, b in zip(m.cache, twin.cache):
            assert torch.equal(a, b), i
    assert int(m.ctx.sum()) == sum(PROMPTS) + STEPS * B and int(twin.ctx.sum()) == int(m.ctx.sum())
    assert not bool(y.isnan().any()) and math.isfinite(float(got.float().abs().max()))


def test_two_models_at_once(fq):
    """Two streams with a model each, their steps interleaved and never waited for: what each
    gives alone."""
    r = np.random.default_rng(52)
    x = [torch.from_numpy(r.standard_normal((sum(PROMPTS), HIDDEN)).astype(np.float32)).half().to(DEV)
         for _ in range(2)]
    rows, new, one = i32(np.repeat(IDS, PROMPTS)), i32(PROMPTS), i32([1] * len(IDS))
    ids = [i32(IDS), i32([2, 2, -1, 0])]

    def run(m, i, outs):
        outs.append(m.step(x[i], new, rows, max(PROMPTS)))
        for k in range(6):
            outs.append(m.step(x[i][k:k + len(IDS)], one, ids[i], 1))

    want = [[], []]
    for i in range(2):
        run(Model(fq, np.random.default_rng(60 + i)), i, want[i])
    models = [Model(fq, np.random.default_rng(60 + i)) for i in range(2)]
    torch.cuda.synchronize()
    got, streams = [[], []], [torch.cuda.Stream() for _ in range(2)]
    for k in range(7):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                m = models[i]
                got[i].append(m.step(x[i], new, rows, max(PROMPTS)) if k == 0 else
                              m.step(x[i][k - 1:k - 1 + len(IDS)], one, ids[i], 1))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i])), i
        assert len(got[i]) == len(want[i]) == 7
