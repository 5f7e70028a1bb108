"""GPU parity of the low-rank adapters (flexq_lora_add) with their definition in 64 bits;
tolerances are derived in kv4_reference.py."""
import math

import numpy as np
import pytest

import kv4_reference as ref

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DEV = "cuda:0"
F16, BF16 = torch.float16, torch.bfloat16
NAN = float("nan")


@pytest.fixture(scope="module")
def fq():
    import w6a6_w6a8_integer_amd as fq
    fq.lib()
    return fq


def say(*a):
    print(*a, flush=True)


def rng(*key):
    return np.random.default_rng([int(k) for k in key])


def normal(r, shape, dtype, by=1.0):
    return torch.from_numpy((r.standard_normal(shape) * by).astype(np.float32)).to(dtype)


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def problem(r, T, N, K, R, L, dtype, ids=None, ranks=None):
    if ids is None:
        ids = r.integers(-1, L, T)
    if ranks is None:
        ranks = r.integers(0, R + 1, L)
        ranks[r.integers(L)] = R
    p = {"x": normal(r, (T, K), dtype), "y": normal(r, (T, N), dtype),
         "a": normal(r, (L, R, K), dtype, K ** -0.5), "b": normal(r, (L, N, R), dtype, 0.2),
         "ids": np.asarray(ids), "ranks": np.asarray(ranks),
         "scales": (r.random(L) * 2 - 0.5).astype(np.float32)}
    for i, n in enumerate(p["ranks"]):     # what lies past a rank does not matter
        n = min(max(int(n), 0), R)
        p["a"][i, n:] = NAN
        p["b"][i, :, n:] = NAN
    return p


def call(fq, p, **kw):
    args = dict(ranks=i32(p["ranks"]), scales=torch.from_numpy(p["scales"]).to(DEV))
    args.update(kw)
    return fq.lora_add(p["x"].to(DEV), p["y"].to(DEV), i32(p["ids"]), p["a"].to(DEV),
                       p["b"].to(DEV), **args)


def check(p, out, ranks=True, scales=True):
    a, b = (np.nan_to_num(p[n].double().numpy()) for n in "ab")
    want, tol = ref.lora(p["x"].double().numpy(), p["y"].double().numpy(), p["ids"], a, b,
                         p["ranks"] if ranks else None, p["scales"] if scales else None,
                         p["x"].dtype)
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= tol).all(), (float(np.nanmax(err / tol)), np.argwhere(~(err <= tol))[:4].tolist())
    # over many outputs: rounding's own root mean square, a step's 1 / sqrt(12), and 2 %
    if err.size >= 2048:
        eps = ref.OUT_EPS[p["x"].dtype]
        off = math.sqrt((err ** 2).sum() / (want ** 2).sum())
        assert off <= 2 * eps / math.sqrt(12) * 1.02, off


SHAPES = [(1, 16, 128, 8, 1), (1, 4096, 4096, 16, 4), (2, 48, 384, 8, 3), (7, 80, 256, 24, 5),
          (16, 1040, 1152, 16, 2), (17, 64, 640, 32, 1), (33, 272, 128, 64, 2), (64, 336, 1024, 128, 40),
          (64, 2064, 2176, 64, 64), (65, 96, 384, 40, 3), (128, 176, 256, 256, 4),
          (130, 528, 896, 200, 7), (300, 144, 1280, 16, 5), (1000, 64, 256, 8, 3),
          (4200, 32, 128, 16, 2)]


@pytest.mark.parametrize("T,N,K,R,L", SHAPES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_lora_add(fq, T, N, K, R, L, dtype):
    say("lora_add", T, N, K, R, L, dtype)
    p = problem(rng(41, T, N, K, R), T, N, K, R, L, dtype)
    y = p["y"].to(DEV)
    out = call(fq, p, out=torch.full_like(y, NAN))
    check(p, out)
    # in place: the same
    args = (p["x"].to(DEV), y, i32(p["ids"]), p["a"].to(DEV), p["b"].to(DEV), i32(p["ranks"]),
            torch.from_numpy(p["scales"]).to(DEV))
    again = fq.lora_add(*args)
    assert again is y or again.data_ptr() == y.data_ptr()
    assert torch.equal(out, y)


# several tiles of 64 tokens, whose rows come through LDS up to rank 64: blocks of 128 outputs that
# end inside one, slices of K summed by the second product and (from eight tiles on) before it
TILES = [(66, 128, 128, 8, 1), (100, 144, 384, 64, 3), (129, 272, 2176, 24, 6), (190, 1040, 512, 48, 2),
         (321, 400, 640, 40, 70), (513, 16, 1152, 64, 5), (700, 272, 384, 32, 9), (1025, 528, 256, 16, 2)]


# rows of up to 128 ranks come through LDS as well, longer ones straight from memory
WIDE = [(65, 16, 128, 72, 2), (150, 400, 640, 128, 3), (520, 272, 1280, 96, 12), (577, 144, 384, 104, 1),
        (140, 208, 384, 136, 2), (600, 80, 256, 256, 3)]


@pytest.mark.parametrize("T,N,K,R,L", TILES + WIDE)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_several_tiles(fq, T, N, K, R, L, dtype):
    """Adapters mixed in every tile, then in runs; out apart, and in place the same."""
    say("lora_add", T, N, K, R, L, dtype)
    r = rng(48, T, N, K, R)
    for ids in (r.integers(-1, L, T), np.sort(r.integers(-1, L, T))):
        p = problem(r, T, N, K, R, L, dtype, ids)
        y = p["y"].to(DEV)
        out = call(fq, p, out=torch.full_like(y, NAN))
        check(p, out)
        p2 = {**p, "y": y}
        assert call(fq, p2).data_ptr() == y.data_ptr() and torch.equal(out, y)


@pytest.mark.parametrize("T,N,R,L", [(64, 4112, 16, 40), (64, 592, 200, 1), (1, 8208, 8, 1), (130, 16, 8, 2),
                                     (4159, 6160, 8, 2)])
def test_tokens_without_an_adapter(fq, T, N, R, L):
    """Whole tiles of them and a few, over blocks of many columns: y bit for bit."""
    r = rng(50, T, N, R)
    for few in (False, True):
        ids = np.full(T, -1)
        if few:
            ids[r.permutation(T)[:max(1, T // 9)]] = r.integers(L)
        p = problem(r, T, N, 128, R, L, BF16, ids)
        y = p["y"].to(DEV)
        out = call(fq, p, out=torch.full_like(y, NAN))
        none = torch.from_numpy(ids < 0).to(DEV)
        assert torch.equal(out[none], y[none])
        if few:
            keep = np.nonzero(ids >= 0)[0][:40]
            check({**p, "x": p["x"][keep], "y": p["y"][keep], "ids": ids[keep]}, out[keep])


@pytest.mark.parametrize("n", [1, 16, 17, 31, 32, 33, 48, 49, 63, 64])
def test_tokens_of_one_adapter_in_several_tiles(fq, n):
    """Every number of tokens that an adapter can have in a tile, others around them."""
    r = rng(49, n)
    ids = r.integers(1, 6, 200)
    for t0 in (0, 64, 128):
        ids[t0 + r.permutation(64)[:n]] = 0
    p = problem(r, 200, 144, 512, 40, 6, BF16, ids)
    check(p, call(fq, p))


@pytest.mark.parametrize("n", [1, 15, 16, 17, 31, 32, 33, 48, 49, 64, 100])
def test_tokens_of_one_adapter(fq, n):
    """Every number of columns that a tile can have, others between them."""
    r = rng(42, n)
    T = n + 9
    ids = np.zeros(T, int)
    ids[r.permutation(T)[:9]] = [1, 2, -1, 1, 3, 2, -1, 5, 1]
    p = problem(r, T, 144, 512, 16, 6, F16, ids)
    check(p, call(fq, p))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_prompts_and_defaults(fq, dtype):
    """Runs of one adapter over many tiles; no ranks and no scales given."""
    r = rng(43)
    lens = [1, 200, 3, 64, 129, 300]
    ids = np.repeat([2, 0, -1, 3, 2, 1], lens)
    p = problem(r, len(ids), 208, 1152, 32, 4, dtype, ids, [32] * 4)
    check(p, call(fq, p, ranks=None, scales=None), ranks=False, scales=False)


def test_adapters_and_ranks_outside_their_ranges(fq):
    """Adapters outside [0, L) are none; ranks are cut to 0 .. R, and rank 0 adds nothing."""
    r = rng(44)
    ids = [0, 1, 2, 3, -1, -7, 4, 1 << 30, -1 << 31, 2, 2, 0]
    p = problem(r, len(ids), 64, 256, 16, 4, F16, ids, [99, 0, -3, 5])
    p["ranks"] = np.array([99, 0, -3, 5])
    out = call(fq, p)
    check(p, out)
    same = [i for i, a in enumerate(ids) if a not in (0, 3)]
    assert torch.equal(out.cpu()[same], p["y"][same])
    # no adapter at all, out apart and in place
    empty = torch.empty(0, 16, 256, dtype=F16, device=DEV), torch.empty(0, 64, 16, dtype=F16, device=DEV)
    y = p["y"].to(DEV)
    out = fq.lora_add(p["x"].to(DEV), y, i32(ids), *empty, out=torch.zeros_like(y))
    assert torch.equal(out, y)


def test_strided_rows_guards_and_stream(fq):
    r = rng(45)
    T, N, K = 70, 112, 384
    p = problem(r, T, N, K, 16, 3, BF16)
    x = torch.zeros(T, K + 64, dtype=BF16, device=DEV)
    x[:, 8:8 + K] = p["x"].to(DEV)
    wide = torch.full((T + 2, 3 * N), 3.0, dtype=BF16, device=DEV)
    wide[1:-1, N:2 * N] = p["y"].to(DEV)
    y = wide[1:-1, N:2 * N]
    args = (x[:, 8:8 + K], y, i32(p["ids"]), p["a"].to(DEV), p["b"].to(DEV), i32(p["ranks"]),
            torch.from_numpy(p["scales"]).to(DEV))
    out = torch.full((T, N + 8), 5.0, dtype=BF16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fq.lora_add(*args, out=out[:, :N])
        fq.lora_add(*args)
    torch.cuda.current_stream().wait_stream(side)
    check(p, out[:, :N])
    assert torch.equal(out[:, :N], y) and bool((out[:, N:] == 5).all())
    wide[1:-1, N:2 * N] = 3
    assert bool((wide == 3).all())
    with pytest.raises(fq.FlexqError):
        fq.lora_add(*args, out=wide[:-2, N:2 * N])


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_sizes_of_h_and_values_that_are_not_finite(fq, dtype):
    """h past fp16's range and far below it; an infinite activation reaches its token alone, a
    NaN weight the tokens of its adapter."""
    r = rng(46)
    for by in (2.0 ** 12, 2.0 ** -11) if dtype == F16 else (2.0 ** 60, 2.0 ** -70):
        p = problem(r, 9, 64, 512, 16, 2, dtype)
        p["x"] *= by
        p["a"] *= 8
        p["scales"] = (p["scales"] / by).astype(np.float32)
        check(p, call(fq, p))
    p = problem(r, 40, 64, 512, 16, 3, dtype, ranks=[16, 9, 4])
    clean = call(fq, p)
    i = int(np.nonzero(p["ids"] >= 0)[0][5])
    p["x"][i, 77] = math.inf
    p["a"][:, :, 77] = p["a"][:, :, 77].abs() + 0.5
    p2 = {**p, "x": p["x"].clone()}
    p2["x"][i, 77] = 0
    base, out = call(fq, p2), call(fq, p)
    rest = [t for t in range(40) if t != i]
    assert torch.equal(out[rest], base[rest]) and not bool(torch.isfinite(out[i]).any())
    assert clean.shape == out.shape
    p2["a"][0, 0, 3] = NAN
    out = call(fq, p2)
    mine = torch.from_numpy(p["ids"] == 0).to(DEV)
    assert bool(out[mine].isnan().all()) and torch.equal(out[~mine], base[~mine])


def test_in_a_graph_beside_a_layer(fq):
    """A 4-bit layer and its adapters captured and replayed, between eager work, with other
    activations and adapters."""
    r = rng(47)
    T, N, K, R, L = 20, 256, 512, 16, 4
    layer = fq.W4Linear(normal(r, (N, K), F16, K ** -0.5).to(DEV))
    p = problem(r, T, N, K, R, L, F16, ranks=[16, 3, 8, 16])
    a, b, ranks = p["a"].to(DEV), p["b"].to(DEV), i32(p["ranks"])
    by = torch.from_numpy(p["scales"]).to(DEV)
    x, ids = torch.zeros(T, K, dtype=F16, device=DEV), i32([0] * T)

    def step():
        return fq.lora_add(x, layer(x), ids, a, b, ranks, by)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(6):
        x.copy_(normal(r, (T, K), F16))
        ids.copy_(i32(r.integers(-1, L, T)))
        torch.cuda.synchronize()
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        assert torch.equal(got, want), i
        base = layer(x)
        p |= {"x": x.cpu(), "y": base.cpu(), "ids": ids.cpu().numpy()}
        check(p, got)
