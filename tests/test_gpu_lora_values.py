"""flexq_lora_add where a step has no adapter loaded, and where weights or sums are infinite or large."""
import pytest

import test_gpu_lora as base

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DEV = "cuda:0"
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def fq():
    import w6a6_w6a8_integer_amd as fq
    fq.lib()
    return fq


@pytest.mark.parametrize("R", [16, 256])
@pytest.mark.parametrize("T", [1, 65, 600, 5000])
def test_no_adapter_is_loaded(fq, T, R):
    """A pool without adapters, over one tile of tokens and many: out is y, apart and in place."""
    base.say("no adapters", T, R)
    r = base.rng(62, T, R)
    N, K = 272, 512
    x, y = base.normal(r, (T, K), F16).to(DEV), base.normal(r, (T, N), F16).to(DEV)
    a, b = torch.empty(0, R, K, dtype=F16, device=DEV), torch.empty(0, N, R, dtype=F16, device=DEV)
    ids = base.i32(r.integers(-1, 4, T))
    assert fq.lora_add_workspace_bytes(T, N, K, R, 0) == 0
    kept = y.clone()
    assert torch.equal(fq.lora_add(x, y, ids, a, b, out=torch.zeros_like(y)), kept)
    fq.lora_add(x, y, ids, a, b)
    torch.cuda.synchronize()
    assert torch.equal(y, kept)


# one tile straight from memory, several through LDS, more than 128 ranks straight from memory
LAYOUTS = [(1, 16), (20, 16), (33, 64), (64, 200), (130, 16), (200, 128), (600, 40), (140, 256)]


def apart(fq, p):
    return base.call(fq, p, out=torch.full_like(p["y"], float("nan")).to(DEV)).cpu()


@pytest.mark.parametrize("T,R", LAYOUTS)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_infinite_weights_of_the_second_product(fq, T, R, dtype):
    """An infinite weight of B gives its column an infinity of h's sign, two of them one or, of
    opposite signs, NaN; a token with h = 0 there has NaN.  Every other output is as it was."""
    base.say("infinite B", T, R, dtype)
    r = base.rng(66, T, R)
    N, K, inf = 144, 256, float("inf")
    ids = r.integers(0, 2, T)
    p = base.problem(r, T, N, K, R, 3, dtype, ids, [R, R - 3, 1])
    p["scales"] = [1.5, -0.5, 1.0]
    p["scales"] = torch.tensor(p["scales"]).numpy()
    if T > 1:
        p["x"][T // 2] = 0
    clean = apart(fq, p)
    spots = {(0, 5, 2): inf, (0, 6, R - 1): -inf, (0, 143, 0): inf, (0, 143, 7): -inf, (1, 5, 3): -inf,
             (1, 77, R - 4): inf}
    for (i, n, k), w in spots.items():
        p["b"][i, n, k] = w
    out = apart(fq, p)
    h = torch.einsum("trk,tk->tr", p["a"].nan_to_num().double()[ids], p["x"].double())
    by = torch.from_numpy(p["scales"]).double()[ids]
    want = torch.zeros(T, N, dtype=torch.float64)
    for (i, n, k), w in spots.items():
        mine = torch.from_numpy(ids == i)
        want[mine, n] += (h[:, k] * by)[mine] * w
    changed = want != 0                                     # (NaN among them)
    assert torch.equal(out[~changed], clean[~changed]) and int(changed.sum()) >= min(T, 3)
    assert torch.equal(out[changed].double().nan_to_num(7.0), want[changed].nan_to_num(7.0))


@pytest.mark.parametrize("T", [3, 140])
def test_infinite_weights_meet_the_least_sums(fq, T):
    """fp16 rows whose h spans more than 40 powers of 2: the least of it is not 0 where B is infinite."""
    N, K, R = 64, 128, 16
    r = base.rng(67, T)
    p = base.problem(r, T, N, K, R, 1, F16, [0] * T, [R])
    p["x"].zero_()
    p["x"][:, 3] = 1.0
    p["a"].zero_()
    p["a"][0, 0, 3], p["a"][0, 1, 3], p["a"][0, 2, 3] = 65504.0, 2.0 ** -24, -(2.0 ** -24)
    p["scales"][:] = 2.0 ** -10
    p["b"].fill_(0.25)
    clean = apart(fq, p)
    base.check(p, clean)
    p["b"][0, 7, 1], p["b"][0, 9, 2] = float("inf"), float("inf")
    out = apart(fq, p)
    assert bool((out[:, 7] == float("inf")).all()) and bool((out[:, 9] == -float("inf")).all())
    rest = [n for n in range(N) if n not in (7, 9)]
    assert torch.equal(out[:, rest], clean[:, rest])


@pytest.mark.parametrize("T,R", LAYOUTS)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_an_infinite_sum_beside_ordinary_ones(fq, T, R, dtype):
    """A token whose h has an infinity among numbers of tens: its outputs are infinities of the sign that
    the infinite one gives, whatever the others'."""
    base.say("infinite h", T, R, dtype)
    r = base.rng(68, T, R)
    N, K = 144, 256
    p = base.problem(r, T, N, K, R, 2, dtype, [1] * T, [R, R])
    p["a"] *= 30
    p["a"][1, 4, 9] = float("inf")
    p["x"][:, 9] = 0
    hit = torch.arange(T) % 3 == 0
    p["x"][hit, 9] = 1.0
    p["a"][1, 4, 10], p["x"][:, 10] = 1.0, 1.0
    rest = {**p, "a": p["a"].clone()}
    rest["a"][1, 4, 9] = 0
    out, base_out = apart(fq, p), apart(fq, rest)
    sign = torch.sign(p["b"][1, :, 4].double()) * float(p["scales"][1])
    want = torch.where(sign == 0, float("nan"), sign * float("inf"))
    got = out[hit].double()
    assert torch.equal(got.nan_to_num(7.0), want.expand_as(got).nan_to_num(7.0))
    assert bool(out[~hit].isnan().all())                   # (0 times infinity)
    assert bool(base_out.isfinite().all())


@pytest.mark.parametrize("T,R", LAYOUTS)
def test_large_bfloat16_weights_and_small_sums(fq, T, R):
    """Weights of B near bfloat16's largest and far below 1 whose products with h are ordinary numbers."""
    base.say("large B", T, R)
    r = base.rng(69, T, R)
    for by in (2.0 ** 118, 2.0 ** -90):
        p = base.problem(r, T, 144, 256, R, 3, BF16)
        p["b"] *= by
        p["a"] /= by
        base.check(p, base.call(fq, p))
