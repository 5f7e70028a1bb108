"""GPU numerics of tree_attention where one fp32 pass can lose them: the two 16-bit parts of
a probability, small probabilities behind a large one, and infinite values of attended
keys.  Bounds come from the definition (softmax in 64 bits) and from what the header says of
the probabilities, not from how the kernel forms them.
"""
import numpy as np
import pytest

import serve_reference as ref

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DEV = "cuda:0"
F16, BF16 = torch.float16, torch.bfloat16
U = 2.0 ** -23
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def fq():
    import w6a6_w6a8_integer_amd as fq
    fq.lib()
    return fq


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def cache_of(fq, keys, values, page):
    """The paged cache of requests' keys and values [len][Hkv][D] (in page order), and its
    block table."""
    Hkv, D = keys[0].shape[1:]
    need = [-(-k.shape[0] // page) for k in keys]
    kc, vc = fq.kv_cache(sum(need), Hkv, D, page, keys[0].dtype, "cpu")
    table = np.full((len(keys), max(need)), -1, np.int32)
    h, d = np.arange(Hkv)[:, None], np.arange(D)
    at = 0
    for b, (k, v) in enumerate(zip(keys, values)):
        table[b, :need[b]] = np.arange(at, at + need[b])
        slot = at * page + np.arange(k.shape[0])[:, None, None]
        ik, iv = ref.cache_index(slot, h, d, Hkv, D, page)
        kc.view(-1)[torch.from_numpy(ik)] = k
        vc.view(-1)[torch.from_numpy(iv)] = v
        at += need[b]
    return kc.to(DEV), vc.to(DEV), i32(table)


def attend(fq, q, keys, values, new, page=16, scale=1.0, mask=None):
    """(out, lse) of requests with new[b] drafted tokens each, in float64 on the CPU."""
    kc, vc, table = cache_of(fq, keys, values, page)
    ctx = [k.shape[0] - n for k, n in zip(keys, new)]
    out, lse = fq.tree_attention(q.to(DEV), kc, vc, table, i32(ctx),
                                 i32(np.concatenate(([0], np.cumsum(new)))), tree_mask=mask,
                                 max_new=max(new), scale=scale, return_lse=True)
    return out.double().cpu(), lse.double().cpu()


@pytest.mark.parametrize("rows", [1, 5])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_parts_of_a_probability(fq, dtype, rows):
    """Each probability as two 16-bit parts is within 2^-17 of itself.  One key of probability
    p and value 1, a few of probability 1 whose values add up to p's first sixteen bits: what
    is left of p has to be right to 2^-17 p (and the fp32 score, exponential and the three
    sums of a handful of terms to 16 u).  The p are those whose bits from the seventeenth on
    are nearly all ones.  With 16 rows a wave and, from 65 rows on, 32."""
    a = torch.arange(1, 2816).to(torch.float64) / 512
    a = a[a == a.to(dtype).double()]
    p = torch.exp(-a)
    unit = 2.0 ** (torch.floor(torch.log2(p)) - 15)
    worst = torch.argsort(p / unit - torch.floor(p / unit), descending=True)[:24]
    a, p, unit = a[worst], p[worst], unit[worst]
    B, L, D, H = len(a), 32, 64, 16
    keys, values = [], []
    for i in range(B):
        k, v = torch.zeros(L, 1, D, dtype=dtype), torch.zeros(L, 1, D, dtype=dtype)
        k[3, 0, 0], v[3] = -a[i], 256
        left = float(torch.floor(p[i] / unit[i]) * unit[i])
        for j in (7, 8, 20):                  # to at most eight bits each, exact in both types
            part = float(torch.tensor(left, dtype=torch.float64).to(BF16))
            v[j], left = -256 * part, left - part
        assert left == 0
        keys.append(k), values.append(v)
    # the last tokens are the drafted ones; their keys are zero, so a chain changes l only
    q = torch.zeros(B * rows, H, D, dtype=dtype)
    q[:, :, 0] = 1
    out, _ = attend(fq, q, keys, values, [rows] * B)
    for b in range(B):
        for t in range(rows):
            total = L - rows + t + float(p[b])
            want = 256 * float(p[b] - torch.floor(p[b] / unit[b]) * unit[b]) / total
            tol = (2.0 ** -17 + 16 * U) * 256 * float(p[b]) / total + ref.OUT_EPS[dtype] * want \
                + ref.OUT_ABS[dtype]
            err = (out[b * rows + t] - want).abs().max()
            assert float(err) <= tol, (b, t, float(err) / tol)


@pytest.mark.parametrize("nats", [6, 10, 12, 14, 17, 20])
@pytest.mark.parametrize("L,new,H", [(256, 1, 4), (255, 9, 16), (4096, 2, 4)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_small_probabilities_behind_a_large_one(fq, dtype, L, new, H, nats):
    """An early key far above all others, of value zero: the output is the others' alone.  The
    header's bound holds for each probability: 2^-17 of itself, in fp16 or 2^-34 of the row's
    largest, whichever is more.  All the other scores are alike (the errors of their
    probabilities all have one sign), and spread over a nat."""
    D = 64
    for spread in (0.0, 1.0):
        r = np.random.default_rng([L, new, nats, int(spread)])
        k = torch.zeros(L, 1, D, dtype=dtype)
        k[:, 0, 0] = torch.from_numpy(-nats - spread * r.random(L)).to(dtype)
        k[2, 0, 0] = 0
        v = torch.from_numpy(64 * r.random((L, 1, D)) + 32).to(dtype)
        v[2] = 0
        q = torch.zeros(new, H, D, dtype=dtype)
        q[:, :, 0] = 1
        out, lse = attend(fq, q, [k], [v], [new])
        for t in range(new):
            n = L - new + t + 1
            s = k[:n, 0, 0].double()
            p = torch.exp(s - s.max())
            want = (p @ v[:n, 0].double()) / p.sum()
            each = torch.maximum(2.0 ** -17 * p, torch.full_like(p, 2.0 ** -34)) \
                if dtype is F16 else 2.0 ** -17 * p
            tol = (each + (n / 32 + 96) * U * p) @ v[:n, 0].double() / p.sum()
            tol = tol + ref.OUT_EPS[dtype] * want * (1 + 2.0 ** -7) + ref.OUT_ABS[dtype]
            err = (out[t] - want).abs()
            assert bool((err <= tol).all()), (spread, t, float((err / tol).max()))
            assert float((lse[t] - p.sum().log() - s.max()).abs().max()) <= (n / 32 + 96) * U


@pytest.mark.parametrize("new,H,Hkv,D", [(1, 4, 2, 64), (3, 16, 1, 128), (9, 16, 1, 128),
                                         (30, 4, 2, 96), (5, 8, 1, 256)])
@pytest.mark.parametrize("ctx", [100, 1500])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_infinite_values_of_attended_keys(fq, dtype, ctx, new, H, Hkv, D):
    """An infinite value of an attended key gives an infinity of its sign, wherever the key
    lies and whatever its (positive) probability is; two of opposite signs, or a NaN, give
    NaN; the other columns keep their results.  With a mask, a drafted key's value reaches
    only the rows that attend it."""
    r = np.random.default_rng([ctx, new, H, D])
    L = ctx + new
    k = torch.from_numpy(r.standard_normal((L, Hkv, D)).astype(np.float32)).to(dtype)
    v = torch.from_numpy(r.standard_normal((L, Hkv, D)).astype(np.float32)).to(dtype)
    q = torch.from_numpy(r.standard_normal((new, H, D)).astype(np.float32)).to(dtype)
    k[5] = 4 * q[0, 0]                          # probabilities of all sizes
    seen = np.tril(np.ones((new, new), bool))
    for t in range(new):
        seen[t, :t] &= r.random(t) < 0.5
    words = torch.zeros(new, 1, dtype=torch.int64)
    for t, j in zip(*np.nonzero(seen)):
        words[t, 0] |= 1 << int(j)
    mask = (words - (words >= 1 << 31) * (1 << 32)).to(torch.int32).to(DEV)
    clean, clean_lse = attend(fq, q, [k], [v], [new], scale=D ** -0.5, mask=mask)
    bad = [(5, 0, INF), (5, 1, -INF), (17, 2, INF), (40, 3, -INF), (64, 4, INF), (70, 5, -INF),
           (33, 6, INF), (34, 6, INF), (20, 7, INF), (90, 7, -INF), (50, 8, NAN),
           (ctx - 1, 9, INF), (0, 10, -INF), (ctx + new // 2, 11, INF), (ctx - 40, 12, INF)]
    for key, col, value in bad:
        v[key, :, col] = value
    out, lse = attend(fq, q, [k], [v], [new], scale=D ** -0.5, mask=mask)
    assert torch.equal(lse, clean_lse)
    want = clean.clone()
    for col in {c for _, c, _ in bad}:
        for t in range(new):
            hit = [x for key, c, x in bad if c == col and (key < ctx or seen[t, key - ctx])]
            if hit:
                want[t, :, col] = sum(hit)
    assert torch.equal(out.nan_to_num(nan=7e9, posinf=8e9, neginf=9e9),
                       want.nan_to_num(nan=7e9, posinf=8e9, neginf=9e9))


@pytest.mark.parametrize("L", [96, 3000])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_infinite_values_far_below_the_maximum(fq, dtype, L):
    """The same where the infinite value's key is 300 nats below the row's maximum, before and
    after it: below fp32's range, and still a positive probability."""
    k, v = torch.zeros(L, 1, 64, dtype=dtype), torch.ones(L, 1, 64, dtype=dtype)
    q = torch.zeros(1, 2, 64, dtype=dtype)
    q[:, :, 0] = 1
    k[3, 0, 0], v[3, 0, 9] = -300, INF
    k[L - 5, 0, 0], v[L - 5, 0, 10] = -300, -INF
    if dtype is BF16:
        v[5, 0, 11], k[5, 0, 0] = 1e38, -300    # finite, and no more than 1e38 e^-600
    k[L // 2, 0, 0] = 300
    k[:L // 2, 0, 0] -= 1
    out, _ = attend(fq, q, [k], [v], [1])
    assert bool((out[..., 9] == INF).all()) and bool((out[..., 10] == -INF).all())
    keep = [c for c in range(64) if c not in (9, 10)]
    assert bool((out[..., keep] == 1).all())
