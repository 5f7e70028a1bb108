"""GPU parity of the decoding-step operators (include/flexq_serve.h) with their
definitions in 64 bits: 4-bit matrix-vector products, block tables and slot maps, cache
writes and attention of drafted tokens.  Tolerances are derived in serve_reference.py;
integers and copies have to be equal.
"""
import math

import numpy as np
import pytest

import serve_reference as ref

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


# ---- 4-bit weights -------------------------------------------------------------------


@pytest.mark.parametrize("N,K,group", [(16, 128, 128), (48, 384, 32), (80, 2176, 64)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_pack_w4(fq, N, K, group, dtype):
    say("pack_w4", N, K, group, dtype)
    r = rng(1, N, K, group)
    w = normal(r, (N, K), dtype, 0.02)
    w[0, :group] = 0                        # scale 0, codes 0
    w[1, 0] = 1.0                           # one large weight: the others round to 0
    w[2, :group] = torch.arange(group) % 15 - 7.0
    w[3, :8] = torch.tensor([7, 3.5, -3.5, 2.5, -0.5, 0.5, 1.5, -6.5])   # ties to even
    q, s = ref.quantize_w4(w.float().numpy(), group)
    w4, sw = fq.pack_w4(w.to(DEV), group)
    assert np.array_equal(w4.cpu().numpy().view(np.uint32), ref.pack_w4(q))
    assert np.array_equal(sw.cpu().numpy().T.view(np.uint16), s.view(np.uint16))


GEMV = [(1, 16, 128, 128), (1, 48, 4096, 128), (2, 80, 384, 32), (5, 208, 1152, 64),
        (13, 1040, 2176, 128), (16, 64, 256, 64), (17, 176, 896, 32), (33, 144, 640, 128),
        (64, 96, 512, 64), (65, 48, 384, 128), (130, 32, 1280, 32), (3, 16, 16512, 128),
        (1, 12304, 256, 64), (40, 4112, 128, 128),
        # two tiles an item with an odd one left, K in slices with a short last chunk, more
        # rows than the activations' room in LDS allows the few-rows kernel
        (2, 32784, 128, 32), (9, 272, 4224, 128), (28, 528, 3200, 32), (61, 336, 2432, 64),
        (4, 48, 8320, 128)]


@pytest.mark.parametrize("M,N,K,group", GEMV)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_gemv_w4(fq, M, N, K, group, dtype):
    say("gemv_w4", M, N, K, group, dtype)
    r = rng(2, M, N, K)
    q = r.integers(-8, 8, (N, K))
    s = (r.random((N, K // group)) * 0.01 + 1e-3).astype(np.float16)
    x = normal(r, (M, K), dtype)
    x[:, ::97] *= 20
    w4 = torch.from_numpy(ref.pack_w4(q).view(np.int32)).to(DEV)
    sw = torch.from_numpy(np.ascontiguousarray(s.T)).to(DEV)
    y = fq.gemv_w4(x.to(DEV), w4, sw, N)
    want, sums = ref.gemv(x.double().numpy(), q, s, group)
    tol = ref.gemv_tolerance(want, sums, dtype)
    err = np.abs(y.double().cpu().numpy() - want)
    assert (err <= tol).all(), (float((err / tol).max()), np.argwhere(err > tol)[:4].tolist())
    assert torch.equal(y, fq.gemv_w4(x.to(DEV), w4, sw, N))


@pytest.mark.parametrize("M,N,K,group", [(40, 32816, 256, 128), (64, 32816, 384, 64),
                                         (70, 32816, 384, 32), (3, 32816, 384, 32),
                                         (2, 9616, 1152, 64), (4, 9616, 384, 128)])
def test_gemv_w4_wide_weights(fq, M, N, K, group):
    """Weights with more tiles than workgroups, odd numbers of them; one row is infinite."""
    say("gemv_w4, wide", M, N, K, group)
    r = rng(61, M, N, K, group)
    q = r.integers(-7, 8, (N, K))
    s = (r.random((N, K // group)) * 0.01).astype(np.float16)
    x = normal(r, (M, K), F16)
    x[M - 1, 37] = float("inf")
    w4 = torch.from_numpy(ref.pack_w4(q).view(np.int32)).to(DEV)
    y = fq.gemv_w4(x.to(DEV), w4, torch.from_numpy(np.ascontiguousarray(s.T)).to(DEV), N)
    y = y.double().cpu().numpy()
    want, sums = ref.gemv(x[:M - 1].double().numpy(), q, s, group)
    assert (np.abs(y[:M - 1] - want) <= ref.gemv_tolerance(want, sums, F16)).all()
    code = np.where(s[:, 37 // group] == 0, 0, q[:, 37])
    assert np.array_equal(y[M - 1], np.where(code == 0, NAN, np.where(code > 0, np.inf, -np.inf)),
                          equal_nan=True)


def test_gemv_w4_strided_rows_guards_and_stream(fq):
    """Rows of a wider tensor, an output between guards, a stream of its own."""
    r = rng(3)
    M, N, K = 7, 96, 384
    q = r.integers(-7, 8, (N, K))
    s = (r.random((N, K // 128)) * 0.01).astype(np.float16)
    wide = normal(r, (M, K + 64), F16).to(DEV)
    x = wide[:, 8:8 + K]
    w4 = torch.from_numpy(ref.pack_w4(q).view(np.int32)).to(DEV)
    sw = torch.from_numpy(np.ascontiguousarray(s.T)).to(DEV)
    buf = torch.full((M * N + 64,), -1, dtype=torch.int16, device=DEV)
    y = buf[4:4 + M * N].view(F16).view(M, N)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fq.gemv_w4(x, w4, sw, N, y=y)
    torch.cuda.current_stream().wait_stream(side)
    want, sums = ref.gemv(x.double().cpu().numpy(), q, s, 128)
    assert (np.abs(y.double().cpu().numpy() - want) <= ref.gemv_tolerance(want, sums, F16)).all()
    assert bool((buf[:4] == -1).all()) and bool((buf[4 + M * N:] == -1).all())


def test_gemv_w4_propagates_infinities_and_nan(fq):
    """A NaN activation reaches its row alone; a zero scale gives zeros."""
    M, N, K = 3, 32, 256
    q = np.ones((N, K), np.int64)
    s = np.full((N, 2), 0.5, np.float16)
    s[5] = 0
    x = torch.ones(M, K, dtype=F16)
    x[1, 200] = NAN
    w4 = torch.from_numpy(ref.pack_w4(q).view(np.int32)).to(DEV)
    y = fq.gemv_w4(x.to(DEV), w4, torch.from_numpy(np.ascontiguousarray(s.T)).to(DEV), N).cpu()
    want = torch.full((N,), 128.0, dtype=F16)
    want[5] = 0
    assert torch.equal(y[0], want) and torch.equal(y[2], want)
    assert bool(y[1].isnan().all())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_gemv_w4_infinities_and_the_top_of_the_range(fq, dtype, group):
    """Infinite activations give infinities of the code's sign (NaN for a zero code), and
    activations at the top of the type's range whose sums stay finite are summed."""
    M, N, K = 20, 64, 256
    r = rng(16, group)
    q = r.integers(-7, 8, (N, K))
    s = np.full((N, K // group), 2.0 ** -8, np.float16)
    x = normal(r, (M, K), dtype)
    x[3, 130] = float("inf")
    x[17, 5] = -float("inf")
    big = torch.finfo(dtype).max
    x[6] = 0
    x[6, 10], x[6, 11] = big, -big
    w4 = torch.from_numpy(ref.pack_w4(q).view(np.int32)).to(DEV)
    y = fq.gemv_w4(x.to(DEV), w4, torch.from_numpy(np.ascontiguousarray(s.T)).to(DEV), N)
    y = y.double().cpu().numpy()
    for row, k, sign in ((3, 130, 1), (17, 5, -1)):
        want = np.where(q[:, k] == 0, NAN, np.where(sign * q[:, k] > 0, np.inf, -np.inf))
        assert np.array_equal(y[row], want, equal_nan=True)
    # products and their sum are fp32: in bfloat16 those of larger codes pass its range
    a, b = float(big) * q[:, 10], float(big) * q[:, 11]
    fits = np.maximum(np.maximum(np.abs(a), np.abs(b)), np.abs(a - b)) < 3.4e38
    assert fits.any()
    assert np.allclose(y[6][fits], ((a - b) * 2.0 ** -8)[fits], rtol=2.0 ** -7)
    other = [m for m in range(M) if m not in (3, 6, 17)]
    want, sums = ref.gemv(x[other].double().numpy(), q, s, group)
    assert (np.abs(y[other] - want) <= ref.gemv_tolerance(want, sums, dtype)).all()


def test_w4_linear(fq):
    r = rng(4)
    w, x = normal(r, (64, 256), BF16, 0.02), normal(r, (3, 256), BF16)
    layer = fq.W4Linear(w.to(DEV), group=32)
    q, s = ref.quantize_w4(w.float().numpy(), 32)
    want, sums = ref.gemv(x.double().numpy(), q, s, 32)
    y = layer(x.to(DEV)).double().cpu().numpy()
    assert (np.abs(y - want) <= ref.gemv_tolerance(want, sums, BF16)).all()


# ---- block tables --------------------------------------------------------------------


@pytest.mark.parametrize("B,ctx_hi,new_hi,page", [(1, 0, 1, 16), (1, 40, 1, 16), (5, 70, 9, 16),
                                                  (64, 300, 1, 32), (300, 100, 40, 16),
                                                  (700, 65, 3, 64), (4096, 30, 2, 16),
                                                  (3, 0, 5000, 128), (9, 20, 30, 1),
                                                  (37, 100, 36000, 16), (6, 5, 300000, 128)])
def test_block_tables(fq, B, ctx_hi, new_hi, page):
    say("block_tables", B, ctx_hi, new_hi, page)
    r = rng(5, B, page)
    ctx, new = r.integers(0, ctx_hi + 1, B), r.integers(0, new_hi + 1, B)
    cols = int(max(1, (-(-(ctx + new) // page)).max())) + 2
    table = r.integers(0, 1 << 20, (B, cols)).astype(np.int32)
    free = r.permutation(1 << 17).astype(np.int32)
    most = int(new.sum()) + 37
    head = int(r.integers(0, 100))
    want = ref.block_tables(ctx, new, free, table, page, most, head)
    d_table = i32(table)
    slots, cu, counts = fq.block_tables(i32(ctx), i32(new), i32(free), d_table, page, most,
                                        free_head=i32([head]))
    for got, w in zip((d_table, slots, cu, counts), want):
        assert np.array_equal(got.cpu().numpy().astype(np.int64), w)


def test_block_tables_that_end_too_soon(fq):
    """Too few free pages, too narrow tables, a slot map shorter than the tokens,
    negative lengths, missing pages in what a request holds, no request at all."""
    ctx, new = np.array([5, -3, 33, 0, 16]), np.array([40, 20, 16, -1, 90])
    table = np.array([[7, 1, 2], [9, 9, 9], [3, 4, -1], [0, 0, 0], [11, 5, 5]], np.int32)
    free = np.array([100, 101, 102, 103], np.int32)
    for most in (0, 60, 200):
        want = ref.block_tables(ctx, new, free, table, 16, most, 1)
        d_table = i32(table)
        got = fq.block_tables(i32(ctx), i32(new), i32(free), d_table, 16, most,
                              free_head=i32([1]))
        for g, w in zip((d_table, *got), want):
            assert np.array_equal(g.cpu().numpy().astype(np.int64), w), (most, g, w)
    empty = torch.zeros((0, 4), dtype=torch.int32, device=DEV)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    slots, cu, counts = fq.block_tables(none, none, none, empty, 16, 5)
    assert slots.tolist() == [-1] * 5 and cu.tolist() == [0] and counts.tolist() == [0, 0, 0]


# ---- cache writes --------------------------------------------------------------------


@pytest.mark.parametrize("T,Hkv,D,page", [(1, 1, 64, 16), (5, 8, 128, 16), (37, 3, 96, 32),
                                          (200, 2, 256, 64), (513, 5, 128, 128),
                                          (300, 2, 64, 256)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_kv_cache_write(fq, T, Hkv, D, page, dtype):
    """Runs of consecutive slots that start anywhere, scattered slots, slots outside
    the cache; keys and values as slices of a fused projection's output."""
    say("kv_cache_write", T, Hkv, D, page, dtype)
    r = rng(6, T, D)
    pages = -(-T // page) * 2 + 3
    kv = normal(r, (T, 2 * Hkv + 1, D), dtype).to(DEV)
    k, v = kv[:, 1:1 + Hkv], kv[:, 1 + Hkv:]
    start = int(r.integers(0, page))
    runs = (np.arange(T) + start) % (pages * page)
    scattered = r.permutation(pages * page)[:T]
    for slots in (runs, scattered, np.where(r.random(T) < 0.3, -1, scattered),
                  np.where(np.arange(T) % 5 == 0, pages * page, runs)):
        kc, vc = fq.kv_cache(pages, Hkv, D, page, dtype, DEV)
        kc.fill_(3), vc.fill_(5)
        want_k = kc.cpu().view(torch.int16).numpy().ravel().copy()
        want_v = vc.cpu().view(torch.int16).numpy().ravel().copy()
        ref.write_cache(want_k, want_v, k.cpu().contiguous().view(torch.int16).numpy(),
                        v.cpu().contiguous().view(torch.int16).numpy(), slots, page)
        fq.kv_cache_write(k, v, i32(slots), kc, vc)
        assert np.array_equal(kc.cpu().view(torch.int16).numpy().ravel(), want_k)
        assert np.array_equal(vc.cpu().view(torch.int16).numpy().ravel(), want_v)


# ---- attention -----------------------------------------------------------------------


def random_tree(r, n, empty=()):
    """Ancestor masks of a random tree of n drafted tokens; tokens in `empty` attend no
    drafted token at all."""
    seen = np.zeros((n, n), bool)
    for t in range(n):
        parent = int(r.integers(-1, t)) if t else -1
        if parent >= 0:
            seen[t] = seen[parent]
        seen[t, t] = True
    for t in empty:
        if t < n:
            seen[t] = False
    return seen


def words_of(masks, words):
    out = np.zeros((sum(m.shape[0] for m in masks), words), np.uint32)
    at = 0
    for m in masks:
        for t in range(m.shape[0]):
            for j in np.nonzero(m[t])[0]:
                out[at + t, j // 32] |= np.uint32(1 << (j % 32))
        at += m.shape[0]
    return torch.from_numpy(out.view(np.int32)).to(DEV)


def fill(v, kind):
    """Unused places: NaN, or infinities of both signs."""
    if kind == "nan":
        v.fill_(NAN)
    else:
        v.view(-1)[0::2] = float("inf")
        v.view(-1)[1::2] = -float("inf")


def problem(r, ctx, new, H, Hkv, D, page, dtype, tree, poison="nan", empty=(), by=1.0):
    """Keys and values of every request in a shuffled cache whose other places are
    poisoned, and what the call takes."""
    import w6a6_w6a8_integer_amd as fq
    need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    pages = sum(need) + 3
    order = r.permutation(pages)
    table = np.full((len(ctx), max(1, max(need)) + 1), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    kc, vc = fq.kv_cache(pages, Hkv, D, page, dtype, "cpu")
    fill(kc, poison), fill(vc, poison)
    keys, values = [], []
    h, d = np.meshgrid(np.arange(Hkv), np.arange(D), indexing="ij")
    for b, (c, n) in enumerate(zip(ctx, new)):
        k, v = normal(r, (c + n, Hkv, D), dtype, by), normal(r, (c + n, Hkv, D), dtype)
        keys.append(k), values.append(v)
        for i in range(c + n):
            slot = int(table[b, i // page]) * page + i % page
            ik, iv = ref.cache_index(slot, h, d, Hkv, D, page)
            kc.view(-1)[torch.from_numpy(ik)] = k[i]
            vc.view(-1)[torch.from_numpy(iv)] = v[i]
    q = normal(r, (sum(new), H, D), dtype, 1.5)
    masks = [random_tree(r, n, empty) if tree else np.tril(np.ones((n, n), bool)) for n in new]
    words = words_of(masks, (max(max(new), 1) + 31) // 32) if tree else None
    return dict(q=q, keys=keys, values=values, masks=masks, kc=kc.to(DEV), vc=vc.to(DEV),
                table=i32(table), ctx=i32(ctx), cu=i32(np.concatenate(([0], np.cumsum(new)))),
                words=words)


def check(p, ctx, new, dtype, out, lse, scale):
    at = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        want, want_lse, tol, tol_lse = ref.attention(
            p["q"][at:at + n].double(), p["keys"][b].double(), p["values"][b].double(), c, n,
            torch.from_numpy(p["masks"][b]), scale)
        got, got_lse = out[at:at + n].double().cpu(), lse[at:at + n].double().cpu()
        tol = tol + ref.OUT_EPS[dtype] * want.abs() * (1 + 2.0 ** -7) + ref.OUT_ABS[dtype]
        err = (got - want).abs()
        assert bool((err <= tol).all()), (b, float((err / tol).max()), bool(got.isnan().any()))
        none = torch.isinf(want_lse)
        assert torch.equal(none, torch.isinf(got_lse)) and bool((got_lse[none] < 0).all())
        assert bool(((got_lse - want_lse).abs()[~none] <= tol_lse[~none]).all())
        at += n


def run(fq, p, max_new, **kw):
    return fq.tree_attention(p["q"].to(DEV), p["kc"], p["vc"], p["table"], p["ctx"], p["cu"],
                             tree_mask=p["words"], max_new=max_new, return_lse=True, **kw)


ATTENTION = [
    # ctx, new, H, Hkv, D, page, tree
    ([0], [1], 1, 1, 64, 16, False),                    # one key in all
    ([37], [1], 4, 4, 128, 16, False),
    ([15, 16, 17, 31, 32, 33], [1] * 6, 8, 2, 128, 16, False),   # around a page and a step
    ([130, 0, 7, 64], [1, 3, 2, 5], 8, 1, 96, 32, True),
    ([63, 200], [13, 6], 14, 2, 128, 16, True),         # 7 heads a key head: ragged rows
    ([5, 0, 97], [48, 33, 1], 2, 2, 64, 64, True),      # masks of two words
    ([100], [21], 16, 1, 256, 16, True),                # 336 rows of one key head
    ([0, 0], [70, 64], 4, 2, 128, 128, False),          # a prompt: a chain over nothing
    ([300, 0, 11, 0], [2, 0, 3, 0], 6, 3, 64, 256, True),        # requests without new tokens
    ([1500], [1], 2, 1, 128, 16, False),
    ([2500, 3], [4, 9], 4, 1, 64, 32, True),
    ([700, 1, 300], [1, 1, 1], 32, 2, 128, 16, False),  # 16 heads a key head
    # many rows of one key head (32 a wave), ragged, with masks, and over several row blocks
    ([90, 7], [13, 17], 16, 2, 64, 16, True),
    ([45, 300], [40, 9], 8, 2, 96, 32, True),
    ([130, 0, 64], [33, 18, 40], 8, 1, 128, 64, True),
    ([11], [75], 4, 2, 96, 16, False),
    # long enough for many parts, of few rows and of many
    ([9000], [2], 4, 2, 96, 16, False),
    ([6000, 20], [3, 1], 16, 1, 256, 16, True),
    ([7000], [18], 4, 1, 64, 16, True),
]


@pytest.mark.parametrize("i", range(len(ATTENTION)))
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_tree_attention(fq, i, dtype):
    ctx, new, H, Hkv, D, page, tree = ATTENTION[i]
    say("tree_attention", *ATTENTION[i], dtype)
    p = problem(rng(7, i), ctx, new, H, Hkv, D, page, dtype, tree,
                poison="nan" if i % 2 else "inf")
    out, lse = run(fq, p, max(new))
    check(p, ctx, new, dtype, out, lse, 1 / math.sqrt(D))
    again, _ = run(fq, p, max(new))
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_rows_that_attend_nothing(fq, dtype):
    """A drafted token whose mask is empty over an empty context: zeros and -inf; over a
    context: the context alone."""
    ctx, new = [0, 40, 0], [5, 4, 2]
    p = problem(rng(8), ctx, new, 4, 2, 64, 16, dtype, True, empty=(0, 3))
    out, lse = run(fq, p, 5)
    check(p, ctx, new, dtype, out, lse, 0.125)
    assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all())
    assert bool((out[9] == 0).all()) and bool((out[6] != 0).any())


@pytest.mark.parametrize("kind", ["nan", "inf"])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("H", [4, 16])
def test_infinities_and_nan_in_masked_places(fq, dtype, kind, H):
    """A drafted token with NaN or infinite keys and values spoils the rows that attend it
    and no other (36 rows and, in wider tiles, 144)."""
    ctx, new = [20], [9]
    p = problem(rng(9), ctx, new, H, 1, 128, 16, dtype, True)
    seen = p["masks"][0]
    bad = 4
    seen[:, bad] = False
    seen[bad, bad] = True
    seen[7, bad] = True
    p["words"] = words_of([seen], 1)
    clean, clean_lse = run(fq, p, 9)
    check(p, ctx, new, dtype, clean, clean_lse, 128 ** -0.5)
    h, d = np.meshgrid(np.arange(1), np.arange(128), indexing="ij")
    slot = int(p["table"][0, (20 + bad) // 16]) * 16 + (20 + bad) % 16
    ik, iv = (torch.from_numpy(x.ravel()).to(DEV) for x in ref.cache_index(slot, h, d, 1, 128, 16))
    p["vc"].view(-1)[iv[3:50]] = NAN if kind == "nan" else float("inf")
    out, lse = run(fq, p, 9)
    other = [t for t in range(9) if t not in (bad, 7)]
    assert torch.equal(out[other], clean[other]) and torch.equal(lse, clean_lse)
    assert not bool(torch.isfinite(out[[bad, 7]][:, :, 3:50]).any())
    assert torch.equal(out[[bad, 7]][:, :, 50:], clean[[bad, 7]][:, :, 50:])
    p["kc"].view(-1)[ik] = NAN if kind == "nan" else float("inf")
    out, lse = run(fq, p, 9)
    assert torch.equal(out[other], clean[other]) and torch.equal(lse[other], clean_lse[other])
    assert not bool(torch.isfinite(out[[bad, 7]][..., 3:50]).any())


def test_large_scores_and_scale(fq):
    """Scores in the hundreds (one key takes all), a negative and a zero scale, and a
    maximum that rises with every key."""
    for by, scale in ((20.0, 0.3), (1.0, -0.5), (1.0, 0.0)):
        ctx, new = [150], [3]
        p = problem(rng(10), ctx, new, 2, 1, 64, 16, F16, False, by=by)
        out, lse = run(fq, p, 3, scale=scale)
        check(p, ctx, new, F16, out, lse, scale)
    ctx, new = [900], [1]
    p = problem(rng(11), ctx, new, 1, 1, 64, 16, F16, False)
    p["q"][:] = 1.0
    ramp = torch.linspace(-3, 3, 901).to(F16)
    h, d = np.meshgrid(np.arange(1), np.arange(64), indexing="ij")
    p["keys"][0] = ramp[:, None, None].expand(901, 1, 64).contiguous()
    kc = p["kc"].cpu()
    table = p["table"].cpu().numpy()
    for i in range(901):
        ik, _ = ref.cache_index(int(table[0, i // 16]) * 16 + i % 16, h, d, 1, 64, 16)
        kc.view(-1)[torch.from_numpy(ik)] = ramp[i]
    p["kc"] = kc.to(DEV)
    out, lse = run(fq, p, 1, scale=0.5)
    check(p, ctx, new, F16, out, lse, 0.5)


def test_pages_that_are_missing_are_left_out(fq):
    """A table entry outside the cache takes its 16-token blocks out of the attention."""
    ctx, new = [100], [2]
    p = problem(rng(12), ctx, new, 2, 1, 64, 32, F16, False)
    for bad in (-1, 1 << 20):
        table = p["table"].clone()
        table[0, 1] = bad
        out, lse = fq.tree_attention(p["q"].to(DEV), p["kc"], p["vc"], table, p["ctx"], p["cu"],
                                     max_new=2, return_lse=True)
        keep = [i for i in range(102) if i // 32 != 1]
        short = dict(p, keys=[p["keys"][0][keep]], values=[p["values"][0][keep]])
        check(short, [68], [2], F16, out, lse, 0.125)


def test_strided_queries_guards_and_lengths_on_the_gpu(fq):
    """Queries as slices of a fused projection, rows past the new tokens untouched, a
    table wider than needed, wide masks, tokens past max_new not computed."""
    ctx, new = [33, 70], [4, 3]
    p = problem(rng(13), ctx, new, 4, 2, 64, 16, BF16, True)
    wide = torch.zeros(9, 8, 64, dtype=BF16, device=DEV)
    wide[:7, 2:6] = p["q"].to(DEV)
    words = torch.zeros(9, 3, dtype=torch.int32, device=DEV)
    words[:7, 0] = p["words"][:, 0]
    words[:, 1:] = -1                      # bits of tokens that do not exist
    out = torch.full((9, 4, 64), 7.0, dtype=BF16, device=DEV)
    lse = torch.full((9, 4), 7.0, device=DEV)
    got = fq.tree_attention(wide[:, 2:6], p["kc"], p["vc"], p["table"], p["ctx"], p["cu"],
                            tree_mask=words, max_new=60, out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    check(p, ctx, new, BF16, out[:7], lse[:7], 0.125)
    assert bool((out[7:] == 7).all()) and bool((lse[7:] == 7).all())
    out.fill_(7.0)
    fq.tree_attention(wide[:, 2:6], p["kc"], p["vc"], p["table"], p["ctx"], p["cu"],
                      tree_mask=words, max_new=3, out=out)
    assert bool((out[3] == 7).all()) and bool((out[4:7] != 7).any())


def test_many_requests(fq):
    """More requests than a workgroup has threads, most of a token or two."""
    r = rng(14)
    ctx = r.integers(0, 40, 400).tolist()
    new = r.integers(0, 3, 400).tolist()
    ctx[17], ctx[399] = 3000, 1999
    p = problem(r, ctx, new, 2, 1, 64, 16, F16, False)
    out, lse = run(fq, p, 2)
    check(p, ctx, new, F16, out, lse, 0.125)


# ---- a step of all of them -----------------------------------------------------------


def test_step_in_a_graph(fq):
    """Block tables, cache write and attention of a step in one captured graph, replayed
    for steps of different lengths with eager work between, against eager calls."""
    r = rng(15)
    B, Hkv, H, D, page, most = 5, 2, 4, 64, 16, 24
    pages = 64
    free = i32(r.permutation(pages))
    state = dict(ctx=i32([0] * B), new=i32([0] * B), head=i32([0]),
                 table=torch.full((B, 8), -1, dtype=torch.int32, device=DEV))
    qkv = torch.zeros(most, H + 2 * Hkv, D, dtype=F16, device=DEV)
    kc, vc = fq.kv_cache(pages, Hkv, D, page, F16, DEV)
    kc.zero_(), vc.zero_()
    slots = torch.empty(most, dtype=torch.int32, device=DEV)
    cu = torch.empty(B + 1, dtype=torch.int32, device=DEV)
    counts = torch.empty(3, dtype=torch.int32, device=DEV)
    out = torch.empty(most, H, D, dtype=F16, device=DEV)
    ws = torch.empty(fq.tree_attention_workspace_bytes(B, most, H, Hkv, D), dtype=torch.uint8,
                     device=DEV)

    def step(kc, vc, table, out):
        fq.block_tables(state["ctx"], state["new"], free, table, page, most,
                        free_head=state["head"], slot_map=slots, cu_new=cu, counts=counts)
        fq.kv_cache_write(qkv[:, H:H + Hkv], qkv[:, H + Hkv:], slots, kc, vc)
        fq.tree_attention(qkv[:, :H], kc, vc, table, state["ctx"], cu, max_new=most, out=out,
                          workspace=ws)

    step(kc, vc, state["table"], out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(kc, vc, state["table"], out)
    scratch = torch.empty(256, 1024, device=DEV)
    eager = [x.clone() for x in (kc, vc, state["table"], out)]
    for rep in range(5):
        new = r.integers(0, 6, B) if rep else np.array([most - 8, 2, 0, 5, 1])
        state["new"].copy_(i32(new))
        qkv.copy_(normal(r, tuple(qkv.shape), F16))
        out.fill_(NAN), eager[3].fill_(NAN), ws.fill_(0xAB)
        scratch.normal_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        first = counts.tolist()
        step(*eager)
        torch.cuda.synchronize()
        n = int(new.sum())
        assert first[0] == n and counts.tolist() == first
        assert torch.equal(state["table"], eager[2])
        assert torch.equal(kc, eager[0]) and torch.equal(vc, eager[1])
        assert torch.equal(out[:n], eager[3][:n]) and bool(torch.isfinite(out[:n]).all())
        assert bool(out[n:].isnan().all())
        state["ctx"].add_(state["new"])
        state["head"].copy_(counts[2:3])
