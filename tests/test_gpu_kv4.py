"""GPU parity of the 4-bit cache's operators (include/flexq_serve.h) with their definitions in 64
bits.  Codes, scales and read rows have to be equal; the attention's tolerances are derived in
kv4_reference.py.  Over many outputs the root mean square error is held to rounding's own as
well: a step is at most 2^-10 (fp16) or 2^-7 (bf16) of a value, and errors spread evenly over it
have 1 / sqrt(12) of it; 2 % are left for chance and for the sums before it.
"""
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


def flat(cache):
    kc, vc, sc = (t.cpu().numpy().ravel() for t in cache)
    return kc.view(np.uint32), vc.view(np.uint32), sc


def random_cache(fq, r, pages, Hkv, D, page):
    """A cache of random codes, its scales NaN."""
    cache = fq.kv4_cache(pages, Hkv, D, page, device=DEV)
    for t in cache[:2]:
        t.copy_(torch.from_numpy(r.integers(-1 << 31, 1 << 31, tuple(t.shape), dtype=np.int32)))
    cache[2].fill_(NAN)
    return cache


# ---- writing and reading -------------------------------------------------------------


def slot_map(r, T, n, kind):
    """T different slots of n, some dropped."""
    if kind == "runs":       # runs that start anywhere, apart from one another
        slots, at = [], 3
        while len(slots) < T:
            m = int(r.integers(1, 40))
            slots += range(at, at + m)
            at += m + int(r.integers(1, 5))
        slots = np.array(slots[:T])
        assert slots.max() < n
    elif kind == "row":
        slots = np.arange(5, 5 + T)
    else:
        slots = r.permutation(n)[:T]
    slots = slots.astype(np.int64)
    if T > 4:
        slots[r.integers(T)] = -1
        slots[r.integers(T)] = n
        slots[r.integers(T)] = (1 << 31) - 1
        slots[r.integers(T)] = -1 << 31
    return slots


WRITES = [(1, 1, 64, 16, "any"), (7, 8, 128, 16, "row"), (8, 3, 96, 32, "runs"), (9, 2, 256, 64, "row"),
          (63, 5, 128, 256, "runs"), (65, 4, 64, 128, "any"), (300, 2, 96, 16, "runs"),
          (130, 1, 256, 32, "row"), (200, 7, 128, 32, "any"),
          # 64 tokens a workgroup
          (4160, 8, 64, 64, "runs"), (4099, 9, 96, 32, "row"), (4097, 8, 128, 16, "any"),
          (2053, 16, 256, 16, "runs")]


@pytest.mark.parametrize("T,Hkv,D,page,kind", WRITES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_write_and_read(fq, T, Hkv, D, page, kind, dtype):
    say("write", T, Hkv, D, page, kind, dtype)
    r = rng(21, T, Hkv, D, page)
    pages = (2 * T + 60) // page + 2
    cache = random_cache(fq, r, pages, Hkv, D, page)
    wide = normal(r, (T, 2 * Hkv + 1, D), dtype, 2.0)
    wide[:, ::2, 3::17] *= 8
    wide = wide.to(DEV)
    k, v = wide[:, :Hkv], wide[:, Hkv + 1:]          # as slices of a fused projection's output
    slots = slot_map(r, T, pages * page, kind)
    want = [x.copy() for x in flat(cache)]
    ref.write(*want, k.float().cpu().numpy(), v.float().cpu().numpy(), slots, page)
    fq.kv4_cache_write(k, v, i32(slots), *cache)
    got = flat(cache)
    for g, w, name in zip(got, want, ("keys", "values", "scales")):
        assert np.array_equal(g.view(np.uint16 if name == "scales" else np.uint32),
                              w.view(np.uint16 if name == "scales" else np.uint32)) \
            or (name == "scales" and np.array_equal(g, w, equal_nan=True)), name
    # and back, through the same map, in both types: fp32's b + s c, rounded
    kept = (slots >= 0) & (slots < pages * page)
    parts = ref.read(*want, np.where(kept, slots, 0), Hkv, D, page)
    for out_type in (F16, BF16):
        for out, (c, s, b) in zip(fq.kv4_cache_read(i32(slots), *cache, dtype=out_type), parts):
            x = (c * s[..., None] + b[..., None]).astype(np.float32)
            x[~kept] = 0
            assert torch.equal(out.cpu(), torch.from_numpy(x).to(out_type))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_rows_at_the_ends_of_the_range(fq, dtype):
    """Constant, tiny, huge and infinite rows, NaN, ties between codes; two rows of one token and of
    neighbouring ones do not meet."""
    D, Hkv, page = 64, 2, 16
    top = torch.finfo(dtype).max
    rows = [torch.zeros(D), torch.full((D,), -0.0), torch.full((D,), 1.25), torch.full((D,), -7e4),
            torch.full((D,), 6e4), torch.linspace(-top, top, D, dtype=torch.float64),
            torch.linspace(0, 65504, D), torch.linspace(-65504, 65504, D),
            torch.linspace(0, 9e4, D), torch.linspace(-2.0 ** -14, 2.0 ** -14, D),
            torch.linspace(0, 2.0 ** -20, D), torch.linspace(0, 2.0 ** -24, D),
            torch.linspace(-2.0 ** -30, 2.0 ** -22, D), torch.arange(D) % 31 * 0.5,
            torch.arange(D) % 16 * 1.0, torch.linspace(100, 101, D)]
    for at, bad in ((0, NAN), (D - 1, NAN), (9, math.inf), (33, -math.inf)):
        x = torch.linspace(-1, 1, D)
        x[at] = bad
        rows.append(x)
    x = torch.stack([row.double() for row in rows]).to(dtype)
    n = len(rows)
    k = torch.stack((x, x.flip(0)), 1).contiguous()
    v = torch.stack((x.roll(3, 0), x.flip(1)), 1).contiguous()
    r = rng(22)
    cache = random_cache(fq, r, 4, Hkv, D, page)
    slots = np.arange(6, 6 + n)
    want = [a.copy() for a in flat(cache)]
    ref.write(*want, k.float().numpy(), v.float().numpy(), slots, page)
    fq.kv4_cache_write(k.to(DEV), v.to(DEV), i32(slots), *cache)
    got = flat(cache)
    assert np.array_equal(got[2], want[2], equal_nan=True)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    out = fq.kv4_cache_read(i32(slots), *cache, dtype=dtype)
    for o, part, src in zip(out, ref.read(*want, slots, Hkv, D, page), (k, v)):
        c, s, b = part
        with np.errstate(over="ignore"):
            x = torch.from_numpy((c * s[..., None] + b[..., None]).astype(np.float32)).to(dtype)
        assert torch.equal(o.cpu().nan_to_num(7, 8, 9), x.nan_to_num(7, 8, 9))
        bad = torch.from_numpy(np.isnan(s))
        assert bool(o.cpu()[bad].isnan().all()) and not bool(o.cpu()[~bad].isnan().any())
        # an element is within half a step of its row's scale, and what the scale's rounding
        # and the offset's add to that: half a step of fp16 on 15 s and on b
        err = (o.cpu().double() - src.double()).abs()[~bad]
        s0, b0 = s[..., None], b[..., None]
        s, b = torch.from_numpy(s)[~bad], torch.from_numpy(b)[~bad]
        room = 0.5 * s + 15 * (s * 2.0 ** -11 + 2.0 ** -25) + b.abs() * 2.0 ** -11 + 2.0 ** -25
        eps = torch.finfo(dtype).eps / 2
        ok = err <= room[:, None] + eps * src.double().abs()[~bad]
        # rows that reach fp16's largest value may read as more: s = fp16(131008 / 15) = 8736 and
        # 15 * 8736 - 65504 = 65536, which in fp16 is infinite
        past = torch.from_numpy(c * s0 + b0)[~bad].abs() >= 65520 if dtype == F16 else ~ok & False
        assert bool((ok | past).all()) and bool(o.cpu()[~bad][past].isinf().all())


def test_calls_that_write_neighbours_at_once(fq):
    """Two streams write the even and the odd slots of the same octets: each code is its own."""
    r = rng(23)
    T, Hkv, D, page = 256, 4, 128, 16
    cache = random_cache(fq, r, T // page, Hkv, D, page)
    k, v = normal(r, (T, Hkv, D), F16).to(DEV), normal(r, (T, Hkv, D), F16).to(DEV)
    want = [a.copy() for a in flat(cache)]
    ref.write(*want, k.float().cpu().numpy(), v.float().cpu().numpy(), np.arange(T), page)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    halves = [(k[i::2].contiguous(), v[i::2].contiguous(), i32(np.arange(i, T, 2))) for i in (0, 1)]
    torch.cuda.synchronize()
    for s, (a, b, at) in zip(streams, halves):
        with torch.cuda.stream(s):
            fq.kv4_cache_write(a, b, at, *cache)
    torch.cuda.synchronize()
    for g, w in zip(flat(cache), want):
        assert np.array_equal(g, w)


# ---- attention ------------------------------------------------------------------------


def random_tree(r, n, empty=()):
    """Ancestor masks bool [n][n]; rows in `empty` attend nothing."""
    m = np.zeros((n, n), bool)
    for t in range(n):
        p = int(r.integers(-1, t)) if t else -1
        if p >= 0:
            m[t] = m[p]
        m[t, t] = True
    for t in empty:
        if t < n:
            m[t] = False
    return m


def words_of(masks, words):
    out = np.zeros((sum(len(m) for m in masks), words), np.uint32)
    at = 0
    for m in masks:
        for t, row in enumerate(m):
            for j in np.nonzero(row)[0]:
                out[at + t, j // 32] |= np.uint32(1 << (j % 32))
        at += len(m)
    return out.view(np.int32)


def problem(fq, r, ctx, new, H, Hkv, D, page, dtype, tree, empty=(), by=1.0, spread=0.0):
    """Requests over a cache whose unused places hold NaN scales and any codes.  spread: how far,
    as a power of 2, the values' scales reach apart."""
    B = len(ctx)
    need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    pages = sum(need) + 3
    cache = random_cache(fq, r, pages, Hkv, D, page)
    order = r.permutation(pages)
    table = np.full((B, max(1, max(need)) + 1), -1)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    kc, vc, sc = flat(cache)
    sc = sc.copy().reshape(pages, Hkv, page // 16, 4, 16)
    for b in range(B):
        for i in range(ctx[b] + new[b]):
            p, row = table[b, i // page], i % page
            s = r.random((Hkv, 2)) * 0.3 + 0.2
            s[:, 1] *= 2.0 ** (r.random(Hkv) * spread - spread / 2)
            at = s * (r.standard_normal((Hkv, 2)) - 7.5)
            sc[p, :, row // 16, 0::2, row % 16] = s
            sc[p, :, row // 16, 1::2, row % 16] = at
    cache[2].copy_(torch.from_numpy(sc))
    masks = [random_tree(r, n, empty) for n in new] if tree else [None] * B
    q = normal(r, (sum(new), H, D), dtype, by)
    return {"cache": cache, "table": i32(table), "ctx": i32(ctx), "new": new, "lens": ctx,
            "cu": i32(np.concatenate(([0], np.cumsum(new)))), "q": q.to(DEV), "masks": masks,
            "words": words_of(masks, max(1, (max(new) + 31) // 32)) if tree else None,
            "page": page, "dtype": dtype}


def run(fq, p, max_new, **kw):
    words = None if p["words"] is None else torch.from_numpy(p["words"]).to(DEV)
    return fq.kv4_attention(p["q"], *p["cache"], p["table"], p["ctx"], p["cu"], tree_mask=words,
                            max_new=max_new, return_lse=True, **kw)


def check(p, out, lse, scale, window=0, sinks=0, skip=(), rms=True):
    """Every row against the definition; `skip`: requests that are not looked at."""
    q, out, lse = p["q"].double().cpu().numpy(), out.double().cpu().numpy(), lse.double().cpu().numpy()
    table, (Hkv, D) = p["table"].cpu().numpy(), (p["cache"][0].shape[1], p["q"].shape[2])
    arrays = flat(p["cache"])
    eps, least = ref.OUT_EPS[p["dtype"]], ref.OUT_ABS[p["dtype"]]
    at, wrong, off, size = 0, [], 0.0, 0.0
    for b, (ctx, n) in enumerate(zip(p["lens"], p["new"])):
        rows = slice(at, at + n)
        at += n
        if b in skip or n == 0:
            continue
        pos = np.arange(ctx + n)
        pages = table[b][pos // p["page"]]
        good = (pages >= 0) & (pages < p["cache"][0].shape[0])
        slots = np.where(good, pages, 0) * p["page"] + pos % p["page"]
        key, value = ref.read(*arrays, slots, Hkv, D, p["page"])
        seen = ref.attended(ctx, n, p["masks"][b], window, sinks) & good
        want, want_lse, tol, tol_lse = ref.attention(q[rows], key, value, seen, scale,
                                                     p["dtype"])
        err = np.abs(out[rows] - want)
        tol = tol + eps * np.abs(want) * (1 + 2.0 ** -7) + least
        wrong += [(b, *i, float(err[tuple(i)]), float(tol[tuple(i)])) for i in np.argwhere(~(err <= tol))[:3]]
        none = np.isneginf(want_lse)
        assert np.array_equal(none, np.isneginf(lse[rows]))
        assert (np.abs(lse[rows][~none] - want_lse[~none]) <= tol_lse[~none]).all()
        off += float((err ** 2).sum())
        size += float((want ** 2).sum())
    assert not wrong, wrong[:5]
    if rms and out.size >= 2048:
        assert math.sqrt(off / size) <= 2 * eps / math.sqrt(12) * 1.02, math.sqrt(off / size)


# ctx, new, H, Hkv, D, page, tree, window, sinks
ATTENTION = [
    ([37], [1], 8, 8, 128, 16, False, 0, 0),
    ([0], [1], 4, 2, 64, 16, False, 0, 0),
    ([0, 5, 0, 31], [3, 0, 0, 1], 4, 2, 64, 16, False, 0, 0),
    ([15, 16, 17, 31, 32, 33], [1] * 6, 16, 2, 128, 16, False, 0, 0),
    ([700, 129, 4, 260], [1] * 4, 40, 5, 128, 32, False, 0, 0),
    ([2500], [1], 16, 1, 128, 64, False, 0, 0),                   # one request in many shares
    ([1025, 90], [1, 1], 9, 3, 256, 128, False, 0, 0),
    ([330, 1200], [1, 1], 7, 7, 96, 256, False, 0, 0),
    ([100, 900, 3], [3, 2, 3], 16, 2, 128, 32, True, 0, 0),       # 24 rows: two groups a wave
    ([300, 40], [7, 5], 16, 2, 64, 16, True, 0, 0),               # 56 rows: two waves
    ([200, 64], [13, 1], 16, 2, 128, 16, True, 0, 0),             # 104 rows: four
    ([129], [40], 8, 2, 96, 32, True, 0, 0),                      # 160 rows: two row blocks, two words
    ([70, 1], [33, 2], 12, 2, 256, 16, True, 0, 0),               # four row blocks
    ([50], [130], 4, 1, 128, 16, False, 0, 0),                    # a chain over several row blocks
    ([900, 30, 411], [1, 1, 1], 8, 2, 128, 16, False, 100, 4),
    ([900, 30, 411], [1, 1, 1], 8, 8, 64, 32, False, 1, 0),
    ([1500], [1], 16, 2, 128, 64, False, 64, 70),
    ([640, 639, 641], [1, 1, 1], 4, 4, 96, 16, False, 32, 32),
    ([500, 60, 0], [6, 9, 4], 16, 2, 128, 16, True, 50, 3),
    ([500, 60], [6, 9], 4, 2, 256, 16, True, 3, 5),               # windows shorter than the paths
    ([400], [150], 8, 2, 128, 16, False, 40, 17),                 # a chain longer than its window
    ([3], [260], 2, 1, 64, 32, False, 20, 0),
    ([80, 20], [4, 4], 4, 2, 64, 16, False, 1000, 9),             # a window longer than all
    ([1 << 10], [2], 4, 2, 64, 16, False, 1 << 40, 1 << 40),
]


@pytest.mark.parametrize("i", range(len(ATTENTION)))
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention(fq, i, dtype):
    ctx, new, H, Hkv, D, page, tree, window, sinks = ATTENTION[i]
    say("attention", ATTENTION[i], dtype)
    p = problem(fq, rng(24, i), ctx, new, H, Hkv, D, page, dtype, tree)
    kw = dict(window=window or None, sinks=sinks)
    out, lse = run(fq, p, max(1, max(new)), **kw)
    check(p, out, lse, D ** -0.5, min(window, 1 << 30), min(sinks, 1 << 30))
    again, _ = run(fq, p, max(1, max(new)), **kw)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("window", [0, 6])
def test_rows_that_attend_nothing(fq, dtype, window):
    """A drafted token whose mask is empty over an empty context: zeros and -inf; over a
    context: the context alone (the window then ends before the drafted tokens)."""
    ctx, new = [0, 40, 0], [5, 4, 2]
    p = problem(fq, rng(25), ctx, new, 4, 2, 64, 16, dtype, True, empty=(0, 3))
    out, lse = run(fq, p, 5, window=window or None, sinks=2)
    check(p, out, lse, 0.125, window, 2 if window else 0)
    assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all())
    assert bool((out[9] == 0).all()) and bool((out[6] != 0).any())


@pytest.mark.parametrize("H", [4, 16])
@pytest.mark.parametrize("part", ["key", "value"])
def test_nan_reaches_the_rows_that_attend_it(fq, H, part):
    ctx, new = [20, 200], [9, 2]
    p = problem(fq, rng(26), ctx, new, H, 1, 128, 16, F16, True)
    seen = p["masks"][0]
    bad = 4
    seen[:, bad] = False
    seen[bad, bad] = seen[7, bad] = True
    p["words"] = words_of(p["masks"], 1)
    clean, clean_lse = run(fq, p, 9)
    check(p, clean, clean_lse, 128 ** -0.5)
    pos = 20 + bad
    page = int(p["table"][0, pos // 16])
    p["cache"][2][page, 0, pos % 16 // 16, 2 * (part == "value"), pos % 16] = NAN
    out, lse = run(fq, p, 9)
    other = [t for t in range(11) if t not in (bad, 7)]
    assert torch.equal(out[other], clean[other]) and torch.equal(lse[other], clean_lse[other])
    assert bool(out[[bad, 7]].isnan().all())
    if part == "value":
        assert torch.equal(lse, clean_lse)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_scores_and_scales_far_apart(fq, dtype):
    """Scores in the hundreds, a negative and a zero scale, values whose scales reach from 2^-12 to
    2^12, queries from tiny to large."""
    for i, (by, scale, spread) in enumerate(((20.0, 0.3, 0), (1.0, -0.5, 0), (1.0, 0.0, 0),
                                             (1.0, 0.125, 24), (6.0, 0.3, 24))):
        p = problem(fq, rng(27, i), [150, 700], [3, 1], 8, 2, 64, 16, dtype, False, by=by,
                    spread=spread)
        out, lse = run(fq, p, 3, scale=scale)
        check(p, out, lse, scale, rms=False)
    for by in (2.0 ** -12, 2.0 ** 9) if dtype == F16 else (2.0 ** -100, 2.0 ** 60):
        p = problem(fq, rng(28), [150], [2], 4, 2, 64, 16, dtype, False, by=by)
        p["q"][0, 0, ::3] *= 2.0 ** -9
        out, lse = run(fq, p, 2, scale=0.125 / by)
        check(p, out, lse, 0.125 / by, rms=False)


def test_a_key_that_takes_all_and_the_many_small_ones(fq):
    """One key 17 powers of 2 above a hundred thousand equal others, which together still are most
    of the sum."""
    n, D = 100_003, 64
    r = rng(29)
    p = problem(fq, r, [40], [1], 1, 1, D, 64, F16, False)
    pages = n // 64 + 1
    cache = fq.kv4_cache(pages, 1, D, 64, device=DEV)
    cache[0].zero_()
    cache[1].copy_(torch.from_numpy(r.integers(-1 << 31, 1 << 31, tuple(cache[1].shape),
                                               dtype=np.int32)))
    sc = torch.zeros(pages, 1, 4, 4, 16)
    sc[..., 1, :] = -17 * math.log(2) / 8              # every key b, its codes 0
    sc[..., 2, :], sc[..., 3, :] = 0.25, -1.75
    sc[0, 0, 0, 1, 5] = 0
    cache[2].copy_(sc)
    p |= {"cache": cache, "table": i32(np.arange(pages)[None]), "ctx": i32([n - 1]), "lens": [n - 1]}
    p["q"].fill_(1.0)
    out, lse = run(fq, p, 1)
    check(p, out, lse, D ** -0.5)


def test_pages_that_are_missing_are_left_out(fq):
    p = problem(fq, rng(30), [100, 130], [2, 1], 4, 2, 64, 32, F16, False)
    for bad in (-1, 1 << 20):
        for at in (0, 1, 3):
            table = p["table"].clone()
            table[0, at] = bad
            q = dict(p, table=table)
            out, lse = run(fq, q, 2)
            check(q, out, lse, 0.125)
    q = dict(p, table=torch.full_like(p["table"], -1))
    out, lse = run(fq, q, 2)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_strides_guards_streams_and_lengths_on_the_gpu(fq):
    """Queries of a wider tensor, outputs between guards, a stream of its own; rows past the last
    request's, requests longer than max_new and rows that q does not hold are left as they were."""
    ctx, new = [40, 3], [2, 5]
    p = problem(fq, rng(31), ctx, new, 8, 2, 64, 16, F16, False)
    wide = torch.zeros(9, 12, 72, dtype=F16, device=DEV)
    wide[:7, 2:10, :64] = p["q"]
    want, want_lse = run(fq, p, 5)
    check(p, want, want_lse, 0.125)
    buf = torch.full((9 * 8 * 64 + 64,), 3.0, dtype=F16, device=DEV)
    out = buf[16:16 + 9 * 8 * 64].view(9, 8, 64)
    lse = torch.full((9, 8), 5.0, device=DEV)
    ws = torch.empty(fq.kv4_attention_workspace_bytes(2, 5, 8, 2, 64), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fq.kv4_attention(wide[:, 2:10, :64], *p["cache"], p["table"], p["ctx"], p["cu"], max_new=5,
                         out=out, lse=lse, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out[:7], want) and torch.equal(lse[:7], want_lse)
    assert bool((out[7:] == 3).all()) and bool((lse[7:] == 5).all())
    assert bool((buf[:16] == 3).all()) and bool((buf[16 + 9 * 8 * 64:] == 3).all())
    # three of the second request's five tokens
    out.fill_(3.0)
    fq.kv4_attention(wide[:, 2:10, :64], *p["cache"], p["table"], p["ctx"], p["cu"], max_new=3,
                     out=out)
    assert torch.equal(out[:5], want[:5]) and bool((out[5:] == 3).all())
    # cu_new reaches past the rows there are
    out = fq.kv4_attention(p["q"][:4].contiguous(), *p["cache"], p["table"], p["ctx"], p["cu"],
                           max_new=5)
    assert torch.equal(out, want[:4])


def test_many_requests(fq):
    r = rng(32)
    ctx = r.integers(0, 90, 300).tolist()
    new = r.integers(0, 3, 300).tolist()
    p = problem(fq, r, ctx, new, 4, 2, 64, 16, BF16, False)
    out, lse = run(fq, p, 2)
    check(p, out, lse, 0.125)
    out, lse = run(fq, p, 2, window=20, sinks=3)
    check(p, out, lse, 0.125, 20, 3)


def test_step_in_a_graph(fq):
    """A step captured once, tables to attention, and replayed with other lengths, between eager
    work: the eager results every time.  Two graphs with workspaces of their own."""
    r = rng(33)
    B, H, Hkv, D, page, most = 3, 8, 2, 128, 16, 12
    cache = fq.kv4_cache(64, Hkv, D, page, device=DEV)
    for t in cache:
        t.zero_()
    table = torch.full((B, 12), -1, dtype=torch.int32, device=DEV)
    free = torch.arange(64, dtype=torch.int32, device=DEV)
    ctx, new, head = i32([0] * B), i32([4, 1, 3]), i32([0])
    q = torch.zeros(most, H, D, dtype=F16, device=DEV)
    kv = torch.zeros(most, 2 * Hkv, D, dtype=F16, device=DEV)

    def step(cache, table, head):
        slots, cu, counts = fq.block_tables(ctx, new, free, table, page, most, free_head=head)
        fq.kv4_cache_write(kv[:, :Hkv], kv[:, Hkv:], slots, *cache)
        out = torch.zeros(most, H, D, dtype=F16, device=DEV)
        lse = torch.zeros(most, H, device=DEV)
        fq.kv4_attention(q, *cache, table, ctx, cu, max_new=4, window=24, sinks=2, out=out, lse=lse)
        back = fq.kv4_cache_read(slots, *cache)
        head.copy_(counts[2:])
        return out, lse, back

    twin = [t.clone() for t in cache], table.clone(), head.clone()
    step([t.clone() for t in cache], table.clone(), head.clone())     # loads the kernels
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(cache, table, head)
    for i in range(12):
        new.copy_(i32(r.integers(0, 5, B)))
        q.copy_(normal(r, (most, H, D), F16))
        kv.copy_(normal(r, (most, 2 * Hkv, D), F16))
        torch.cuda.synchronize()
        graph.replay()
        want = step(*twin)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), i
        assert torch.equal(got[2][0], want[2][0]) and torch.equal(got[2][1], want[2][1]), i
        for a, b in zip(cache, twin[0]):
            assert torch.equal(a, b), i
        ctx.add_(new)
    assert int(ctx.sum()) > 30


@pytest.mark.parametrize("ctx,H,Hkv,D,page,first", [(300_001, 8, 2, 64, 128, 0),
                                                    (70_000, 2, 2, 128, 64, 40_000)])
def test_long_contexts_and_large_caches(fq, ctx, H, Hkv, D, page, first):
    """Contexts of hundreds of thousands of tokens; codes past 2^32 bytes of a cache."""
    pages = (ctx + page) // page + first
    while first and pages * Hkv * page * D // 2 < (1 << 32) + (1 << 28):
        pages += 1000
    g = torch.Generator(device=DEV).manual_seed(5)
    cache = fq.kv4_cache(pages, Hkv, D, page, device=DEV)
    use = torch.arange(pages - (ctx + page) // page, pages, device=DEV).flip(0)
    for t in cache[:2]:
        part = torch.randint(-1 << 31, 1 << 31, (len(use), *t.shape[1:]), generator=g, device=DEV)
        t[use] = part.to(torch.int32)
    cache[2][use] = torch.tensor([0.25, -2.0, 0.5, -3.75], dtype=F16, device=DEV)[:, None]
    table = use.to(torch.int32)[None].contiguous()
    q = torch.randn(1, H, D, generator=g, device=DEV).to(F16)
    out, lse = fq.kv4_attention(q, *cache, table, i32([ctx - 1]), i32([0, 1]), return_lse=True)
    slots = torch.arange(ctx, device=DEV)
    slots = (use[slots // page] * page + slots % page).to(torch.int32)
    k = torch.empty(ctx, Hkv, D, dtype=torch.float64, device=DEV)
    v = torch.empty_like(k)
    for at in range(0, ctx, 1 << 16):                  # (codes times a power of 2: exact in fp16)
        a, b = fq.kv4_cache_read(slots[at:at + (1 << 16)], *cache)
        k[at:at + len(a)], v[at:at + len(b)] = a, b
    for h in range(H):
        s = k[:, h // (H // Hkv)] @ q[0, h].double() * D ** -0.5
        want = torch.softmax(s, 0) @ v[:, h // (H // Hkv)]
        assert abs(float(lse[0, h]) - float(torch.logsumexp(s, 0))) < 2e-5
        # scores to 2^-18 or so, probabilities in proportion, sums over ten thousand steps
        room = 2.0 ** -16 * float(v.abs().max()) + 2.0 ** -11 * want.abs()
        assert bool(((out[0, h].double() - want).abs() <= room).all())
