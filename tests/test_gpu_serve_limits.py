"""GPU tests of the decoding-step operators at the ends of what they accept: strides of axes
of length one, the most weight rows, the forms that large calls take, long contexts and
caches whose offsets pass 32 bits.
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


@pytest.fixture(scope="module")
def fq():
    import w6a6_w6a8_integer_amd as fq
    fq.lib()
    return fq


def say(*a):
    print(*a, flush=True)


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def gather(cache_k, cache_v, slots, page):
    """Keys and values [slots][Hkv][D] as they stand in a cache (the header's layout)."""
    s = torch.as_tensor(slots, device=DEV).long()
    at, block, r = s // page, s % page // 16, s % 16
    k = cache_k[at, :, block, :, r]
    return k.reshape(len(s), cache_k.shape[1], -1), cache_v[at, :, block, :, r]


def test_strides_of_axes_of_length_one(fq):
    """A single token, and a single head, from a tensor whose rows are no multiple of eight
    elements apart: the stride of an axis of length one is never used."""
    D, page = 64, 16
    g = torch.Generator(device=DEV).manual_seed(1)
    wide = torch.randn(2, 3 * 2 * D + 4, generator=g, device=DEV).half()
    one = wide[:, :6 * D].unflatten(1, (6, D))[:1]       # [1][6][D], 388 elements a token
    assert one.stride(0) % 8 and one.data_ptr() % 16 == 0
    kc, vc = fq.kv_cache(2, 2, D, page, F16, DEV)
    kc.zero_(), vc.zero_()
    fq.kv_cache_write(one[:, 2:4], one[:, 4:], i32([17]), kc, vc)
    k, v = gather(kc, vc, [17], page)
    assert torch.equal(k, one[:, 2:4]) and torch.equal(v, one[:, 4:])
    args = (kc, vc, i32([[1, 0]]), i32([1]), i32([0, 1]))
    got = fq.tree_attention(one[:, :2], *args)
    assert torch.equal(got, fq.tree_attention(one[:, :2].contiguous(), *args))
    # one head, four elements from the next of a tensor that has no other
    head = torch.randn(3, D, generator=g, device=DEV).half().as_strided((3, 1, D), (D, 4, 1))
    kc, vc = fq.kv_cache(2, 1, D, page, F16, DEV)
    kc.zero_(), vc.zero_()
    fq.kv_cache_write(head, head, i32([3, 18, 19]), kc, vc)
    k, v = gather(kc, vc, [3, 18, 19], page)
    assert torch.equal(k, head) and torch.equal(v, head)
    args = (kc, vc, i32([[0, 1]]), i32([17]), i32([0, 3]))
    assert torch.equal(fq.tree_attention(head, *args),
                       fq.tree_attention(head.reshape(3, D).view(3, 1, D), *args))


def test_pack_w4_of_the_most_rows(fq):
    """2^24 rows, as many as are accepted: the last ones, the first, and some between."""
    N, K, group = 1 << 24, 128, 128
    say("pack_w4", N, K)
    g = torch.Generator(device=DEV).manual_seed(2)
    w = torch.zeros(N, K, dtype=F16, device=DEV)
    rows = [0, 16, 5 << 20, (1 << 23) - 16, 1 << 23, N - 16]
    for r in rows:
        w[r:r + 16] = torch.randn(16, K, generator=g, device=DEV).half()
    w4, sw = fq.pack_w4(w, group)
    for r in rows:
        q, s = ref.quantize_w4(w[r:r + 16].float().cpu().numpy(), group)
        at = r * K // 8
        assert np.array_equal(w4[at:at + 2 * K].cpu().numpy().view(np.uint32), ref.pack_w4(q))
        assert np.array_equal(sw[:, r:r + 16].cpu().numpy().T, s)
    assert int((sw != 0).sum()) == 16 * len(rows)
    assert int((w4 == 0x08080808 * 17 - (1 << 32)).sum()) >= N * K // 8 - len(rows) * 2 * K


def test_block_tables_slots_past_32_bits(fq):
    """A slot that int32 does not hold is -1, not another request's."""
    page = 65536
    table = i32([[32767, 32768, 65536, 65537], [1, -1, -1, -1]])
    slots, cu, counts = fq.block_tables(i32([page - 2, 0]), i32([3 * page, 2]), i32([70000]), table,
                                        page, 3 * page + 2)
    want = torch.full((3 * page + 2,), -1, dtype=torch.int32, device=DEV)
    want[:2] = i32([32767 * page + page - 2, 32767 * page + page - 1])
    assert torch.equal(slots[:3 * page], want[:3 * page])
    assert table[0].tolist() == [32767, 70000, -1, -1] and counts.tolist() == [3 * page + 2, 4, 4]


@pytest.mark.parametrize("T,Hkv,D,page", [(2100, 16, 64, 16), (1089, 32, 96, 32),
                                          (4131, 8, 128, 64), (1025, 40, 256, 128),
                                          (700, 64, 128, 16)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_kv_cache_write_of_prompts(fq, T, Hkv, D, page, dtype):
    """The form of prompts, 64 tokens a workgroup (ceil(T / 64) Hkv of at least two a compute
    unit): runs that start inside a half block and so cross the workgroups' ends inside one,
    scattered slots, dropped tokens, slots outside the cache, requests that begin anywhere."""
    assert -(-T // 64) * Hkv >= 512
    say("kv_cache_write, prompts", T, Hkv, D, page, dtype)
    r = np.random.default_rng([T, Hkv, D])
    pages = -(-T // page) + 9
    g = torch.Generator(device=DEV).manual_seed(T)
    kv = torch.randn(T, 2 * Hkv + 1, D, generator=g, device=DEV).to(dtype)
    k, v = kv[:, 1:1 + Hkv], kv[:, 1 + Hkv:]
    run = np.arange(T) + int(r.integers(1, 8))
    requests = run.copy()                      # ragged requests on pages of their own
    order, at, t = r.permutation(pages), 0, 0
    while t < T:
        n = min(int(r.integers(1, 3 * page)), T - t, (pages - at) * page)
        if n <= 0:
            requests[t:] = -1
            break
        pos = np.arange(n)
        requests[t:t + n] = order[at + pos // page] * page + pos % page
        at, t = at + -(-n // page), t + n
    scattered = r.permutation(pages * page)[:T]
    for slots in (run, requests, scattered, np.where(r.random(T) < 0.3, -1, run),
                  np.where(np.arange(T) % 61 == 0, pages * page + 5, run)):
        kc, vc = fq.kv_cache(pages, Hkv, D, page, dtype, DEV)
        kc.fill_(3), vc.fill_(5)
        want_k, want_v = kc.clone(), vc.clone()
        kept = np.nonzero((slots >= 0) & (slots < pages * page))[0]
        s = torch.from_numpy(slots[kept]).to(DEV)
        src = torch.from_numpy(kept).to(DEV)
        want_k[s // page, :, s % page // 16, :, s % 16] = k[src].reshape(-1, Hkv, D // 32, 32)
        want_v[s // page, :, s % page // 16, :, s % 16] = v[src]
        fq.kv_cache_write(k, v, i32(slots), kc, vc)
        assert torch.equal(kc.view(torch.int16), want_k.view(torch.int16))
        assert torch.equal(vc.view(torch.int16), want_v.view(torch.int16))


# M, N, K, group: activations that fill the few-rows kernel's LDS with one tile an item and
# with two, and do not fit it; the longest K of the benchmark's layers
LONG = [(1, 48, 24320, 128), (4, 48, 5888, 64), (4, 32784, 5888, 32), (1, 32784, 24320, 128),
        (1, 64, 24448, 128), (1, 8192, 28672, 128), (2, 272, 28672, 64), (33, 528, 28672, 32)]


@pytest.mark.parametrize("M,N,K,group", LONG)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_gemv_w4_long_rows(fq, M, N, K, group, dtype):
    """Against the definition in 64 bits on the GPU, from random packed dwords."""
    say("gemv_w4, long", M, N, K, group, dtype)
    g = torch.Generator(device=DEV).manual_seed(N + K)
    w4 = torch.randint(-1 << 31, 1 << 31, (N * K // 8,), generator=g, device=DEV).to(torch.int32)
    s = (torch.rand(K // group, N, generator=g, device=DEV) * 0.01 + 1e-3).half()
    x = torch.randn(M, K, generator=g, device=DEV).to(dtype)
    y = fq.gemv_w4(x, w4, s, N).double()
    xd = x.double()
    for n0 in range(0, N, 1024):
        n1 = min(N, n0 + 1024)
        # [tile][k-block][k % 32 / 8][row][k % 128 / 32], codes 4 (c / 2) + 16 (c % 2)
        d = w4.view(N // 16, K // 128, 4, 16, 4)[n0 // 16:n1 // 16]
        q = torch.empty(n1 - n0, K, dtype=torch.float64, device=DEV)
        by_k = q.view(-1, 16, K // 128, 4, 4, 8)
        for c in range(8):
            by_k[..., c] = (((d >> (4 * (c // 2) + 16 * (c % 2))) & 15) - 8) \
                .permute(0, 3, 1, 4, 2).double()
        q *= s[:, n0:n1].t().double().repeat_interleave(group, 1)
        want, total = xd @ q.t(), xd.abs() @ q.t().abs()
        tol = (group + K // group + 16) * 2.0 ** -23 * total \
            + ref.OUT_EPS[dtype] * want.abs() * (1 + 2.0 ** -7) + ref.OUT_ABS[dtype]
        err = (y[:, n0:n1] - want).abs()
        assert bool((err <= tol).all()), (n0, float((err / tol).max()))


def attention_in_64_bits(q, k, v, scale):
    """out and lse of rows q [n][H][D] that attend all of k, v [L][Hkv][D]."""
    n, H, D = q.shape
    group = H // k.shape[1]
    out = torch.empty(n, H, D, dtype=torch.float64, device=DEV)
    lse = torch.empty(n, H, dtype=torch.float64, device=DEV)
    for h in range(H):
        s = scale * (q[:, h].double() @ k[:, h // group].double().t())
        out[:, h] = torch.softmax(s, 1) @ v[:, h // group].double()
        lse[:, h] = torch.logsumexp(s, 1)
    return out, lse


@pytest.mark.parametrize("ctx,H,Hkv,D,page,first", [(300_001, 8, 2, 64, 128, 0),
                                                    (1_000_000, 2, 1, 64, 256, 0),
                                                    (5000, 4, 2, 128, 64, 140_000),
                                                    (777, 40, 8, 96, 16, 180_000)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_tree_attention_long_contexts_and_large_caches(fq, ctx, H, Hkv, D, page, first, dtype):
    """Contexts of a million tokens, and pages that lie more than 2^32 bytes into the cache.
    Scores and values of order one: the error of a sum of L terms is that of fp32."""
    say("tree_attention, long", ctx, H, Hkv, D, page, first, dtype)
    need = -(-(ctx + 1) // page)
    pages = first + need
    assert first == 0 or first * Hkv * page * D * 2 > 1 << 32
    kc, vc = fq.kv_cache(pages, Hkv, D, page, dtype, DEV)
    g = torch.Generator(device=DEV).manual_seed(ctx)
    order = first + torch.randperm(need, generator=g, device=DEV)
    kc[first:].copy_(torch.randn(kc[first:].shape, generator=g, device=DEV))
    vc[first:].copy_(torch.randn(vc[first:].shape, generator=g, device=DEV) + 0.25)
    q = torch.randn(1, H, D, generator=g, device=DEV).to(dtype)
    out, lse = fq.tree_attention(q, kc, vc, order.to(torch.int32)[None], i32([ctx]), i32([0, 1]),
                                 max_new=1, return_lse=True)
    pos = torch.arange(ctx + 1, device=DEV)
    k, v = gather(kc, vc, order[pos // page] * page + pos % page, page)
    want, want_lse = attention_in_64_bits(q, k, v, 1 / math.sqrt(D))
    L = ctx + 1
    u = 2.0 ** -23
    # scores: |q k| scale is at most about 4 sqrt(D) here; the sums as in the definition
    d = (D + 8) * u * 4 * math.sqrt(D)
    tol = 2 * (2 * d + 2.0 ** -17 + (L / 32 + 64) * u) * (1.25 + want.abs()) \
        + ref.OUT_EPS[dtype] * want.abs() + ref.OUT_ABS[dtype]
    assert bool(((out.double() - want).abs() <= tol).all())
    assert bool(((lse.double() - want_lse).abs() <= 2 * d + (L / 32 + 64) * u + 1e-6).all())
    # and written through the same offsets
    new = torch.randn(3, 2 * Hkv, D, generator=g, device=DEV).to(dtype)
    slots = (order[-1] * page + torch.arange(3, device=DEV)).to(torch.int32)
    fq.kv_cache_write(new[:, :Hkv], new[:, Hkv:], slots, kc, vc)
    k, v = gather(kc, vc, slots, page)
    assert torch.equal(k, new[:, :Hkv]) and torch.equal(v, new[:, Hkv:])
