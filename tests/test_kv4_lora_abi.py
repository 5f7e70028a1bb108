"""The 4-bit cache's operators and the low-rank adapters without a GPU: bad arguments are refused
on the host before any HIP call, and the references that the GPU results are held to."""
import os

import numpy as np
import pytest

import kv4_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "w6a6_w6a8_integer_amd", "libflexq.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libflexq.so not built")

SUCCESS, INVALID, UNSUPPORTED = 0, 1, 2
A = 1 << 32   # fake addresses 4 GiB apart: never dereferenced on error paths


@pytest.fixture(scope="module")
def fq():
    import torch  # noqa: F401  (the HIP runtime must be the one torch loads)
    import w6a6_w6a8_integer_amd as fq
    fq.lib()
    return fq


def test_kv4_cache_write_rejects_bad_arguments(fq):
    def call(k=A, kt=256, kh=64, v=2 * A, vt=256, vh=64, dtype=0, slots=3 * A, T=4, Hkv=4, D=64,
             pages=3, page=16, kc=4 * A, vc=5 * A, sc=6 * A):
        return fq.lib().flexq_kv4_cache_write(k, kt, kh, v, vt, vh, dtype, slots, T, Hkv, D, pages,
                                              page, kc, vc, sc, None)

    for kw in (dict(k=None), dict(v=None), dict(slots=None), dict(kc=None), dict(vc=None),
               dict(sc=None), dict(T=-1), dict(Hkv=0), dict(D=0), dict(pages=-1), dict(page=0),
               dict(kt=-8), dict(vh=-64), dict(dtype=2), dict(kc=A + 64), dict(vc=2 * A + 64),
               dict(kc=3 * A), dict(vc=4 * A + 64), dict(sc=5 * A + 16), dict(sc=3 * A),
               dict(sc=A + 128)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(D=80), dict(page=8), dict(page=48), dict(kt=260), dict(vh=4), dict(k=A + 8),
               dict(v=2 * A + 2), dict(slots=3 * A + 2), dict(kc=4 * A + 8), dict(sc=6 * A + 2),
               dict(T=1 << 27), dict(pages=1 << 30), dict(kt=1 << 41)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(T=0, k=None, v=None) == SUCCESS


def test_kv4_cache_read_rejects_bad_arguments(fq):
    def call(kc=A, vc=2 * A, sc=3 * A, slots=4 * A, T=4, Hkv=4, D=64, pages=3, page=16, dtype=1,
             k=5 * A, v=6 * A):
        return fq.lib().flexq_kv4_cache_read(kc, vc, sc, slots, T, Hkv, D, pages, page, dtype, k, v,
                                             None)

    for kw in (dict(kc=None), dict(vc=None), dict(sc=None), dict(slots=None), dict(k=None),
               dict(v=None), dict(T=-1), dict(Hkv=-1), dict(pages=-1), dict(dtype=-1),
               dict(k=A + 16), dict(v=3 * A), dict(v=5 * A + 64), dict(k=4 * A)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(D=72), dict(page=512), dict(kc=A + 4), dict(sc=3 * A + 2), dict(k=5 * A + 8),
               dict(slots=4 * A + 1), dict(T=1 << 27), dict(Hkv=1 << 17, T=1)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(T=0, k=None, v=None) == SUCCESS


def test_kv4_attention_rejects_bad_arguments(fq):
    f = fq.lib().flexq_kv4_attention_workspace_bytes
    assert f(4, 9, 8, 2, 128) >= 16
    for bad in ((0, 9, 8, 2, 128), (4, 0, 8, 2, 128), (4, 9, 8, 3, 128), (4, 9, 8, 2, 100),
                (4097, 9, 8, 2, 128), (4, 9, 8192, 2, 128), (-1, 9, 8, 2, 128)):
        assert f(*bad) == 0, bad

    def call(q=A, dtype=0, qt=512, qh=64, kc=2 * A, vc=3 * A, sc=11 * A, pages=7, page=16,
             table=4 * A, cols=6, ctx=5 * A, cu=6 * A, B=2, T=6, max_new=5, H=8, Hkv=2, D=64,
             mask=7 * A, words=1, window=0, sinks=0, scale=0.125, ws=8 * A, wb=None, out=9 * A,
             lse=10 * A):
        wb = f(2, 5, 8, 2, 64) if wb is None else wb
        return fq.lib().flexq_kv4_attention(q, dtype, qt, qh, kc, vc, sc, pages, page, table, cols,
                                            ctx, cu, B, T, max_new, H, Hkv, D, mask, words, window,
                                            sinks, scale, ws, wb, out, lse, None)

    for kw in (dict(q=None), dict(kc=None), dict(vc=None), dict(sc=None), dict(table=None),
               dict(ctx=None), dict(cu=None), dict(ws=None), dict(out=None), dict(B=-1),
               dict(T=-1), dict(max_new=-1), dict(H=7), dict(Hkv=0), dict(D=0), dict(pages=0),
               dict(cols=-1), dict(words=-1), dict(dtype=3), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(max_new=33), dict(wb=8), dict(qt=-8),
               dict(out=A + 64), dict(out=2 * A), dict(lse=5 * A), dict(ws=3 * A), dict(ws=9 * A),
               dict(lse=8 * A), dict(out=7 * A), dict(lse=9 * A + 16), dict(out=11 * A + 64),
               dict(window=-1), dict(sinks=-1)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(D=72), dict(page=24), dict(qt=516), dict(qh=4), dict(H=8192),
               dict(B=4097), dict(T=(1 << 24) + 1), dict(max_new=65537, mask=None),
               dict(cols=1 << 23), dict(pages=1 << 31), dict(q=A + 2), dict(out=9 * A + 8),
               dict(ws=8 * A + 4), dict(lse=10 * A + 2), dict(kc=2 * A + 8), dict(sc=11 * A + 8),
               dict(mask=7 * A + 2)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(B=0, q=None) == SUCCESS
    assert call(T=0, q=None) == SUCCESS
    assert call(max_new=0, out=None) == SUCCESS


def test_lora_add_rejects_bad_arguments(fq):
    f = fq.lib().flexq_lora_add_workspace_bytes
    assert f(64, 256, 1024, 16, 4) >= 64 * 16 * 4
    for bad in ((0, 256, 1024, 16, 4), (64, 0, 1024, 16, 4), (64, 24, 1024, 16, 4),
                (64, 256, 100, 16, 4), (64, 256, 1024, 12, 4), (64, 256, 1024, 264, 4),
                (64, 256, 1024, 16, 0), (64, 256, 1024, 16, -1)):
        assert f(*bad) == 0, bad

    def call(x=A, dtype=0, xs=1024, y=2 * A, ys=256, ids=3 * A, a=4 * A, b=5 * A, ranks=6 * A,
             scales=7 * A, T=64, N=256, K=1024, R=16, L=4, ws=8 * A, wb=None, out=9 * A, os=256):
        wb = f(64, 256, 1024, 16, 4) if wb is None else wb
        return fq.lib().flexq_lora_add(x, dtype, xs, y, ys, ids, a, b, ranks, scales, T, N, K, R, L,
                                       ws, wb, out, os, None)

    for kw in (dict(x=None), dict(y=None), dict(ids=None), dict(a=None), dict(b=None),
               dict(out=None), dict(ws=None), dict(wb=16), dict(T=-1), dict(N=-16), dict(K=0),
               dict(R=0), dict(L=-1), dict(dtype=2), dict(xs=1016), dict(ys=248), dict(os=128),
               dict(out=A + 64), dict(out=3 * A), dict(out=4 * A), dict(out=5 * A + 32),
               dict(out=6 * A), dict(out=7 * A), dict(out=8 * A), dict(ws=A), dict(ws=2 * A),
               dict(ws=4 * A), dict(out=2 * A + 16), dict(out=2 * A, os=264)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(N=24), dict(K=96), dict(R=12), dict(R=264), dict(L=(1 << 20) + 1),
               dict(T=4194241), dict(xs=1028), dict(ys=260), dict(os=1 << 41), dict(x=A + 8),
               dict(y=2 * A + 8), dict(a=4 * A + 2), dict(b=5 * A + 8), dict(ids=3 * A + 2),
               dict(ranks=6 * A + 1), dict(scales=7 * A + 2), dict(ws=8 * A + 8),
               dict(out=9 * A + 4)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(T=0, x=None, out=None) == SUCCESS
    assert call(N=0, y=None, out=None) == SUCCESS


def test_binding_checks_arguments(fq):
    """Types, shapes, strides and devices are checked before the C ABI sees a pointer."""
    import torch
    f16, bf16, i32, f32 = torch.float16, torch.bfloat16, torch.int32, torch.float32

    def z(*shape, dtype=f16):
        return torch.zeros(shape, dtype=dtype)

    def refuse(err, match, fn, *a, **kw):
        with pytest.raises(err, match=match):
            fn(*a, **kw)

    refuse(ValueError, "page_size", fq.kv4_cache, 4, 2, 64, 24, device="cpu")
    refuse(ValueError, "D one of", fq.kv4_cache, 4, 2, 80, 16, device="cpu")
    kc, vc, sc = cache = fq.kv4_cache(4, 2, 64, 32, device="cpu")
    n, k = z(3, dtype=i32), z(3, 2, 64)
    refuse(TypeError, "float16 or bfloat16", fq.kv4_cache_write, k.float(), k, n, *cache)
    refuse(ValueError, "k must have shape", fq.kv4_cache_write, z(3, 4, 64), z(3, 4, 64), n, *cache)
    refuse(ValueError, "v must have shape", fq.kv4_cache_write, k, z(2, 2, 64), n, *cache)
    refuse(TypeError, "v must be", fq.kv4_cache_write, k, k.bfloat16(), n, *cache)
    refuse(ValueError, "v_codes must have shape", fq.kv4_cache_write, k, k, n, kc, vc[:3], sc)
    refuse(ValueError, "scales must have shape", fq.kv4_cache_write, k, k, n, kc, vc, sc[:, :1])
    refuse(TypeError, "scales must be", fq.kv4_cache_write, k, k, n, kc, vc, sc.float())
    refuse(TypeError, "k_codes must be", fq.kv4_cache_write, k, k, n, kc.long(), vc, sc)
    refuse(ValueError, "k_codes must be", fq.kv4_cache_write, k, k, n, kc[..., :5], vc, sc)
    refuse(ValueError, "5-D", fq.kv4_cache_write, k, k, n, kc[0], vc, sc)
    refuse(ValueError, "slot_map must have shape", fq.kv4_cache_write, k, k, n[:2], *cache)
    refuse(ValueError, "last dimension", fq.kv4_cache_write, z(3, 2, 128)[:, :, ::2], k, n, *cache)
    refuse(TypeError, "CUDA", fq.kv4_cache_write, k, k, n, *cache)
    refuse(TypeError, "slot_map must be", fq.kv4_cache_read, n.long(), *cache)
    refuse(ValueError, "1-D", fq.kv4_cache_read, z(3, 1, dtype=i32), *cache)
    refuse(ValueError, "float16 or torch.bfloat16", fq.kv4_cache_read, n, *cache, dtype=f32)
    refuse(ValueError, "float16 or torch.bfloat16", fq.kv4_cache_read, n, *cache, dtype=7)
    refuse(TypeError, "k must be", fq.kv4_cache_read, n, *cache, k=k.bfloat16())
    refuse(ValueError, "v must have shape", fq.kv4_cache_read, n, *cache, v=k[:2])
    refuse(TypeError, "CUDA", fq.kv4_cache_read, n, *cache)
    q, cu, table = z(3, 4, 64), z(4, dtype=i32), z(3, 4, dtype=i32)
    args = (q, *cache, table, n, cu)
    refuse(ValueError, "does not fit", fq.kv4_attention, z(3, 3, 64), *args[1:])
    refuse(ValueError, "does not fit", fq.kv4_attention, z(3, 4, 128), *args[1:])
    refuse(TypeError, "float16 or bfloat16", fq.kv4_attention, q.float(), *args[1:])
    refuse(ValueError, "cu_new must have shape", fq.kv4_attention, *args[:6], n)
    refuse(ValueError, "bits a token", fq.kv4_attention, *args, max_new=40,
           tree_mask=z(3, 1, dtype=i32))
    refuse(ValueError, "tree_mask must have shape", fq.kv4_attention, *args,
           tree_mask=z(2, 1, dtype=i32))
    for window in (0, -3):
        refuse(ValueError, "window", fq.kv4_attention, *args, window=window)
    refuse(TypeError, "window", fq.kv4_attention, *args, window=1.5)
    refuse(ValueError, "sinks", fq.kv4_attention, *args, window=4, sinks=-1)
    refuse(TypeError, "sinks", fq.kv4_attention, *args, sinks=None)
    refuse(ValueError, "out must have shape", fq.kv4_attention, *args, out=z(3, 4, 32))
    refuse(TypeError, "lse must be", fq.kv4_attention, *args, lse=z(3, 4))
    refuse(ValueError, "workspace holds", fq.kv4_attention, *args,
           workspace=z(8, dtype=torch.uint8))
    refuse(TypeError, "CUDA", fq.kv4_attention, *args, window=4, sinks=2)
    x, y, a, b = z(3, 256), z(3, 48), z(2, 8, 256), z(2, 48, 8)
    args = (x, y, n, a, b)
    refuse(TypeError, "float16 or bfloat16", fq.lora_add, x.float(), *args[1:])
    refuse(TypeError, "y must be", fq.lora_add, x, y.bfloat16(), *args[2:])
    refuse(ValueError, "rows", fq.lora_add, x, z(2, 48), *args[2:])
    refuse(ValueError, "multiple of 128", fq.lora_add, z(3, 200), y, n, z(2, 8, 200), b)
    refuse(ValueError, "multiple of 16", fq.lora_add, x, z(3, 40), n, a, z(2, 40, 8))
    refuse(ValueError, "rank", fq.lora_add, x, y, n, z(2, 12, 256), z(2, 48, 12))
    refuse(ValueError, "rank", fq.lora_add, x, y, n, z(2, 264, 256), z(2, 48, 264))
    refuse(ValueError, "a must have shape", fq.lora_add, x, y, n, z(2, 8, 128), b)
    refuse(ValueError, "b must have shape", fq.lora_add, x, y, n, a, z(2, 8, 48))
    refuse(TypeError, "b must be", fq.lora_add, x, y, n, a, b.bfloat16())
    refuse(ValueError, "adapters must have shape", fq.lora_add, x, y, n[:2], a, b)
    refuse(TypeError, "adapters must be", fq.lora_add, x, y, n.long(), a, b)
    refuse(TypeError, "CUDA", fq.lora_add, *args)


def test_workspaces_fit_what_a_call_is_laid_out_for(fq):
    """Bytes are a whole number of fp32 sums, and grow with the tokens."""
    f = fq.lora_add_workspace_bytes
    for R in (8, 16, 24, 64, 200, 256):
        padded = next(p for p in (16, 32, 64, 128, 256) if p >= R)
        for T in (1, 7, 64, 65, 4000):
            assert f(T, 4096, 4096, R, 8) % (T * padded * 4) == 0
    assert fq.kv4_attention_workspace_bytes(1, 1, 4, 4, 64) >= 16


# ---- the references -------------------------------------------------------------------


def test_reference_codes_own_their_bits():
    """Every code of a cache has four bits to itself, and the scales a place each."""
    for D, page in ((64, 16), (96, 64), (128, 32)):
        Hkv, slots = 3, 4 * page
        s, h, d = np.meshgrid(np.arange(slots), np.arange(Hkv), np.arange(D), indexing="ij")
        key, value, scale = ref.places(s, h, d, Hkv, D, page)
        for word, bit in (key, value):
            assert np.array_equal(np.sort((8 * word + bit // 4).ravel()),
                                  np.arange(slots * Hkv * D))
        at = np.stack([scale[..., 0] + 16 * i for i in range(4)])
        assert np.array_equal(np.sort(at.ravel()), np.arange(slots * Hkv * 4))
    # page 1, head 1, row 5 of block 0: block (1 * 2 + 1) * 2 = 6
    key, value, scale = ref.places(37, 1, 70, 2, 96, 32)
    assert key == (6 * 192 + 5 * 12 + 8, 4 * 3) and value == (6 * 192 + 70 + 1, 8 * 2)
    assert scale == 6 * 64 + 5
    # byte 1 of a dword is the third token's, odd d above even d
    assert ref.places(2, 0, 3, 1, 64, 16)[1] == (2, 12)


def test_reference_write_and_read():
    r = np.random.default_rng(2)
    Hkv, D, page = 2, 64, 16
    k, v = (r.standard_normal((5, Hkv, D)).astype(np.float32) for _ in range(2))
    k[1, 0] = 0.25                       # constant: no scale, the offset alone
    k[2, 1, 7] = np.nan
    v[3, 0, 0], v[3, 0, 1] = -8, 7       # a whole step of 1: codes 0 and 15
    v[3, 0, 2:] = r.integers(-8, 8, D - 2)
    kc, vc = (r.integers(0, 1 << 32, 3 * Hkv * 2 * D, dtype=np.uint32) for _ in range(2))
    sc = np.zeros(3 * Hkv * 64, np.float16)
    before = kc.copy()
    slots = [17, 3, -1, 46, 48]
    ref.write(kc, vc, sc, k, v, slots, page)
    assert (kc != before).sum() <= 3 * Hkv * D // 8
    (c, s, b), (vcode, vs, vb) = ref.read(kc, vc, sc, [17, 3, 46], Hkv, D, page)
    assert np.array_equal(c[1, 0], np.zeros(D)) and s[1, 0] == 0 and b[1, 0] == 0.25
    want = [0, 1, 3]
    x = c * s[..., None] + b[..., None]
    assert (np.abs(x - k[want]) <= s[..., None] * 0.5 * 1.02).all()
    assert np.array_equal((vcode * vs[..., None] + vb[..., None])[2, 0], v[3, 0])
    c, s, b = ref.quantize(np.stack((k[2, 1], np.full(D, np.inf, np.float32),
                                     np.linspace(0, 1e5, D, dtype=np.float32),
                                     np.linspace(-1e5, 0, D, dtype=np.float32))))
    assert np.isnan(s[:2]).all() and np.isnan(b[:2]).all() and not np.isnan(s[2])
    assert np.isnan(s[3]) and (c[[0, 1, 3]] == 0).all()


def test_reference_windows():
    seen = ref.attended(10, 3, None, 4, 2)
    assert [np.nonzero(s)[0].tolist() for s in seen] == [[0, 1, 7, 8, 9, 10], [0, 1, 8, 9, 10, 11],
                                                        [0, 1, 9, 10, 11, 12]]
    tree = np.array([[1, 0, 0], [1, 1, 0], [1, 0, 1]], bool)
    seen = ref.attended(10, 3, tree, 2, 0)
    assert [np.nonzero(s)[0].tolist() for s in seen] == [[9, 10], [10, 11], [10, 12]]
    # a window shorter than a path: a tree's bits hold all the same
    seen = ref.attended(10, 3, tree, 1, 1)
    assert [np.nonzero(s)[0].tolist() for s in seen] == [[0, 10], [0, 10, 11], [0, 10, 12]]
    assert ref.attended(4, 2, None, 0, 3).sum() == 5 + 6
    assert np.nonzero(ref.attended(0, 5, None, 2, 1)[4])[0].tolist() == [0, 3, 4]


def test_reference_attention_against_a_direct_sum():
    r = np.random.default_rng(3)
    D, L = 8, 6
    key, value = (tuple([r.integers(0, 16, (L, 1, D)).astype(float), r.random((L, 1)),
                         r.standard_normal((L, 1))]) for _ in range(2))
    q = r.standard_normal((1, 2, D))
    seen = np.array([[True, False, True, True, False, True]])
    out, lse, tol, _ = ref.attention(q, key, value, seen, 0.5)
    for h in range(2):
        w, total = np.zeros(D), 0.0
        for j in np.nonzero(seen[0])[0]:
            e = np.exp(0.5 * float(q[0, h] @ (key[0][j, 0] * key[1][j, 0] + key[2][j, 0])))
            w += e * (value[0][j, 0] * value[1][j, 0] + value[2][j, 0])
            total += e
        assert np.allclose(out[0, h], w / total, atol=1e-12)
        assert abs(lse[0, h] - np.log(total)) < 1e-12
    assert (tol > 0).all()
    out, lse, _, _ = ref.attention(q, key, value, seen & False, 0.5)
    assert (out == 0).all() and (lse == -np.inf).all()


def test_reference_lora_by_hand():
    import torch
    x, y = np.array([[1.0, 2.0], [3.0, 4.0]]), np.array([[10.0], [20.0]])
    a = np.array([[[1.0, 0.0], [0.0, 1.0]], [[1.0, 1.0], [np.nan, np.nan]]])
    b = np.array([[[2.0, 3.0]], [[5.0, np.nan]]])
    out, _ = ref.lora(x, y, [0, 1], a, b, [2, 1], [1.0, 0.5], torch.float16)
    assert out.tolist() == [[10 + 2 * 1 + 3 * 2], [20 + 0.5 * 5 * 7]]
    out, _ = ref.lora(x, y, [-1, 2], a, b, None, None, torch.float16)
    assert out.tolist() == y.tolist()
