"""The decoding-step operators of include/flexq_serve.h without a GPU: every symbol is
exported and bound, and bad arguments are refused on the host before any HIP call."""
import os
import re
import subprocess

import numpy as np
import pytest

import serve_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "flexq_serve.h")
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


def test_every_declared_symbol_is_exported_and_bound(fq):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(flexq_[a-z0-9_]+)\s*\(", text))
    assert names == set(fq.SERVE_SIGNATURES)
    out = subprocess.check_output(["nm", "-D", "--defined-only", LIB]).decode()
    assert names <= {line.split()[-1] for line in out.splitlines() if " T " in line}


def test_pack_w4_rejects_bad_arguments(fq):
    assert fq.lib().flexq_packed_w4_bytes(4096, 4096) == 4096 * 4096 // 2
    assert fq.lib().flexq_packed_w4_bytes(16, 64) == 0
    assert fq.lib().flexq_packed_w4_bytes(0, 128) == 0

    def call(w=A, dtype=0, N=16, K=128, group=128, w4=2 * A, s=3 * A):
        return fq.lib().flexq_pack_w4(w, dtype, N, K, group, w4, s, None)

    for kw in (dict(w=None), dict(w4=None), dict(s=None), dict(N=-16), dict(K=0), dict(dtype=2),
               dict(w4=A + 16), dict(s=A + 64), dict(s=2 * A + 8)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(group=16), dict(group=256), dict(K=192), dict(N=24), dict(w=A + 8),
               dict(w4=2 * A + 4), dict(s=3 * A + 1), dict(N=(1 << 24) + 16)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(N=0, w=None, w4=None, s=None) == SUCCESS


def test_gemv_w4_rejects_bad_arguments(fq):
    need = fq.lib().flexq_gemv_w4_workspace_bytes
    assert need(1, 4096, 4096) == 0 and need(64, 57344, 8192) == 0
    assert need(13, 5120, 13824) % (13 * 5120 * 4) == 0 and need(13, 5120, 13824) > 0
    assert need(0, 16, 128) == 0 and need(5, 24, 128) == 0 and need(5, 16, 100) == 0

    def call(x=A, dtype=0, stride=128, w4=2 * A, s=3 * A, M=4, N=16, K=128, group=128, y=4 * A,
             ws=None, wb=0):
        return fq.lib().flexq_gemv_w4(x, dtype, stride, w4, s, M, N, K, group, ws, wb, y, None)

    big = dict(M=13, N=512, K=2048, stride=2048)    # K in slices: a workspace is needed
    wb = need(13, 512, 2048)
    assert wb > 0
    assert call(**big) == INVALID and call(**big, ws=5 * A, wb=wb - 1) == INVALID
    assert call(**big, ws=5 * A + 8, wb=wb) == UNSUPPORTED
    for over in (A, 2 * A + 64, 3 * A, 4 * A - 64):
        assert call(**big, ws=over, wb=wb) == INVALID, over
    for kw in (dict(x=None), dict(w4=None), dict(s=None), dict(y=None), dict(M=-1), dict(N=-16),
               dict(K=0), dict(dtype=-1), dict(stride=120), dict(y=A + 64), dict(y=2 * A + 64),
               dict(y=3 * A + 8), dict(stride=1 << 20, y=A + (3 << 20))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(group=48), dict(K=100), dict(N=8), dict(x=A + 8), dict(w4=2 * A + 8),
               dict(s=3 * A + 2), dict(y=4 * A + 4), dict(stride=132), dict(M=1 << 21),
               dict(stride=(1 << 24) + 8), dict(N=1 << 23, K=1 << 14, group=128)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(M=0, x=None, y=None) == SUCCESS
    assert call(N=0, w4=None, y=None) == SUCCESS


def test_block_tables_rejects_bad_arguments(fq):
    def call(ctx=A, new=2 * A, B=4, free=3 * A, nf=9, head=4 * A, page=16, table=5 * A, cols=8,
             most=64, slots=6 * A, cu=7 * A, counts=8 * A):
        return fq.lib().flexq_block_tables(ctx, new, B, free, nf, head, page, table, cols, most,
                                           slots, cu, counts, None)

    for kw in (dict(ctx=None), dict(new=None), dict(free=None), dict(table=None),
               dict(slots=None), dict(cu=None), dict(counts=None), dict(B=-1), dict(nf=-1),
               dict(cols=-1), dict(most=-1), dict(page=0), dict(page=-16), dict(table=A + 4),
               dict(slots=3 * A + 8), dict(cu=4 * A), dict(counts=2 * A), dict(cu=5 * A + 8),
               dict(counts=7 * A + 12), dict(slots=7 * A)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(page=24), dict(page=1 << 17), dict(B=4097), dict(nf=(1 << 30) + 1),
               dict(cols=(1 << 30) + 1), dict(most=(1 << 30) + 1), dict(ctx=A + 2),
               dict(table=5 * A + 1), dict(counts=8 * A + 2)):
        assert call(**kw) == UNSUPPORTED, kw


def test_kv_cache_write_rejects_bad_arguments(fq):
    def call(k=A, kt=256, kh=64, v=2 * A, vt=256, vh=64, slots=3 * A, T=4, Hkv=4, D=64, pages=3,
             page=16, kc=4 * A, vc=5 * A):
        return fq.lib().flexq_kv_cache_write(k, kt, kh, v, vt, vh, slots, T, Hkv, D, pages, page,
                                             kc, vc, None)

    for kw in (dict(k=None), dict(v=None), dict(slots=None), dict(kc=None), dict(vc=None),
               dict(T=-1), dict(Hkv=0), dict(D=0), dict(pages=-1), dict(page=0), dict(kt=-8),
               dict(vh=-64), dict(kc=A + 64), dict(vc=2 * A + 64), dict(kc=3 * A),
               dict(vc=4 * A + 64)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(D=80), dict(page=8), dict(page=48), dict(kt=260), dict(vh=4), dict(k=A + 8),
               dict(v=2 * A + 2), dict(slots=3 * A + 2), dict(kc=4 * A + 8), dict(T=1 << 27),
               dict(pages=1 << 30), dict(kt=1 << 41)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(T=0, k=None, v=None) == SUCCESS


def test_tree_attention_rejects_bad_arguments(fq):
    f = fq.lib().flexq_tree_attention_workspace_bytes
    assert f(4, 9, 8, 2, 128) >= 16
    for bad in ((0, 9, 8, 2, 128), (4, 0, 8, 2, 128), (4, 9, 8, 3, 128), (4, 9, 8, 2, 100),
                (4097, 9, 8, 2, 128), (4, 9, 8192, 2, 128), (-1, 9, 8, 2, 128)):
        assert f(*bad) == 0, bad

    def call(q=A, dtype=0, qt=512, qh=64, kc=2 * A, vc=3 * A, pages=7, page=16, table=4 * A,
             cols=6, ctx=5 * A, cu=6 * A, B=2, T=6, max_new=5, H=8, Hkv=2, D=64, mask=7 * A,
             words=1, scale=0.125, ws=8 * A, wb=None, out=9 * A, lse=10 * A):
        wb = f(2, 5, 8, 2, 64) if wb is None else wb
        return fq.lib().flexq_tree_attention(q, dtype, qt, qh, kc, vc, pages, page, table, cols,
                                             ctx, cu, B, T, max_new, H, Hkv, D, mask, words,
                                             scale, ws, wb, out, lse, None)

    for kw in (dict(q=None), dict(kc=None), dict(vc=None), dict(table=None), dict(ctx=None),
               dict(cu=None), dict(ws=None), dict(out=None), dict(B=-1), dict(T=-1),
               dict(max_new=-1), dict(H=7), dict(Hkv=0), dict(D=0), dict(pages=0), dict(cols=-1),
               dict(words=-1), dict(dtype=3), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(max_new=33), dict(wb=8), dict(qt=-8), dict(out=A + 64), dict(out=2 * A),
               dict(lse=5 * A), dict(ws=3 * A), dict(ws=9 * A), dict(lse=8 * A), dict(out=7 * A),
               dict(lse=9 * A + 16)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(D=72), dict(page=24), dict(qt=516), dict(qh=4), dict(H=8192),
               dict(B=4097), dict(T=(1 << 24) + 1), dict(max_new=65537, mask=None),
               dict(cols=1 << 23), dict(pages=1 << 31), dict(q=A + 2), dict(out=9 * A + 8),
               dict(ws=8 * A + 4), dict(lse=10 * A + 2), dict(kc=2 * A + 8), dict(mask=7 * A + 2)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(B=0, q=None) == SUCCESS
    assert call(T=0, q=None) == SUCCESS
    assert call(max_new=0, out=None) == SUCCESS


def test_binding_checks_arguments(fq):
    """Types, shapes, strides and devices are checked before the C ABI sees a pointer."""
    import torch
    f16, bf16, i32, f32 = torch.float16, torch.bfloat16, torch.int32, torch.float32

    def z(*shape, dtype=f16):
        return torch.zeros(shape, dtype=dtype)

    def refuse(err, match, fn, *a, **kw):
        with pytest.raises(err, match=match):
            fn(*a, **kw)

    refuse(TypeError, "float16 or bfloat16", fq.pack_w4, z(16, 128, dtype=f32))
    refuse(ValueError, "2-D", fq.pack_w4, z(128))
    refuse(ValueError, "multiple of 128", fq.pack_w4, z(16, 96))
    refuse(ValueError, "multiple of 16", fq.pack_w4, z(8, 128))
    refuse(ValueError, "group", fq.pack_w4, z(16, 128), 16)
    refuse(ValueError, "w4 holds", fq.pack_w4, z(16, 128), w4=z(4, dtype=i32))
    refuse(TypeError, "CUDA", fq.pack_w4, z(16, 128))
    w4, sw = z(16 * 256 // 8, dtype=i32), z(2, 16)
    refuse(TypeError, "float16 or bfloat16", fq.gemv_w4, z(2, 256, dtype=f32), w4, sw, 16)
    refuse(ValueError, "rows for K", fq.gemv_w4, z(2, 256), w4, z(3, 16), 16)
    refuse(ValueError, "group", fq.gemv_w4, z(2, 256), w4, z(1, 16), 16)
    refuse(ValueError, "s_w must have shape", fq.gemv_w4, z(2, 256), w4, z(2, 32), 16)
    refuse(ValueError, "w4 holds", fq.gemv_w4, z(2, 256), w4[:9], sw, 16)
    refuse(ValueError, "contiguous", fq.gemv_w4, z(256, 2).t(), w4, sw, 16)
    refuse(TypeError, "y must be", fq.gemv_w4, z(2, 256), w4, sw, 16, y=z(2, 16, dtype=bf16))
    refuse(TypeError, "CUDA", fq.gemv_w4, z(2, 256), w4, sw, 16)
    n = z(3, dtype=i32)
    table = z(3, 4, dtype=i32)
    refuse(ValueError, "ctx_lens must have shape", fq.block_tables, n[:2], n, n, table, 16, 8)
    refuse(TypeError, "new_lens must be", fq.block_tables, n, n.long(), n, table, 16, 8)
    refuse(ValueError, "2-D", fq.block_tables, n, n, n, n, 16, 8)
    refuse(ValueError, "max_tokens", fq.block_tables, n, n, n, table, 16, -1)
    refuse(ValueError, "slot_map must have shape", fq.block_tables, n, n, n, table, 16, 8,
           slot_map=n)
    refuse(ValueError, "free_head must have shape", fq.block_tables, n, n, n, table, 16, 8,
           free_head=n)
    refuse(TypeError, "CUDA", fq.block_tables, n, n, n, table, 16, 8)
    refuse(ValueError, "page_size", fq.kv_cache, 4, 2, 64, 24, device="cpu")
    kc, vc = fq.kv_cache(4, 2, 64, 32, device="cpu")
    k = z(3, 2, 64)
    refuse(ValueError, "k must have shape", fq.kv_cache_write, z(3, 4, 64), z(3, 4, 64), n, kc, vc)
    refuse(ValueError, "v must have shape", fq.kv_cache_write, k, z(2, 2, 64), n, kc, vc)
    refuse(TypeError, "v_cache must be", fq.kv_cache_write, k.bfloat16(), k.bfloat16(), n, kc, vc)
    refuse(ValueError, "k_cache must have shape", fq.kv_cache_write, k, k, n, kc[:3], vc)
    refuse(ValueError, "slot_map must have shape", fq.kv_cache_write, k, k, n[:2], kc, vc)
    refuse(ValueError, "last dimension", fq.kv_cache_write, z(3, 2, 128)[:, :, ::2], k, n, kc, vc)
    refuse(TypeError, "CUDA", fq.kv_cache_write, k, k, n, kc, vc)
    q, cu = z(3, 4, 64), z(4, dtype=i32)
    args = (q, kc, vc, table, n, cu)
    refuse(ValueError, "does not fit", fq.tree_attention, z(3, 3, 64), *args[1:])
    refuse(ValueError, "does not fit", fq.tree_attention, z(3, 4, 128), *args[1:])
    refuse(TypeError, "v_cache must be", fq.tree_attention, q.bfloat16(), *args[1:])
    refuse(ValueError, "cu_new must have shape", fq.tree_attention, *args[:5], n)
    refuse(ValueError, "bits a token", fq.tree_attention, *args, max_new=40,
           tree_mask=z(3, 1, dtype=i32))
    refuse(ValueError, "tree_mask must have shape", fq.tree_attention, *args,
           tree_mask=z(2, 1, dtype=i32))
    refuse(ValueError, "out must have shape", fq.tree_attention, *args, out=z(3, 4, 32))
    refuse(TypeError, "lse must be", fq.tree_attention, *args, lse=z(3, 4))
    refuse(ValueError, "workspace holds", fq.tree_attention, *args,
           workspace=z(8, dtype=torch.uint8))
    refuse(TypeError, "CUDA", fq.tree_attention, *args)


# ---- the reference the GPU results are held to ----------------------------------------


def test_reference_packing_places_every_code():
    """Each code owns four bits of its own, at the place the header's formula gives."""
    N, K = 32, 256
    seen = set()
    for n, k in [(0, 0), (15, 127), (16, 128), (31, 255), (3, 37), (20, 200)]:
        q = np.full((N, K), -8)
        q[n, k] = 7
        at = np.nonzero(ref.pack_w4(q))[0]
        assert len(at) == 1
        seen.add((int(at[0]), int(ref.pack_w4(q)[at[0]])))
        c = k % 8
        assert int(ref.pack_w4(q)[at[0]]) == 15 << (4 * (c // 2) + 16 * (c % 2))
    assert len(seen) == 6
    # row 3, column 37: tile 0, k-block 0, j = 1, lane 16 * 0 + 3, code 5
    q = np.full((N, K), -8)
    q[3, 37] = 1
    assert ref.pack_w4(q)[3 * 4 + 1] == 9 << 24


def test_reference_cache_indexes_are_a_bijection():
    for D, page in ((64, 16), (96, 64)):
        Hkv, slots = 3, 4 * page
        s, h, d = np.meshgrid(np.arange(slots), np.arange(Hkv), np.arange(D), indexing="ij")
        for flat in ref.cache_index(s, h, d, Hkv, D, page):
            assert np.array_equal(np.sort(flat.ravel()), np.arange(slots * Hkv * D))
    ik, iv = ref.cache_index(37, 1, 70, 2, 96, 32)
    # page 1, head 1, block 0, row 5: block (1 * 2 + 1) * 2 = 6
    assert ik == 6 * 1536 + 2 * 512 + 5 * 32 + 6 and iv == 6 * 1536 + 70 * 16 + 5


def test_reference_attention_against_a_direct_sum():
    import torch
    g = torch.Generator().manual_seed(3)
    q = torch.randn(2, 2, 8, generator=g, dtype=torch.float64)
    k = torch.randn(5, 1, 8, generator=g, dtype=torch.float64)
    v = torch.randn(5, 1, 8, generator=g, dtype=torch.float64)
    mask = torch.tensor([[True, False], [False, False]])
    out, lse, _, _ = ref.attention(q, k, v, 3, 2, mask, 0.5)
    for t, keys in ((0, [0, 1, 2, 3]), (1, [0, 1, 2])):
        for h in range(2):
            w = np.exp([0.5 * float(q[t, h] @ k[j, 0]) for j in keys])
            want = sum(x * v[j, 0] for x, j in zip(w, keys)) / w.sum()
            assert torch.allclose(out[t, h], want, atol=1e-12)
            assert abs(float(lse[t, h]) - np.log(w.sum())) < 1e-12
    out, lse, _, _ = ref.attention(q, k[3:], v[3:], 0, 2, mask & False, 0.5)
    assert bool((out == 0).all()) and bool((lse == -np.inf).all())


def test_reference_block_tables_by_hand():
    table = np.full((2, 3), -1)
    table[0, 0] = 7
    t, slots, cu, counts = ref.block_tables([3, 0], [3, 5], [20, 21, 22, 23], table, 4, 10, 1)
    assert t.tolist() == [[7, 21, -1], [22, 23, -1]]
    assert slots.tolist() == [31, 84, 85, 88, 89, 90, 91, 92, -1, -1]
    assert cu.tolist() == [0, 3, 8] and counts.tolist() == [8, 3, 4]
