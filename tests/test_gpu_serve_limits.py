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
