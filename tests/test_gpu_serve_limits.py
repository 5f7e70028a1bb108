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
