"""Defaults of the decoding-step calls, without a GPU: what is left out is not refused."""
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "w6a6_w6a8_integer_amd", "libflexq.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libflexq.so not built")


def test_max_new_is_at_most_the_bits_of_the_mask():
    """Forty tokens of several requests and one word of mask for each: no request has more
    than 32, and the call goes on to the next check (the tensors are on the CPU)."""
    import torch
    import w6a6_w6a8_integer_amd as fq
    kc, vc = fq.kv_cache(4, 2, 64, 32, device="cpu")

    def i32(*shape):
        return torch.zeros(shape, dtype=torch.int32)

    args = (torch.zeros(40, 4, 64, dtype=torch.float16), kc, vc, i32(3, 4), i32(3), i32(4))
    with pytest.raises(TypeError, match="CUDA"):
        fq.tree_attention(*args, tree_mask=i32(40, 1))
    with pytest.raises(ValueError, match="bits a token"):
        fq.tree_attention(*args, tree_mask=i32(40, 1), max_new=33)
