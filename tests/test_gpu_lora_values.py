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
