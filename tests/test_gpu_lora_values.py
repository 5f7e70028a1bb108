"""flexq_lora_add where a step has no adapter loaded, and where weights or sums are infinite or large."""
import math

import numpy as np
import pytest

import kv4_reference as ref
import test_gpu_lora as base

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DEV = "cuda:0"
F16, BF16 = torch.float16, torch.bfloat16
