"""What flexq_lora_add launches, seen on the host: a library that stands before the HIP runtime
counts the launches, and nothing runs on a GPU."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "w6a6_w6a8_integer_amd", "libflexq.so")

pytestmark = [pytest.mark.skipif(not os.path.exists(LIB), reason="libflexq.so not built"),
              pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")]

COUNTER = """
#include <stddef.h>
struct Grid { unsigned x, y, z; };
static int launches;
extern "C" int hipLaunchKernel(const void*, Grid, Grid, void**, size_t, void*) { return ++launches, 0; }
extern "C" int taken() { const int n = launches; launches = 0; return n; }
"""

CALLS = """
import ctypes, sys
counter = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
import torch
import w6a6_w6a8_integer_amd as fq
A = 1 << 32   # addresses 4 GiB apart that nothing reads
def launches(T, K, R, L, apart, N=272):
    ws = fq.lora_add_workspace_bytes(T, N, K, R, L)
    loaded = (4 * A, 5 * A) if L else (None, None)
    status = fq.lib().flexq_lora_add(A, 0, K, 2 * A, N, 3 * A, *loaded, None, None, T, N, K, R, L,
                                     6 * A if ws else None, ws, 7 * A if apart else 2 * A, N, None)
    assert status == 0, status
    return counter.taken()
for T, K, R in ((1, 128, 8), (64, 512, 16), (65, 4096, 128), (449, 256, 16), (600, 512, 16),
                (600, 512, 256), (4096, 4096, 64), (16384, 256, 128), (70000, 256, 200)):
    print(T, K, R, launches(T, K, R, 0, False), launches(T, K, R, 0, True),
          launches(T, K, R, 3, False), launches(T, K, R, 3, True), flush=True)
"""


def test_no_adapter_is_loaded(tmp_path):
    """Without adapters there is no workspace, and only what copies y to an output apart from it is
    launched; with some, two products and from eight tiles of tokens on the slices' sums."""
    so = str(tmp_path / "counter.so")
    (tmp_path / "counter.cpp").write_text(COUNTER)
    subprocess.run(["g++", "-shared", "-fPIC", "-o", so, str(tmp_path / "counter.cpp")], check=True)
    out = subprocess.run([sys.executable, "-c", CALLS, so], cwd=ROOT, check=True, text=True,
                         stdout=subprocess.PIPE, timeout=300).stdout
    rows = [[int(x) for x in line.split()] for line in out.splitlines()]
    assert len(rows) == 9
    for T, K, R, in_place, apart, *loaded in rows:
        assert (in_place, apart) == (0, 1), (T, K, R, in_place, apart)
        assert loaded[0] == loaded[1] and loaded[0] in ((2,) if T < 449 else (2, 3)), (T, K, R, loaded)
    assert rows[4][5] == 3


def test_tensors_that_require_grad_are_refused():
    """There is no backward pass: what would lose a gradient without a word is refused, unless the
    caller has said that none is wanted."""
    import torch
    import w6a6_w6a8_integer_amd as fq

    def tensors():
        return {"x": torch.zeros(3, 256, dtype=torch.float16), "y": torch.zeros(3, 48, dtype=torch.float16),
                "adapters": torch.zeros(3, dtype=torch.int32),
                "a": torch.zeros(2, 8, 256, dtype=torch.float16), "b": torch.zeros(2, 48, 8, dtype=torch.float16),
                "scales": torch.ones(2), "out": torch.zeros(3, 48, dtype=torch.float16)}

    for name in ("x", "y", "a", "b", "scales", "out"):
        args = tensors()
        args[name].requires_grad_()
        with pytest.raises(ValueError, match=f"{name} requires grad"):
            fq.lora_add(**args)
        args = {k: v for k, v in args.items() if k in ("x", "y", "adapters", "a", "b", name)}
        with pytest.raises(ValueError, match=f"{name} requires grad"):
            fq.lora_add(**args)
        for off in (torch.no_grad, torch.inference_mode):
            with off(), pytest.raises(TypeError, match="CUDA"):       # the next refusal
                fq.lora_add(**args)
    with pytest.raises(TypeError, match="CUDA"):
        fq.lora_add(**tensors())
