"""GPU numerics of gemv_w4: large activations where the codes are zero, and the forms a
product takes by its sizes.  Bounds come from the definition: fp32 products (exact) and
sums, the output rounded once.
"""
import numpy as np
import pytest

import serve_reference as ref

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DEV = "cuda:0"
F16, BF16 = torch.float16, torch.bfloat16
U = 2.0 ** -23


@pytest.fixture(scope="module")
def fq():
    import w6a6_w6a8_integer_amd as fq
    fq.lib()
    return fq


def bound(x, q, s, group, dtype):
    """(Y, tolerance) in 64 bits, x [M][K], q [N][K], s [N][K / group]: n fp32 additions in any
    order err by at most n u times the sum of what is added."""
    w = q.astype(np.float64) * np.repeat(s.astype(np.float64), group, 1)
    y, total = x @ w.T, np.abs(x) @ np.abs(w).T
    adds = group + q.shape[1] // group + 16
    return y, adds * U * total + ref.OUT_EPS[dtype] * np.abs(y) * (1 + 2.0 ** -7) \
        + ref.OUT_ABS[dtype]


@pytest.mark.parametrize("M", [1, 4, 13, 29, 50])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_large_activations_at_zero_codes(fq, dtype, group, M):
    """One activation of a group is 100,000 times the others (a down projection's outliers), and
    the codes there are zero: the sum is the others', to their own precision."""
    r = np.random.default_rng([M, group])
    N, K = 80, 512
    q = r.integers(-8, 8, (N, K))
    s = np.full((N, K // group), 2.0 ** -6, np.float16)
    x = (0.02 * r.standard_normal((M, K))).astype(np.float32)
    for g in range(K // group):
        at = g * group + int(r.integers(group))
        x[:, at] = 2000 * (1 - 2 * r.integers(0, 2, M))
        q[:, at] = 0
    x = torch.from_numpy(x).to(dtype)
    y = fq.gemv_w4(x.to(DEV), torch.from_numpy(ref.pack_w4(q).view(np.int32)).to(DEV),
                   torch.from_numpy(np.ascontiguousarray(s.T)).to(DEV), N)
    want, tol = bound(x.double().numpy(), q, s, group, dtype)
    err = np.abs(y.double().cpu().numpy() - want)
    assert (err <= tol).all(), float((err / tol).max())
