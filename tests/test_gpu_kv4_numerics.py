"""Precision of the attention over the 4-bit cache (flexq_kv4_attention) where the values cancel, their
scales lie far apart, or the scale of the scores vanishes.  Bounds are those that
kv4_reference.py derives for two halves of p s, for both types of rows."""
import numpy as np
import pytest

import kv4_reference as ref
import test_gpu_kv4 as base

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def fq():
    import w6a6_w6a8_integer_amd as fq
    fq.lib()
    return fq


def check_two_parts(p, out, lse, scale):
    """Every row against the definition, p s in two halves whatever the type of the rows."""
    q, out, lse = (x.double().cpu().numpy() for x in (p["q"], out, lse))
    table, Hkv, D = p["table"].cpu().numpy(), p["cache"][0].shape[1], p["q"].shape[2]
    arrays, at = base.flat(p["cache"]), 0
    for b, (ctx, n) in enumerate(zip(p["lens"], p["new"])):
        rows, pos = slice(at, at + n), np.arange(ctx + n)
        at += n
        slots = table[b][pos // p["page"]] * p["page"] + pos % p["page"]
        key, value = ref.read(*arrays, slots, Hkv, D, p["page"])
        seen = ref.attended(ctx, n, p["masks"][b], 0, 0)
        want, want_lse, tol, tol_lse = ref.attention(q[rows], key, value, seen, scale, F16)
        tol = tol + ref.OUT_EPS[p["dtype"]] * np.abs(want) * (1 + 2.0 ** -7) + ref.OUT_ABS[p["dtype"]]
        err = np.abs(out[rows] - want)
        wrong = np.argwhere(~(err <= tol))
        assert len(wrong) == 0, (b, len(wrong), wrong[:3].tolist(), float((err / tol).max()))
        assert (np.abs(lse[rows] - want_lse) <= tol_lse).all()


# ctx, new, H, Hkv, D, tree: 1, 2, 4 rows a lane's columns and two groups of them, one and several shares
CANCEL = [([2, 4, 1], [1, 1, 1], 4, 2, 64, False), ([5], [1], 16, 2, 128, False),
          ([3, 9], [1, 2], 12, 1, 96, False), ([7, 2], [3, 3], 16, 2, 128, True),
          ([4, 30], [7, 5], 16, 2, 64, True), ([6], [2], 4, 1, 256, False), ([1500], [1], 8, 1, 64, False)]


@pytest.mark.parametrize("ctx,new,H,Hkv,D,tree", CANCEL)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_values_that_cancel(fq, ctx, new, H, Hkv, D, tree, dtype):
    """Rows of values whose offset takes off what their codes give, so that what a probability errs
    by stands alone in the output: codes of 15 and b = -15 s, so that every row is 0."""
    r = base.rng(61, *ctx, H, D)
    p = base.problem(fq, r, ctx, new, H, Hkv, D, 16, dtype, tree, by=0.001)
    p["cache"][1].fill_(-1)
    p["cache"][2][..., 2, :], p["cache"][2][..., 3, :] = 1.0, -15.0
    out, lse = base.run(fq, p, max(new))
    check_two_parts(p, out, lse, D ** -0.5)
