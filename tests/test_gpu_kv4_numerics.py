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


def two_kinds(fq, r, n, H, Hkv, D, dtype, first, rest, drop):
    """One request of n tokens whose keys are one number each, so that a score is scale * sum(q) times it:
    0.37 for every seventh token from the first on, and less by `drop` powers of 2 for the others.
    Their values' scales are 2^first and 2^rest, and all values are 0."""
    p = base.problem(fq, r, [n - 1], [1], H, Hkv, D, 16, dtype, False)
    scores = np.full(n, 0.37 - drop * np.log(2) / D ** 0.5)
    steps = np.full(n, 2.0 ** rest)
    scores[::7], steps[::7] = 0.37, 2.0 ** first
    sc = base.flat(p["cache"])[2].copy().reshape(-1, Hkv, 1, 4, 16)
    for i in range(n):
        page = int(p["table"][0, i // 16])
        sc[page, :, 0, :, i % 16] = 0.0, scores[i], steps[i], -15 * steps[i]
    p["cache"][1].fill_(-1)
    p["cache"][2].copy_(torch.from_numpy(sc))
    near = 1 + 0.03 * r.random((1, H, 1))                 # (sums of q that differ from head to head)
    p["q"].copy_(torch.from_numpy(np.broadcast_to(near, (1, H, D)).copy()).to(dtype))
    return p


# of every eight keys that a lane holds some take nearly all, with scales far below the others'
@pytest.mark.parametrize("n,H,Hkv", [(2, 4, 1), (8, 8, 1), (9, 16, 1), (30, 32, 1), (50, 4, 4), (900, 4, 2)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_small_scales_of_the_keys_that_count(fq, n, H, Hkv, dtype):
    """The scales of the values that count are 2^30 below those of the ones that do not, whose p s is still
    the smaller: p s of the first keep their bits."""
    p = two_kinds(fq, base.rng(63, n, H), n, H, Hkv, 64, dtype, -18, 12, 36)
    out, lse = base.run(fq, p, 1)
    check_two_parts(p, out, lse, 0.125)


@pytest.mark.parametrize("n,H,Hkv", [(2, 4, 1), (9, 16, 1), (30, 32, 1), (900, 4, 2)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_rows_without_a_scale(fq, n, H, Hkv, dtype):
    """Constant rows of values (scale 0) that take nearly all, others far below them with the largest
    scales: neither probabilities nor sums leave their range."""
    for drop in (40, 90):
        p = two_kinds(fq, base.rng(64, n, H, drop), n, H, Hkv, 64, dtype, 0, 12, drop)
        sc = p["cache"][2]
        first = sc[:, :, :, 2] == 1.0
        sc[:, :, :, 2][first] = 0.0
        sc[:, :, :, 3][first] = 1.25
        out, lse = base.run(fq, p, 1)
        check_two_parts(p, out, lse, 0.125)
        assert bool(((out.float() - 1.25).abs() < 0.01).all())


@pytest.mark.parametrize("by,scale,dtype", [(2.0 ** -50, 1e-30, BF16), (2.0 ** -120, 0.125, BF16), (1.0, 1e-44, F16),
                                            (1.0, 1e-44, BF16), (2.0 ** -20, -1e-42, F16)])
def test_scores_that_vanish(fq, by, scale, dtype):
    """A scale and queries whose product fp32 does not hold: every attended key counts alike, and masked
    ones (the ends of steps, a tree's, those before a window) not at all."""
    for tree, window in ((False, 0), (True, 0), (False, 33)):
        p = base.problem(fq, base.rng(65, tree, window), [40, 133, 3], [2, 1, 4], 4, 2, 64, 16, dtype, tree, by=by)
        out, lse = base.run(fq, p, 4, scale=scale, window=window or None, sinks=3)
        base.check(p, out, lse, scale, window, 3 if window else 0, rms=False)


@pytest.mark.parametrize("ctx,new,H,Hkv,D,tree", CANCEL[:6])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_query_that_is_not_finite_stays_alone(fq, ctx, new, H, Hkv, D, tree, bad):
    """Its row of one head is not finite, and every other row has the bits it had."""
    p = base.problem(fq, base.rng(70, *ctx, H, D), ctx, new, H, Hkv, D, 16, BF16, tree)
    clean, clean_lse = base.run(fq, p, max(new))
    t, h = sum(new) - 1, H // 2
    p["q"][t, h, 3] = bad
    out, lse = base.run(fq, p, max(new))
    assert not bool(out[t, h].isfinite().any())
    out[t, h], lse[t, h] = clean[t, h], clean_lse[t, h]
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse)


def test_most_requests_with_windows(fq):
    """As many requests as a step may have, some without new tokens, under a window."""
    r = base.rng(71)
    ctx, new = r.integers(0, 40, 4096).tolist(), r.integers(0, 3, 4096).tolist()
    p = base.problem(fq, r, ctx, new, 2, 1, 64, 16, F16, False)
    out, lse = base.run(fq, p, 2, window=9, sinks=2)
    base.check(p, out, lse, 0.125, 9, 2)
