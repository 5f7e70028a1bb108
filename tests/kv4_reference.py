"""The 4-bit cache's operators and the low-rank adapters from their definitions, in 64 bits on
the CPU, and the error bounds the GPU results are held to.

Bounds, with u = 2^-23 the largest relative error of one fp32 operation (a matrix instruction
may truncate); a sum of n products in any order errs by at most n u sum|products|.

* attention: a score is s (q.(c - 8) + 8 Q) + b Q with Q = sum q.  The product and Q are sums
  of D terms, so the score errs by d = (D + 16) u scale S, S = sum|q| (s (|c - 8| + 8) + |b|); a
  query below 2^-24 of the row's largest |q| errs by 2^-34 of that, in the product.  (Formed as
  s (q.(64 + c) - 64 Q), D / 32 steps that each round a sum of at most (64 + 79) sum|q| err by
  4.5 D u s sum|q|, less than the 8 D u s sum|q| that are in d.)  A probability
  errs by a factor 1 +- 2 d; the sums over the keys add (L / 32 + 64) u, and p s enters as two
  halves, within 2^-22 of itself or 2^-35 of the row's largest p s.  A value is
  (p s) (c - 8) + p (b + 8 s), so all of that is relative to V = s |c - 8| + |b| + 8 s.  For
  bfloat16 p s enters as one half, p s (1 + e) with |e| <= 2^-11, in (p s) (c - 8) and in 8 (p s)
  alike: together (p s) c e, so out errs by 2^-11 of the mean of s c besides.
* adapters: h = A x errs by (K + 16) u sum|a||x|, and enters as two parts, within e = 2^-17
  (fp16: 2^-22) of itself or 2^-38 of the token's largest; B h by (2 R + 64) u sum|b||h|.
* an output is rounded once: half a step (2^-11 fp16, 2^-8 bf16), subnormal ones half of the
  least one.
"""
import math

import numpy as np
import torch

U = 2.0 ** -23
OUT_EPS = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
OUT_ABS = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}


def quantize(x):
    """(codes int64 [..][D], scales, offsets fp16 [..]) of fp32 rows x [..][D]."""
    x = x.astype(np.float32)
    with np.errstate(all="ignore"):
        low, high = x.min(-1), x.max(-1)
        b = low.astype(np.float16)
        s = ((high - low) / np.float32(15)).astype(np.float16)
        bad = np.isnan(x).any(-1) | ~np.isfinite(b) | ~np.isfinite(s)
        b, s = np.where(bad, np.float16(np.nan), b), np.where(bad, np.float16(np.nan), s)
        sf, bf = s.astype(np.float32)[..., None], b.astype(np.float32)[..., None]
        c = np.clip(np.rint((x - bf) / sf), 0, 15)
    c = np.where((sf == 0) | bad[..., None], 0, c)
    return c.astype(np.int64), s, b


def places(slot, h, d, Hkv, D, page):
    """((dword, bit) of a key's code, of a value's, place of the key's scale) of (slot, head, d):
    the header's formulas."""
    block = (slot // page * Hkv + h) * (page // 16) + slot % page // 16
    r = slot % 16
    byte = np.array([0, 2, 1, 3])[r % 4]
    return ((block * 2 * D + r * (D // 8) + d // 8, 4 * (d % 8 // 2) + 16 * (d % 2)),
            (block * 2 * D + r // 8 * D + d // 2 * 2 + r % 8 // 4, 8 * byte + 4 * (d % 2)),
            block * 64 + r)


def write(kc, vc, sc, k, v, slots, page):
    """Flat caches (uint32, uint32, fp16) with tokens k, v [T][Hkv][D] (fp32) written at slots,
    dropped outside."""
    T, Hkv, D = k.shape
    n = sc.size // (4 * Hkv)
    h, d = np.meshgrid(np.arange(Hkv), np.arange(D), indexing="ij")
    for x, at, codes in ((k, 0, kc), (v, 1, vc)):
        c, s, b = quantize(x)
        for t in range(T):
            slot = int(slots[t])
            if not 0 <= slot < n:
                continue
            p = places(slot, h, d, Hkv, D, page)
            word, bit = p[at]
            np.bitwise_and.at(codes, word.ravel(), ~(np.uint32(15) << bit.ravel().astype(np.uint32)))
            np.bitwise_or.at(codes, word.ravel(),
                             (c[t].astype(np.uint32) << bit.astype(np.uint32)).ravel())
            sc[p[2][:, 0] + 32 * at], sc[p[2][:, 0] + 32 * at + 16] = s[t], b[t]


def read(kc, vc, sc, slots, Hkv, D, page):
    """(codes, scales, offsets) of keys and of values at slots, float64 [T][Hkv][D] and [T][Hkv]."""
    slot, h, d = np.meshgrid(np.asarray(slots), np.arange(Hkv), np.arange(D), indexing="ij")
    p = places(slot, h, d, Hkv, D, page)
    out = []
    for at, codes in ((0, kc), (1, vc)):
        word, bit = p[at]
        c = (codes[word] >> bit.astype(np.uint32)) & 15
        place = p[2][:, :, 0] + 32 * at
        out.append((c.astype(np.float64), sc[place].astype(np.float64),
                    sc[place + 16].astype(np.float64)))
    return out


def attended(ctx, n, mask, window, sinks):
    """bool [n][ctx + n]: what each drafted token attends; mask bool [n][n], None for a chain."""
    pos = np.arange(ctx + n)
    seen = np.zeros((n, ctx + n), bool)
    for t in range(n):
        drafted = np.arange(n) <= t if mask is None else np.asarray(mask[t])
        since = ctx + int(drafted.sum()) - window if window else 0
        inside = (pos >= since) | (pos < (sinks if window else 0))
        seen[t, :ctx] = inside[:ctx]
        seen[t, ctx:] = drafted & inside[ctx:] if mask is None else drafted
    return seen


def attention(q, key, value, seen, scale, dtype=torch.float16):
    """One request: q float64 [n][H][D]; key, value as read() gives them, for its tokens (NaN in
    places that are not attended does not matter); seen bool [n][L].  Returns (out, lse,
    tolerance of out without its rounding, of lse)."""
    n, H, D = q.shape
    Hkv = key[0].shape[1]
    group = H // Hkv
    out, tol = np.zeros((n, H, D)), np.zeros((n, H, D))
    lse, tol_lse = np.full((n, H), -math.inf), np.zeros((n, H))
    for t in range(n):
        at = np.nonzero(seen[t])[0]
        if len(at) == 0:
            continue
        L = len(at)
        for h in range(Hkv):
            kc, ks, kb = (x[at, h] for x in key)
            vc, vs, vb = (x[at, h] for x in value)
            k = kc * ks[:, None] + kb[:, None]
            v = vc * vs[:, None] + vb[:, None]
            size = np.abs(kc - 8) * ks[:, None] + (8 * ks + np.abs(kb))[:, None]
            V = np.abs(vc - 8) * vs[:, None] + (8 * vs + np.abs(vb))[:, None]
            rows = q[t, h * group:(h + 1) * group]
            s = scale * (rows @ k.T)                                       # [group][L]
            d = (abs(scale) * ((D + 16) * U * (np.abs(rows) @ size.T) + 2.0 ** -34
                               * np.abs(rows).max(1, keepdims=True) * size.sum(1))).max(1)
            top = s.max(1, keepdims=True)
            e = np.exp(s - top)
            w = e / e.sum(1, keepdims=True)
            g = slice(h * group, (h + 1) * group)
            out[t, g] = w @ v
            lse[t, g] = top[:, 0] + np.log(e.sum(1))
            rel = 2 * d + 2.0 ** -22 + (L / 32 + 64) * U
            least = 2.0 ** -35 * (w * vs).max(1, keepdims=True) * 8 * L
            tol[t, g] = 2 * rel[:, None] * (w @ V) + least
            if dtype == torch.bfloat16:
                tol[t, g] += 2.0 ** -11 * (w @ (vc * vs[:, None]))
            tol_lse[t, g] = 2 * d + (L / 32 + 64) * U + 4 * U * np.abs(lse[t, g])
    return out, lse, tol, tol_lse


def lora(x, y, adapters, a, b, ranks, scales, dtype):
    """(out, tolerance with its rounding): float64 x [T][K], y [T][N], a [L][R][K], b [L][N][R]
    (what they hold past a rank does not matter)."""
    out = y.copy()
    tol = np.zeros_like(y)
    part = 2.0 ** -22 if dtype == torch.float16 else 2.0 ** -17
    K = x.shape[1]
    L, R = a.shape[:2]
    for t, i in enumerate(adapters):
        if not 0 <= i < L:
            continue
        r = R if ranks is None else min(max(0, int(ranks[i])), R)
        by = 1.0 if scales is None else float(scales[i])
        A, B = a[i, :r], b[i, :, :r]
        h, size = A @ x[t], np.abs(A) @ np.abs(x[t])
        out[t] += by * (B @ h)
        most = np.abs(h).max() if r else 0.0
        tol[t] = abs(by) * (np.abs(B) @ (((K + 2 * R + 80) * U + part) * size + 2.0 ** -38 * most))
    return out, tol + OUT_EPS[dtype] * np.abs(out) * (1 + 2.0 ** -7) + OUT_ABS[dtype]
