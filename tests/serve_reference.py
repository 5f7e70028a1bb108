"""The decoding-step operators from their definitions, in 64 bits on the CPU, and the
error bounds the GPU results are held to.

Bounds.  u = 2^-23 is the largest relative error of one fp32 operation (a matrix
instruction may truncate).  A sum of n products in any order errs by at most
n u sum|products|.

* gemv_w4: a group's codes enter as q + 24 and 24 sum x is taken off, so its partial sums
  reach 31 sum|x|; 32 products an instruction, eight instructions a group: 40 u of that.
  The group sums add (G + 16) u S with S = sum |s x q|, and the output is rounded
  (2^-11 fp16, 2^-8 bf16, and an absolute 2^-24 for a subnormal fp16).
* attention: a score errs by d = (D + 8) u scale sum|q k| (the conversion to base 2 and
  the maximum's subtraction included), so a probability by a factor 1 +- 2 d; the sum
  over the keys adds (L / 32 + 64) u and the two-part probabilities 2^-16 of each, in the
  numerator and in the denominator alike; below the fp16 normals a part errs by 2^-25
  absolute, where the largest probability is at least 1 before the division.
"""
import math

import numpy as np
import torch

U = 2.0 ** -23
OUT_EPS = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
OUT_ABS = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}


# ---- 4-bit weights -------------------------------------------------------------------


def quantize_w4(w, group):
    """(codes int [N][K], scales fp16 [N][K / group]) of float32 weights."""
    N, K = w.shape
    g = w.astype(np.float32).reshape(N, K // group, group)
    s16 = (np.abs(g).max(2) / np.float32(7)).astype(np.float16)
    s = s16.astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.clip(np.rint(g / s), -7, 7)
    q = np.where(s == 0, 0, q)
    return q.reshape(N, K).astype(np.int64), s16


def pack_w4(q):
    """Packed dwords of codes [N][K], by the header's formula."""
    N, K = q.shape
    n, k = np.meshgrid(np.arange(N), np.arange(K), indexing="ij")
    dword = ((n // 16) * (K // 128) + k // 128) * 256 + ((k % 32) // 8 * 16 + n % 16) * 4 \
        + (k % 128) // 32
    c = k % 8
    out = np.zeros(N * K // 8, np.uint32)
    np.bitwise_or.at(out, dword.ravel(),
                     ((q + 8).astype(np.uint32) << (4 * (c // 2) + 16 * (c % 2)).astype(np.uint32))
                     .ravel())
    return out


def gemv(x, q, s, group):
    """(Y, bound of the fp32 sums' error) in 64 bits: x [M][K], q [N][K], s [N][K / group]."""
    s = np.repeat(s.astype(np.float64), group, 1)
    w, x = q.astype(np.float64) * s, x.astype(np.float64)
    groups = q.shape[1] // group
    return x @ w.T, U * ((groups + 16) * (np.abs(x) @ np.abs(w).T) + 40 * 31 * (np.abs(x) @ s.T))


def gemv_tolerance(y, sums, dtype):
    return sums + OUT_EPS[dtype] * np.abs(y) * (1 + 2.0 ** -7) \
        + OUT_ABS[dtype]


# ---- the paged cache -----------------------------------------------------------------


def block_tables(ctx, new, free, table, page, most, head=0):
    """(table, slots, cu, counts); -1 where a table or the free list ends too soon."""
    table = table.copy()
    B, cols = table.shape
    slots = np.full(most, -1, np.int64)
    cu, taken = [0], 0
    for b in range(B):
        c, n = max(0, int(ctx[b])), max(0, int(new[b]))
        have, need = -(-c // page), -(-(c + n) // page)
        for i in range(have, need):
            f = head + taken
            if i < cols:
                table[b, i] = free[f] if 0 <= f < len(free) else -1
            taken += 1
        for i in range(n):
            t, p = cu[-1] + i, c + i
            if t < most and p // page < cols and table[b, p // page] >= 0:
                slots[t] = int(table[b, p // page]) * page + p % page
        cu.append(cu[-1] + n)
    return table, slots, np.array(cu), np.array([cu[-1], taken, head + taken])


def cache_index(slot, h, d, Hkv, D, page):
    """Flat element indexes of (slot, head, d) in the key and the value cache."""
    block = (slot // page * Hkv + h) * (page // 16) + slot % page // 16
    r = slot % 16
    return block * 16 * D + d // 32 * 512 + r * 32 + d % 32, block * 16 * D + d * 16 + r


def write_cache(kc, vc, k, v, slots, page):
    """Flat caches with tokens k, v [T][Hkv][D] written at slots (dropped outside)."""
    T, Hkv, D = k.shape
    n = kc.size // (Hkv * D)
    h, d = np.meshgrid(np.arange(Hkv), np.arange(D), indexing="ij")
    for t in range(T):
        if 0 <= slots[t] < n:
            ik, iv = cache_index(int(slots[t]), h, d, Hkv, D, page)
            kc[ik], vc[iv] = k[t], v[t]


def attention(q, keys, values, ctx, new, mask, scale):
    """One request: q [n][H][D], keys and values [ctx + n][Hkv][D] (float64 tensors; NaN
    in places that are not attended does not matter), mask bool [n][n] of the drafted
    tokens.  Returns (out, lse, tolerance of out without its rounding, of lse)."""
    n, H, D = q.shape
    L, Hkv = keys.shape[0], keys.shape[1]
    out = torch.zeros(n, H, D, dtype=torch.float64)
    lse = torch.full((n, H), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for t in range(n):
        at = torch.cat((torch.arange(ctx), ctx + torch.nonzero(mask[t])[:, 0])).long()
        if at.numel() == 0:
            continue
        for h in range(H):
            k, v = keys[at, h // (H // Hkv)], values[at, h // (H // Hkv)]
            s = scale * (k @ q[t, h])
            d = float(((D + 8) * U * abs(scale) * (k.abs() @ q[t, h].abs())).max())
            w = torch.softmax(s, 0)
            out[t, h] = w @ v
            lse[t, h] = torch.logsumexp(s, 0)
            top = float(w.max())
            tol[t, h] = 2 * (2 * d + 2.0 ** -16 + (L / 32 + 64) * U) * (w @ v.abs()) \
                + 2.0 ** -24 * top * v.abs().sum(0)
            tol_lse[t, h] = 2 * d + (L / 32 + 64) * U + 4 * U * abs(float(lse[t, h]))
    return out, lse, tol, tol_lse
