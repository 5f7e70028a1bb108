// serve_attention.hip -- attention of drafted tokens over the paged cache.
//
// For the rows of one request and key head (new tokens x query heads of the group), with
// K and V of up to ctx + new tokens: S = scale K Q^T, P = 2^(S log2 e - m) with a running
// maximum m per row, O = V^T P, l = sum P; out = O / l.  One pass over the cache.
//
// Both products are 16x16x32 MFMAs with the rows as columns, so a lane owns one row's
// statistics: D of K Q^T gives lane l the scores of row l % 16 at four keys, and the
// fragment of P that V^T P takes wants eight consecutive keys of that row.  The keys of
// a 32-key step are dealt to the two score tiles so that they are the same eight: row r
// of score tile t holds key 8 (r / 4) + 4 t + r % 4, so lane l ends up with keys
// 8 (l / 16) .. + 7 and no exchange between lanes is needed.  K and V fragments come
// straight from memory, 16 bytes a lane, in the cache's own order.
#include <algorithm>

#include "kernels.h"
#include "serve_device.h"
#include "serve_kernels.h"

namespace flexq {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWaves = 4;

// (max, sum) over the four lanes that hold one row (l, l ^ 16, l ^ 32, l ^ 48)
__device__ __forceinline__ float row_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float row_sum(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

// the low n bits, n clamped to 0 .. 8
__device__ __forceinline__ uint32_t low_bits(int64_t n) {
  return n <= 0 ? 0u : (n >= 8 ? 0xFFu : (1u << (int)n) - 1u);
}

}  // namespace

// One workgroup = one request, key head and block of 16 NT rows; its four waves take the
// 32-key steps in turn and join their (m, l, O) through LDS at the end.
template <class E, int DT, int NT>
__global__ __launch_bounds__(64 * kWaves) void tree_attention_kernel(const AttentionArgs a) {
  constexpr int D = 32 * DT;
  constexpr int OT = 2 * DT;  // 16-wide slices of D
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 15, p = lane >> 4;
  const int b = blockIdx.x, hk = blockIdx.y;
  const int group = a.H / a.Hkv;
  const int cu = a.cu[b];
  const int n_new = min(max(0, a.cu[b + 1] - cu), a.max_new);
  const int64_t ctx = min(max(0, a.ctx[b]), a.max_blocks << a.page_shift);
  const int rows = n_new * group;
  const int row0 = blockIdx.z * (16 * NT);
  if (row0 >= rows) return;
  const int64_t len = min(ctx + n_new, (int64_t)a.max_blocks << a.page_shift);
  const int steps = (int)((len + 31) >> 5);

  u32x4 qf[NT][DT];
  int tok[NT];  // the row's token in its request
#pragma unroll
  for (int rt = 0; rt < NT; ++rt) {
    const int r = row0 + rt * 16 + c;
    tok[rt] = r / group;
    const int64_t t = (int64_t)cu + tok[rt];
    const bool in = r < rows && t >= 0 && t < a.T;
    const uint16_t* src = a.q + t * a.q_st + (int64_t)(hk * group + r % group) * a.q_sh + 8 * p;
#pragma unroll
    for (int ks = 0; ks < DT; ++ks)
      qf[rt][ks] = in ? *reinterpret_cast<const u32x4*>(src + 32 * ks) : u32x4{};
  }

  const int per_page = 1 << (a.page_shift - 4);  // 16-token blocks of a page
  const int32_t* table = a.table + (int64_t)b * a.max_blocks;
  // 16-token block of the step's token at 32 step + 16 half, -1 where there is none
  auto block_of = [&](int step, int half) {
    const int64_t pos = (int64_t)step * 32 + half * 16;
    if (pos >= len) return -1;
    const int id = table[pos >> a.page_shift];
    if ((unsigned)id >= (unsigned)a.num_pages) return -1;
    return (id * a.Hkv + hk) * per_page + (int)((pos >> 4) & (per_page - 1));
  };

  f32x4 o[NT][OT] = {};
  float m[NT], l[NT];
#pragma unroll
  for (int rt = 0; rt < NT; ++rt) {
    m[rt] = -INFINITY;
    l[rt] = 0.0f;
  }
  const float scale = a.scale * kLog2e;

  for (int step = wave; step < steps; step += kWaves) {
    const int kblk = block_of(step, c >> 3), vblk = block_of(step, p >> 1);
    u32x4 kf[2][DT], vf[OT];
    const uint16_t* ksrc =
        a.kc + (int64_t)max(kblk, 0) * (16 * D) + (8 * ((c >> 2) & 1) + (c & 3)) * 32 + 8 * p;
    const uint16_t* vsrc = a.vc + (int64_t)max(vblk, 0) * (16 * D) + c * 16 + 8 * (p & 1);
#pragma unroll
    for (int ks = 0; ks < DT; ++ks)
#pragma unroll
      for (int t = 0; t < 2; ++t)
        kf[t][ks] = *reinterpret_cast<const u32x4*>(ksrc + ks * 512 + t * 128);
#pragma unroll
    for (int dt = 0; dt < OT; ++dt)
      vf[dt] = *reinterpret_cast<const u32x4*>(vsrc + dt * 256);

    // Keys that are no context (drafted, or none at all) or on no page: the wave masks.
    const int64_t key0 = (int64_t)step * 32 + 8 * p;  // this lane's first key
    const bool masked = __ballot(vblk < 0 || key0 + 8 > ctx) != 0;
    const uint32_t there = vblk < 0 ? 0u : low_bits(len - key0);  // keys that exist
    bool poison = false;  // a value in this step is infinite or NaN
    u32x4 vbad[OT];
    if (masked) {
      bool bad = false;
#pragma unroll
      for (int dt = 0; dt < OT; ++dt) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t keep = ((there >> (2 * i)) & 1u) * 0xFFFFu;
          keep |= ((there >> (2 * i + 1)) & 1u) * 0xFFFF0000u;
          const uint32_t v = vf[dt][i] & keep;
          uint32_t ex = (v & E::kExponent) == E::kExponent ? 0xFFFFu : 0u;
          ex |= ((v >> 16) & E::kExponent) == E::kExponent ? 0xFFFF0000u : 0u;
          bad |= ex != 0;
          vbad[dt][i] = v & ex;
          vf[dt][i] = v & ~ex;
        }
      }
      poison = __ballot(bad) != 0;
    }

#pragma unroll
    for (int rt = 0; rt < NT; ++rt) {
      f32x4 s[2] = {};
#pragma unroll
      for (int ks = 0; ks < DT; ++ks)
#pragma unroll
        for (int t = 0; t < 2; ++t) s[t] = E::mfma(kf[t][ks], qf[rt][ks], s[t]);
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = s[e >> 2][e & 3] * scale;
      uint32_t seen = 0xFFu;
      if (masked) {
        // attended keys among this lane's eight: the context, then the tree's bits (or,
        // for a chain, the tokens up to the row's own)
        const int64_t j0 = key0 - ctx;  // drafted index of the first key (may be negative)
        if (a.mask) {
          seen = low_bits(-j0);
          const int64_t t = (int64_t)cu + tok[rt];
          if (j0 > -8 && tok[rt] < n_new && t >= 0 && t < a.T) {
            const int32_t* words = a.mask + t * a.mask_words;
            const int64_t w = j0 >> 5;
            const uint32_t w0 = w >= 0 && w < a.mask_words ? (uint32_t)words[w] : 0u;
            const uint32_t w1 = w + 1 < a.mask_words ? (uint32_t)words[w + 1] : 0u;
            seen |= (uint32_t)(((uint64_t)w1 << 32 | w0) >> (j0 & 31)) & 0xFFu;
          }
        } else {
          seen = low_bits(tok[rt] + 1 - j0);
        }
        seen &= there;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (!((seen >> e) & 1u)) x[e] = -INFINITY;
      }
      float top = x[0];
#pragma unroll
      for (int e = 1; e < 8; ++e) top = fmaxf(top, x[e]);
      top = fmaxf(m[rt], row_max(top));
      const float ref = top == -INFINITY ? 0.0f : top;
      const float by = exp2f(m[rt] - ref);
      m[rt] = top;
      l[rt] *= by;
#pragma unroll
      for (int dt = 0; dt < OT; ++dt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[rt][dt][i] *= by;
      // P as the sum of two 16-bit parts
      u32x4 hi, lo;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t h[2], w[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float v = exp2f(x[2 * i + k] - ref);
          l[rt] += v;
          h[k] = E::bits(v);
          w[k] = E::bits(v - E::value((uint16_t)h[k]));
        }
        hi[i] = h[0] | h[1] << 16;
        lo[i] = w[0] | w[1] << 16;
      }
#pragma unroll
      for (int dt = 0; dt < OT; ++dt) {
        o[rt][dt] = E::mfma(vf[dt], hi, o[rt][dt]);
        o[rt][dt] = E::mfma(vf[dt], lo, o[rt][dt]);
      }
      if (poison) {
        // infinite or NaN values reach only the rows that attend their keys: one key at
        // a time, and a row that does not attend it keeps its sum
        for (int k = 0; k < 32; ++k) {
          const bool mine = p == (k >> 3);
          const int e = k & 7;
          const uint32_t keep = mine ? 0xFFFFu << (16 * (e & 1)) : 0u;
          const bool attends = (__shfl((int)seen, (k >> 3) * 16 + c) >> e) & 1;
          u32x4 one = {};
#pragma unroll
          for (int i = 0; i < 4; ++i) one[i] = i == (e >> 1) ? hi[i] & keep : 0u;
#pragma unroll
          for (int dt = 0; dt < OT; ++dt) {
            u32x4 v = {};
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = i == (e >> 1) ? vbad[dt][i] & keep : 0u;
            const f32x4 with = E::mfma(v, one, o[rt][dt]);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[rt][dt][i] = attends ? with[i] : o[rt][dt][i];
          }
        }
      }
    }
  }

  // Join the four waves, one 16-row tile at a time.
  __shared__ f32x4 part[kWaves][16][D / 4 + 1];  // [wave][row][d / 4], padded rows
  __shared__ float stat[2][kWaves][16];
#pragma unroll
  for (int rt = 0; rt < NT; ++rt) {
    const float sum = row_sum(l[rt]);
#pragma unroll
    for (int dt = 0; dt < OT; ++dt) part[wave][c][4 * dt + p] = o[rt][dt];
    if (p == 0) {
      stat[0][wave][c] = m[rt];
      stat[1][wave][c] = sum;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * (D / 4); i += 64 * kWaves) {
      const int r = i / (D / 4), d4 = i % (D / 4);
      const int row = row0 + rt * 16 + r;
      const int64_t t = (int64_t)cu + row / group;
      float top = -INFINITY, total = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top = fmaxf(top, stat[0][w][r]);
      const float ref = top == -INFINITY ? 0.0f : top;
      float acc[4] = {};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float by = exp2f(stat[0][w][r] - ref);
        total = fmaf(stat[1][w][r], by, total);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] = fmaf(part[w][r][d4][k], by, acc[k]);
      }
      if (row < rows && t >= 0 && t < a.T) {
        const int h = hk * group + row % group;
        u32x2 v;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float x = total != 0.0f ? acc[2 * k] / total : 0.0f;
          const float y = total != 0.0f ? acc[2 * k + 1] / total : 0.0f;
          v[k] = E::bits(x) | (uint32_t)E::bits(y) << 16;
        }
        *reinterpret_cast<u32x2*>(a.out + (t * a.H + h) * D + 4 * d4) = v;
        if (a.lse && d4 == 0)
          a.lse[t * a.H + h] = total != 0.0f ? (ref + log2f(total)) * kLn2 : -INFINITY;
      }
    }
    __syncthreads();
  }
}

namespace {

template <class E, int DT>
hipError_t launch_rows(const AttentionArgs& a, hipStream_t stream) {
  const int64_t rows = (int64_t)a.max_new * (a.H / a.Hkv);
  const int nt = rows <= 16 ? 1 : 2;
  const dim3 grid((unsigned)a.B, (unsigned)a.Hkv, (unsigned)((rows + 16 * nt - 1) / (16 * nt)));
  return launch_kernel(nt == 1 ? tree_attention_kernel<E, DT, 1> : tree_attention_kernel<E, DT, 2>,
                       grid, dim3(64 * kWaves), stream, a);
}

template <class E>
hipError_t launch_width(const AttentionArgs& a, hipStream_t stream) {
  switch (a.D) {
    case 64: return launch_rows<E, 2>(a, stream);
    case 96: return launch_rows<E, 3>(a, stream);
    case 128: return launch_rows<E, 4>(a, stream);
    default: return launch_rows<E, 8>(a, stream);
  }
}

}  // namespace

size_t attention_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t) { return 16; }

hipError_t launch_tree_attention(const AttentionArgs& a, bool bf16, hipStream_t stream) {
  return bf16 ? launch_width<Bfloat>(a, stream) : launch_width<Half>(a, stream);
}

}  // namespace flexq
