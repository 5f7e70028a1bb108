// serve_lora.hip -- low-rank adapters of many requests at once, added to a shared projection's
// output: out[t] = y[t] + s_a B_a (A_a x[t]) for the adapter a of token t.
//
// Two launches: h = A x (fp32, slices of K apart), then out = y + s B h.  Tokens come in any order
// of adapters.  A workgroup takes a tile of 64 consecutive tokens and, one after the other, the
// adapters that occur in it: a lane holds a token's adapter, one ballot finds the tokens that
// share it, and they become the columns of 16x16x32 MFMAs, 16 at a time.  An adapter's rows
// are read once a tile, so a decoding step (one tile) reads each adapter once, and prompts
// (long runs of one adapter) once a tile, from L2.  No sorting launch comes before.
//
// What bounds it: one token with 16 ranks through 4096 x 4096 8.8 us in two launches, chains of latencies
// (adapters, ranks, rows, sums); 64 tokens over 40 adapters of 64 ranks through 10240 x 8192 26.3 us for
// 57 MB (the same chains, and few loads an adapter on their way); prompts of 3500 tokens there 68 us
// for 203 MB: x at 2.9 TB/s through LDS (20), h's slices joined (5), y and out at 3.4 with an
// adapter's rows again for each tile (43).
//
// h enters the second product as two 16-bit parts, for fp16 after a power of two that takes a token's
// largest to 2^14 .. 2^15: within 2^-17 of itself, for fp16 2^-22 or 2^-39 of the largest.
#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "serve_device.h"
#include "serve_kernels.h"

namespace flexq {

namespace {

constexpr int kWaves = 4;
constexpr int kTile = 64;  // tokens, one a lane

// over the lanes that hold one column
__device__ __forceinline__ float column_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}

// The power of 2 that a token's sums enter the second product with, h the lane's of the token (0 past its
// rank): for fp16 it takes the largest that is finite to 2^14 .. 2^15; bfloat16 holds them as they are, and
// weights near its largest would take more past fp32.
template <class E, int KS>
__device__ __forceinline__ int power_of(const float (&h)[KS][8]) {
  if constexpr (!std::is_same_v<E, Half>) return 0;
  float most = 0.0f;
#pragma unroll
  for (int s = 0; s < KS; ++s)
#pragma unroll
    for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(h[s][e]));
  most = column_max(most);
  if (__builtin_expect(__ballot(most == INFINITY) != 0, 0)) {
    most = 0.0f;
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(h[s][e]) < INFINITY ? fabsf(h[s][e]) : 0.0f);
    most = column_max(most);
  }
  return 15 - __builtin_amdgcn_frexp_expf(most);
}

// The adapter of token t0 + lane, -1 where it has none.
__device__ __forceinline__ int adapter_of(const LoraArgs& a, int64_t t0, int lane) {
  const int id = t0 + lane < a.T ? a.adapters[t0 + lane] : -1;
  return id >= 0 && id < a.L ? id : -1;
}

// The tile's members of one adapter in order: member i's token (of the tile) in lane i.
__device__ __forceinline__ int members_list(uint64_t members, int lane) {
  const int n = __builtin_popcountll(members);
  const bool mine = members >> lane & 1;
  // (behind the members the other tokens follow: every lane has a place)
  const int rank = __builtin_popcountll(members & ((1ull << lane) - 1));
  return __builtin_amdgcn_ds_permute((mine ? rank : n + lane - rank) << 2, lane);
}

// The tokens of one adapter in the tile, as this wave sees them: its 16 columns, if it has any, and which
// part of the other axis it takes.
struct Columns {
  int token;        // of the lane's column in the tile; where there is none, the first
  bool in;          // the column exists
  int parts, part;  // waves that share the columns, and which of them this is
  bool idle;
};

__device__ __forceinline__ Columns columns_of(uint64_t members, int lane, int wave) {
  const int n = __builtin_popcountll(members);
  const int list = members_list(members, lane);
  Columns c;
  const int shift = n <= 16 ? 2 : n <= 32 ? 1 : 0;
  c.parts = 1 << shift;
  c.part = wave & (c.parts - 1);
  const int first = (wave >> shift) * 16, column = first + (lane & 15);
  c.in = column < n;
  c.token = __builtin_amdgcn_ds_bpermute((c.in ? column : 0) << 2, list);
  c.idle = first >= n;
  return c;
}

// sum[k] += the eight fp32 at from + r[k] in each `step`-th of `slices` planes `apart` from one another,
// from the `first` on and in order, a few of them on their way at once.
template <int KS>
__device__ __forceinline__ void sum_slices(const float* from, const int (&r)[KS], int64_t apart, int first,
                                           int step, int slices, f32x4 (&sum)[KS][2]) {
  constexpr int U = KS <= 2 ? 4 : 1;
  int q = first;
  for (; q + step < slices; q += U * step) {  // (two at least)
    f32x4 v[U][KS][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float* at = from + min(q + u * step, slices - 1) * apart;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) v[u][k][i] = *reinterpret_cast<const f32x4*>(at + r[k] + 4 * i);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (q + u * step < slices)
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) sum[k][i] += v[u][k][i];
  }
  if (q < slices)
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        sum[k][i] += *reinterpret_cast<const f32x4*>(from + q * apart + r[k] + 4 * i);
}

// h times 2^up as two parts each (an infinite or NaN one is its first part alone).  An h that is not 0 is at
// least the type's least value in its first part, so that an infinite weight gives it an infinity: rounded
// to 0 it is looked for by the smallest of the bits without the sign, less one.
template <class E, int KS>
__device__ __forceinline__ void two_parts(const float (&h)[KS][8], int up, u32x4 (&hi)[KS], u32x4 (&lo)[KS]) {
  uint32_t least = ~0u;
#pragma unroll
  for (int s = 0; s < KS; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v0 = __builtin_amdgcn_ldexpf(h[s][2 * i], up), v1 = __builtin_amdgcn_ldexpf(h[s][2 * i + 1], up);
      const uint32_t b0 = E::bits(v0), b1 = E::bits(v1);
      const float r0 = v0 - E::value((uint16_t)b0), r1 = v1 - E::value((uint16_t)b1);
      hi[s][i] = b0 | b1 << 16;
      lo[s][i] = E::bits(fabsf(r0) < INFINITY ? r0 : 0.0f) |
                 (uint32_t)E::bits(fabsf(r1) < INFINITY ? r1 : 0.0f) << 16;
      least = min(least, min((__float_as_uint(h[s][2 * i]) << 1) - 1, (__float_as_uint(h[s][2 * i + 1]) << 1) - 1));
    }
  // (half of the least value, times 2^-up)
  const float half = __builtin_amdgcn_ldexpf(1.0f, (std::is_same_v<E, Half> ? -25 : -134) - up);
  if (__builtin_expect(__ballot(least < __float_as_uint(half) << 1) != 0, 0)) {
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (h[s][2 * i + k] != 0.0f && (hi[s][i] >> 16 * k & 0x7FFFu) == 0) {
            hi[s][i] |= 1u << 16 * k;
            const float v = __builtin_amdgcn_ldexpf(h[s][2 * i + k], up);
            lo[s][i] = (lo[s][i] & 0xFFFF0000u >> 16 * k) |
                       (uint32_t)E::bits(v - E::value((uint16_t)(hi[s][i] >> 16 * k))) << 16 * k;
          }
  }
}

// An infinite weight times two parts, of which the second may be 0 or of the other sign, is NaN where the
// first part alone gives the infinity: a wave that finds a NaN among its sums forms them again, zeros in
// the place of weights that are not finite where the second parts meet them.  (Looking at the sums
// costs less than looking at every weight: prompts with 128 ranks 98 us against 106.)
template <int N>
__device__ __forceinline__ bool any_nan(const f32x4 (&o)[N]) {
  bool nan = false;
#pragma unroll
  for (int i = 0; i < N; ++i)
    nan |= __builtin_isunordered(o[i][0], o[i][1]) | __builtin_isunordered(o[i][2], o[i][3]);
  return __ballot(nan) != 0;
}
template <class E>
__device__ __forceinline__ u32x4 finite(u32x4 f) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    f[e] &= ((f[e] & E::kExponent) == E::kExponent ? 0xFFFF0000u : ~0u) &
            ((f[e] >> 16 & E::kExponent) == E::kExponent ? 0xFFFFu : ~0u);
  return f;
}

// out = y for the tile's tokens `rows` and columns n0 .. n1: a wave 16 tokens and 256 columns at a time, all
// of them on their way together (one after the other, a tile without adapters took 20 us).
__device__ __forceinline__ void copy_rows(const LoraArgs& a, int64_t t0, uint64_t rows, int n0, int n1, int lane,
                                          int wave) {
  const int count = __builtin_popcountll(rows), list = members_list(rows, lane);
  if (16 * wave >= count) return;
  int64_t token[4];
  bool in[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = 16 * wave + 4 * u + (lane >> 4);
    in[u] = i < count;
    token[u] = t0 + __builtin_amdgcn_ds_bpermute((in[u] ? i : 0) << 2, list);
  }
  for (int n = n0 + 8 * (lane & 15); n < n1; n += 256) {
    u32x4 v[2][4];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int u = 0; u < 4; ++u)
        v[c][u] = __builtin_nontemporal_load(
            reinterpret_cast<const u32x4*>(a.y + token[u] * a.y_st + (n + 128 * c < n1 ? n + 128 * c : n)));
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (in[u] && n + 128 * c < n1)
          __builtin_nontemporal_store(v[c][u],
                                      reinterpret_cast<u32x4*>(a.out + token[u] * a.out_st + n + 128 * c));
  }
}

// f(adapter, tokens that have it) for the adapters of the tile, in the order of their first tokens, from
// the turn-th on every turns-th.
template <class F>
__device__ __forceinline__ void each_adapter(int id, int turn, int turns, F&& f) {
  uint64_t left = __ballot(id >= 0);
  for (int i = 0; left != 0; ++i) {
    const int cur = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
    const uint64_t members = __ballot(id == cur);
    if (i == turn) {
      f(cur, members);
      turn += turns;
    }
    left &= ~members;
  }
}

}  // namespace

// h: one workgroup = a tile's adapters (those of its turn) and a slice of K.  Waves that the columns
// leave over share the slice and add up in LDS.  RT: 16-row tiles of an adapter at most.
template <class E, int RT>
__global__ __launch_bounds__(64 * kWaves) void lora_shrink_kernel(const LoraArgs a, int turns,
                                                                 int slices) {
  __shared__ __attribute__((aligned(16))) f32x4 sums[(kWaves - 1) * RT * 64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, p = lane >> 4;
  const int slice = blockIdx.x % slices, turn = blockIdx.x / slices;
  const int64_t t0 = (int64_t)blockIdx.y * kTile;
  // whole groups of 128
  const int groups = a.K / 128;
  const int k0 = (int)((int64_t)groups * slice / slices) * 128;
  const int k1 = (int)((int64_t)groups * (slice + 1) / slices) * 128;
  const int id = adapter_of(a, t0, lane);
  each_adapter(id, turn, turns, [&](int cur, uint64_t members) {
    const int rank = a.ranks ? min(max(0, a.ranks[cur]), a.R) : a.R;
    const int tiles = (rank + 15) / 16;
    const Columns col = columns_of(members, lane, wave);
    f32x4 h[RT] = {};
    if (!col.idle) {
      const int n = (k1 - k0) / col.parts, at = k0 + n * col.part + 8 * p;
      const uint16_t* x = a.x + (t0 + col.token) * a.x_st + at;
      const uint16_t* w[RT];  // (rows past the adapter's last are read again, and not used)
#pragma unroll
      for (int i = 0; i < RT; ++i)
        w[i] = a.a + ((int64_t)cur * a.R + min(16 * i + c, a.R - 1)) * a.K + at;
      // The adapter's tiles, rounded up to a quarter of the most, as a constant: loads without branches
      // between them can stay on their way while the chunk before is worked on.
      auto run = [&](auto number) __attribute__((always_inline)) {
        constexpr int NT = decltype(number)::value;
        constexpr int U = NT <= 2 ? 8 : NT <= 4 ? 4 : 1;  // steps of a chunk
        struct Chunk {
          u32x4 x[U], w[U][NT];
        };
        auto load = [&](Chunk& f, int k) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            f.x[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(x + k + 32 * u));
#pragma unroll
            for (int i = 0; i < NT; ++i) f.w[u][i] = *reinterpret_cast<const u32x4*>(w[i] + k + 32 * u);
          }
        };
        auto add = [&](const Chunk& f) {
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < NT; ++i) h[i] = E::mfma(f.w[u][i], f.x[u], h[i]);
        };
        int k = 0;
        if (n >= 32 * U) {
          Chunk now;
          load(now, 0);
          for (; k + 64 * U <= n; k += 32 * U) {
            Chunk then;
            load(then, k + 32 * U);
            add(now);
            now = then;
          }
          add(now);
          k += 32 * U;
        }
        for (; k < n; k += 32) {
          const u32x4 xf = *reinterpret_cast<const u32x4*>(x + k);
#pragma unroll
          for (int i = 0; i < NT; ++i)
            h[i] = E::mfma(*reinterpret_cast<const u32x4*>(w[i] + k), xf, h[i]);
        }
      };
      constexpr int Q = RT < 4 ? 1 : RT / 4;
      if (tiles > 3 * Q && RT >= 4)
        run(std::integral_constant<int, RT < 4 ? 1 : RT>{});
      else if (tiles > 2 * Q && RT >= 4)
        run(std::integral_constant<int, RT < 4 ? 1 : 3 * Q>{});
      else if (tiles > Q && RT >= 2)
        run(std::integral_constant<int, RT < 2 ? 1 : 2 * Q>{});
      else if (tiles > 0)
        run(std::integral_constant<int, Q>{});
    }
    if (col.parts > 1) {
      auto place = [&](int of, int i) { return ((of - of / col.parts - 1) * RT + i) * 64 + lane; };
      __syncthreads();  // the sums of the adapter before have been read
      if (col.part > 0)
#pragma unroll
        for (int i = 0; i < RT; ++i) sums[place(wave, i)] = h[i];
      __syncthreads();
      if (col.part > 0) return;
      for (int q = 1; q < col.parts; ++q)
#pragma unroll
        for (int i = 0; i < RT; ++i) h[i] += sums[place(wave + q, i)];
    }
    if (!col.in) return;
    float* to = a.h + ((int64_t)slice * a.T + t0 + col.token) * (16 * RT) + 4 * p;
#pragma unroll
    for (int i = 0; i < RT; ++i)
      if (i < tiles) *reinterpret_cast<f32x4*>(to + 16 * i) = h[i];
  });
}

// The slices' sums, into the first slice's place.  (What lies past a token's rank is summed as it is, and
// not used.)
__global__ __launch_bounds__(256) void lora_join_kernel(float* h, int64_t quads, int slices) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= quads) return;
  f32x4* at = reinterpret_cast<f32x4*>(h) + i;
  f32x4 sum = at[0];
#pragma unroll 4
  for (int q = 1; q < slices; ++q) sum += at[q * quads];
  at[0] = sum;
}

// out: one workgroup = a tile's adapters (those of its turn) and a block of out's columns, in units of 64
// that the waves which share a token's take in turn, the next one's loads on their way while
// one is worked on.  Row r of the MFMA's 16-row tile i is n = 16 (r / 4) + 4 i + r % 4 of the
// unit, so that a lane ends up with 16 consecutive n of its tokens.
template <class E, int RT>
__global__ __launch_bounds__(64 * kWaves, RT <= 4 ? 3 : 1) void lora_expand_kernel(const LoraArgs a, int turns,
                                                                 int blocks, int slices) {
  constexpr int KS = (RT + 1) / 2;  // 32-deep steps over the rank
  __shared__ __attribute__((aligned(16))) f32x4 sums[kWaves * KS * 2 * 64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, p = lane >> 4;
  const int block = blockIdx.x % blocks, turn = blockIdx.x / blocks;
  const int64_t t0 = (int64_t)blockIdx.y * kTile;
  const int units = (a.N + 63) / 64;
  const int unit0 = (int)((int64_t)units * block / blocks);
  const int unit1 = (int)((int64_t)units * (block + 1) / blocks);
  const int id = adapter_of(a, t0, lane);
  if (turn == 0 && a.out != a.y) {  // tokens without an adapter
    const uint64_t rows = __ballot(id < 0 && t0 + lane < a.T);
    copy_rows(a, t0, rows, 64 * unit0, min(64 * unit1, a.N), lane, wave);
  }
  each_adapter(id, turn, turns, [&](int cur, uint64_t members) {
    const int rank = a.ranks ? min(max(0, a.ranks[cur]), a.R) : a.R;
    const float by = a.scales ? a.scales[cur] : 1.0f;
    const Columns col = columns_of(members, lane, wave);
    if (col.idle) return;
    const uint16_t* w = a.b + (int64_t)cur * a.N * a.R;
    const int n_of = 16 * (c >> 2) + (c & 3);
    struct Unit {
      u32x4 y[2], f[KS][4];
    };
    auto load = [&](Unit& u, int unit) {
      const int n0 = 64 * unit, mine = min(n0 + 16 * p, a.N - 16);  // the lane's 16 of out
#pragma unroll
      for (int i = 0; i < 2; ++i)
        u.y[i] = __builtin_nontemporal_load(
            reinterpret_cast<const u32x4*>(a.y + (t0 + col.token) * a.y_st + mine + 8 * i));
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int r = 32 * s + 8 * p < rank ? 32 * s + 8 * p : 0;  // (past the rank: masked below)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t n = min(n0 + n_of + 4 * i, a.N - 1);
          u.f[s][i] = *reinterpret_cast<const u32x4*>(w + n * a.R + r);
        }
      }
    };
    // h's slices: waves that share the tokens sum some each, and exchange
    int at[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) at[s] = 32 * s + 8 * p < rank ? 32 * s + 8 * p : 0;
    f32x4 sum[KS][2] = {};
    sum_slices<KS>(a.h + (t0 + col.token) * (16 * RT), at, a.T * (16 * RT), col.part, col.parts, slices, sum);
    int unit = unit0 + col.part;
    const bool works = unit < unit1;
    Unit now;
    if (works) load(now, unit);
    if (col.parts > 1) {
      f32x4* mine = sums + wave * (KS * 2 * 64) + lane;
      lds_barrier();  // the sums of the adapter before have been read
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) mine[(2 * s + i) * 64] = sum[s][i];
      lds_barrier();
      const f32x4* all = sums + (wave - col.part) * (KS * 2 * 64) + lane;
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          sum[s][i] = all[(2 * s + i) * 64];
          for (int w = 1; w < col.parts; ++w) sum[s][i] += all[(w * KS * 2 + 2 * s + i) * 64];
        }
    }
    if (!works) return;

    // the lane's eight of each 32 of h, scaled, and, after the token's power of 2, their two parts
    u32x4 hi[KS], lo[KS];
    int up;
    {
      float h[KS][8];
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) h[s][e] = 32 * s + 8 * p + e < rank ? sum[s][e >> 2][e & 3] * by : 0.0f;
      up = power_of<E, KS>(h);
      two_parts<E, KS>(h, up, hi, lo);
    }

    auto finish = [&](Unit& now, int unit) __attribute__((always_inline)) {
      const int mine = 64 * unit + 16 * p;
      f32x4 o[4] = {};
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        if (32 * s >= rank) break;
        if (32 * s + 32 > rank)  // what an adapter's rows hold past its rank does not matter
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = 32 * s + 8 * p + 2 * e;
            const uint32_t keep = (r < rank ? 0xFFFFu : 0u) | (r + 1 < rank ? 0xFFFF0000u : 0u);
#pragma unroll
            for (int i = 0; i < 4; ++i) now.f[s][i][e] &= keep;
          }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[i] = E::mfma(now.f[s][i], hi[s], o[i]);
          o[i] = E::mfma(now.f[s][i], lo[s], o[i]);
        }
      }
      if (__builtin_expect(any_nan(o), 0)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[i] = f32x4{};
#pragma unroll
          for (int s = 0; s < KS; ++s)
            if (32 * s < rank) {
              o[i] = E::mfma(now.f[s][i], hi[s], o[i]);
              o[i] = E::mfma(finite<E>(now.f[s][i]), lo[s], o[i]);
            }
        }
      }
      if (!col.in || mine >= a.N) return;
      u32x4 out[2];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          const uint32_t was = now.y[i >> 1][2 * (i & 1) + k / 2];
          const float v0 = E::value((uint16_t)(was & 0xFFFFu)) + __builtin_amdgcn_ldexpf(o[i][k], -up);
          const float v1 = E::value((uint16_t)(was >> 16)) + __builtin_amdgcn_ldexpf(o[i][k + 1], -up);
          out[i >> 1][2 * (i & 1) + k / 2] = E::bits(v0) | (uint32_t)E::bits(v1) << 16;
        }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        __builtin_nontemporal_store(
            out[i], reinterpret_cast<u32x4*>(a.out + (t0 + col.token) * a.out_st + mine + 8 * i));
    };
    // (no branch between a unit's loads and the next one's, so that the wait for the first leaves the
    // second on their way)
    for (; unit + col.parts < unit1; unit += col.parts) {
      Unit then;
      load(then, unit + col.parts);
      finish(now, unit);
      now = then;
    }
    finish(now, unit);
  });
}

// Prompts.  The kernels above take fragments straight from memory: 16 rows, a piece of 16 bytes of each in
// neighbouring lanes, which the address units take one by one (64 cycles a load, the bound with 64
// tokens of one adapter: 62 us of 95).  Here tiles of rows come into LDS in whole lines, four waves'
// worth at once, and fragments from there; pieces change places by their row so that eight lanes'
// reads meet different banks.

// Sixteen-byte piece `piece` of row `row` in a tile whose rows are PR pieces: its place in the row.
template <int PR>
__device__ __forceinline__ int placed(int row, int piece) {
  return piece ^ (PR >= 16 ? row & 15 : PR == 8 ? row & 7 : row >> 1 & 3);
}

typedef __attribute__((address_space(1))) const void* global_ptr_t;

// h of a tile and a slice of K, 128 deep stages of it in LDS, two of them.  A wave takes 32 tokens and half
// of a stage's depth.
template <class E, int RT>
__global__ __launch_bounds__(64 * kWaves, 2) void lora_shrink_tiles_kernel(const LoraArgs a, int turns,
                                                                           int slices) {
  constexpr int kRows = kTile + 16 * RT, kStage = kRows * 256;  // x's rows, then the adapter's
  constexpr int kLoads = kRows / 4 / kWaves;                    // four rows each
  static_assert(kRows % (4 * kWaves) == 0, "whole loads");
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, p = lane >> 4;
  const int slice = blockIdx.x % slices, turn = blockIdx.x / slices;
  const int64_t t0 = (int64_t)blockIdx.y * kTile;
  const int groups = a.K / 128;
  const int g0 = (int)((int64_t)groups * slice / slices), g1 = (int)((int64_t)groups * (slice + 1) / slices);
  const int id = adapter_of(a, t0, lane);
  each_adapter(id, turn, turns, [&](int cur, uint64_t members) {
    const int rank = a.ranks ? min(max(0, a.ranks[cur]), a.R) : a.R;
    const int tiles = (rank + 15) / 16, n = __builtin_popcountll(members);
    const int list = members_list(members, lane);
    // the rows that this wave stages, four a load: lane / 16 of them, piece lane % 16
    const uint16_t* from[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = (i * kWaves + wave) * 4 + p, piece = placed<16>(row, c);
      const int token = __builtin_amdgcn_ds_bpermute((row < n ? row : 0) << 2, list);
      from[i] = (row < kTile ? a.x + (t0 + token) * a.x_st
                             : a.a + ((int64_t)cur * a.R + min(row - kTile, a.R - 1)) * a.K) +
                piece * 8;
    }
    auto stage = [&](int g, int slot) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int row = (i * kWaves + wave) * 4;
        if (row < kTile && row >= (n + 15) / 16 * 16) continue;  // (no token's)
        __builtin_amdgcn_global_load_lds((global_ptr_t)(from[i] + g * 128),
                                         (lds_ptr_t)(lds + slot * kStage + row * 256), 16, 0, 0);
      }
    };
    f32x4 h[2][RT] = {};
    const int first = wave >> 1 << 5, half = wave & 1;  // the wave's tokens, its half of a stage
    if (g0 < g1) stage(g0, 0);
    for (int g = g0; g < g1; ++g) {
      wait_vm<0>();
      lds_barrier();  // the stage has come, and the one before has been read
      const int slot = g - g0 & 1;
      if (g + 1 < g1) stage(g + 1, slot ^ 1);
      const char* at = lds + slot * kStage;
      if (first >= n) continue;
      auto fragment = [&](int row, int step) {
        return *reinterpret_cast<const u32x4*>(at + row * 256 + placed<16>(row, half * 8 + step * 4 + p) * 16);
      };
#pragma unroll
      for (int step = 0; step < 2; ++step) {
        const u32x4 x0 = fragment(first + c, step), x1 = fragment(first + 16 + c, step);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const u32x4 w = fragment(kTile + 16 * i + c, step);
          h[0][i] = E::mfma(w, x0, h[0][i]);
          h[1][i] = E::mfma(w, x1, h[1][i]);
        }
      }
    }
    // the two halves of the depth
    f32x4* sums = reinterpret_cast<f32x4*>(lds) + (wave >> 1) * (2 * RT * 64) + lane;
    lds_barrier();
    if (half == 1)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < RT; ++i) sums[(j * RT + i) * 64] = h[j][i];
    lds_barrier();
    if (half == 0)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int column = first + 16 * j + c;
        const int token = __builtin_amdgcn_ds_bpermute((column < n ? column : 0) << 2, list);
        if (column >= n) continue;
        float* to = a.h + ((int64_t)slice * a.T + t0 + token) * (16 * RT) + 4 * p;
#pragma unroll
        for (int i = 0; i < RT; ++i)
          if (i < tiles) *reinterpret_cast<f32x4*>(to + 16 * i) = h[j][i] + sums[(j * RT + i) * 64];
      }
    lds_barrier();  // the sums have been read
  });
}

// out of a tile and a block of its columns, 128 at a time: B's rows in LDS, two such units of them.  A wave
// takes 16 tokens, as the MFMAs' rows; column c of tile i is n = 8 c + i, so that a lane has eight
// consecutive n of four tokens, and 16 lanes 256 bytes of each.
template <class E, int RT>
__global__ __launch_bounds__(64 * kWaves, RT > 4 ? 2 : 3) void lora_expand_tiles_kernel(const LoraArgs a, int turns,
                                                                           int blocks, int slices) {
  constexpr int KS = (RT + 1) / 2, PR = 4 * KS, kStage = 128 * PR * 16;
  constexpr int kLoads = kStage / 1024 / kWaves;
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, p = lane >> 4;
  const int block = blockIdx.x % blocks, turn = blockIdx.x / blocks;
  const int64_t t0 = (int64_t)blockIdx.y * kTile;
  const int units = (a.N + 127) / 128;
  const int unit0 = (int)((int64_t)units * block / blocks);
  const int unit1 = (int)((int64_t)units * (block + 1) / blocks);
  const int id = adapter_of(a, t0, lane);
  if (turn == 0 && a.out != a.y) {  // tokens without an adapter
    const uint64_t rows = __ballot(id < 0 && t0 + lane < a.T);
    copy_rows(a, t0, rows, 128 * unit0, min(128 * unit1, a.N), lane, wave);
  }
  if (unit0 >= unit1) return;
  each_adapter(id, turn, turns, [&](int cur, uint64_t members) {
    const int rank = a.ranks ? min(max(0, a.ranks[cur]), a.R) : a.R;
    const float by = a.scales ? a.scales[cur] : 1.0f;
    const int n_members = __builtin_popcountll(members);
    const int list = members_list(members, lane);
    const bool works = 16 * wave < n_members;
    int token[4];  // of the lane's four rows; where there is none, the first
    bool in[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = 16 * wave + 4 * p + k;
      in[k] = row < n_members;
      token[k] = __builtin_amdgcn_ds_bpermute((in[k] ? row : 0) << 2, list);
    }
    const uint16_t* w = a.b + (int64_t)cur * a.N * a.R;
    auto stage = [&](int unit) {  // row 16 i + c of the stage is n = 8 c + i
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int at = (wave * kLoads + i) * 64 + lane, row = at / PR, piece = placed<PR>(row, at % PR);
        const int64_t n = min(128 * unit + 8 * (row & 15) + (row >> 4), a.N - 1);
        __builtin_amdgcn_global_load_lds((global_ptr_t)(w + n * a.R + (8 * piece < rank ? 8 * piece : 0)),
                                         (lds_ptr_t)(lds + (unit & 1) * kStage + (wave * kLoads + i) * 1024),
                                         16, 0, 0);
      }
    };
    u32x4 y[4], then[4];
    auto load = [&](u32x4 (&to)[4], int unit) {
      const int n = min(128 * unit + 8 * c, a.N - 8);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        to[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(a.y + (t0 + token[k]) * a.y_st + n));
    };
    stage(unit0);
    load(y, unit0);

    // h of the lane's token c as the first factor: two parts each of its eight of every 32, and the power
    // of 2 that is taken off again, of the tokens that the lane ends up with
    u32x4 hi[KS], lo[KS];
    int down[4];
    {
      const int column = 16 * wave + c;
      const int mine = __builtin_amdgcn_ds_bpermute((column < n_members ? column : 0) << 2, list);
      int at[KS];
#pragma unroll
      for (int s = 0; s < KS; ++s) at[s] = 32 * s + 8 * p < rank ? 32 * s + 8 * p : 0;
      f32x4 sum[KS][2] = {};
      if (works) sum_slices<KS>(a.h + (t0 + mine) * (16 * RT), at, a.T * (16 * RT), 0, 1, slices, sum);
      float h[KS][8];
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) h[s][e] = 32 * s + 8 * p + e < rank ? sum[s][e >> 2][e & 3] * by : 0.0f;
      const int up = power_of<E, KS>(h);
      two_parts<E, KS>(h, up, hi, lo);
#pragma unroll
      for (int k = 0; k < 4; ++k) down[k] = -__builtin_amdgcn_ds_bpermute((4 * p + k) << 2, up);
    }
    wait_vm<0>();
    lds_barrier();
    for (int unit = unit0; unit < unit1; ++unit) {
      const bool more = unit + 1 < unit1;
      if (more) stage(unit + 1);
      load(then, more ? unit + 1 : unit);
      u32x4 out[4];
      if (works) {
        const char* at = lds + (unit & 1) * kStage;
        f32x4 o[8];
        auto multiply = [&](auto once_more) __attribute__((always_inline)) {
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = f32x4{};
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            if (32 * s >= rank) break;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int row = 16 * i + c;
              u32x4 f = *reinterpret_cast<const u32x4*>(at + (row * PR + placed<PR>(row, 4 * s + p)) * 16);
              if (32 * s + 32 > rank)  // what an adapter's rows hold past its rank does not matter
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int r = 32 * s + 8 * p + 2 * e;
                  f[e] &= (r < rank ? 0xFFFFu : 0u) | (r + 1 < rank ? 0xFFFF0000u : 0u);
                }
              o[i] = E::mfma(hi[s], f, o[i]);
              if constexpr (decltype(once_more)::value) f = finite<E>(f);
              o[i] = E::mfma(lo[s], f, o[i]);
            }
          }
        };
        multiply(std::false_type{});
        if (__builtin_expect(any_nan(o), 0)) multiply(std::true_type{});
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const uint32_t was = y[k][i >> 1];
            const float v0 = E::value((uint16_t)(was & 0xFFFFu)) + __builtin_amdgcn_ldexpf(o[i][k], down[k]);
            const float v1 = E::value((uint16_t)(was >> 16)) + __builtin_amdgcn_ldexpf(o[i + 1][k], down[k]);
            out[k][i >> 1] = E::bits(v0) | (uint32_t)E::bits(v1) << 16;
          }
      }
      // (the next unit has come; the stores behind are waited for a unit later)
      wait_vm<0>();
      if (works) {
        const int n = 128 * unit + 8 * c;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (in[k] && n < a.N)
            __builtin_nontemporal_store(out[k], reinterpret_cast<u32x4*>(a.out + (t0 + token[k]) * a.out_st + n));
      }
      lds_barrier();  // this unit has been read, by every wave, and the next one is there
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = then[k];
    }
  });
}

namespace {

struct Layout {
  int row_tiles, tiles, turns, slices, blocks;
  bool join, staged;
};

Layout layout_of(int64_t T, int64_t N, int64_t K, int64_t R, int64_t L) {
  Layout p;
  const int64_t need = (R + 15) / 16;
  p.row_tiles = need <= 1 ? 1 : need <= 2 ? 2 : need <= 4 ? 4 : need <= 8 ? 8 : 16;
  p.tiles = (int)((T + kTile - 1) / kTile);
  const int64_t cu = device_cu_count();
  auto within = [](int64_t v, int64_t low, int64_t high) { return (int)std::max(low, std::min(v, high)); };
  // Workgroups for each adapter of a decoding step's tile, where many may occur (as many as the pool has:
  // 64 tokens over 40 adapters 28.6 us, with workgroups for 64 that 35.2); prompts' tiles hold few, which
  // one workgroup takes after the other.
  p.turns = within(p.tiles == 1 ? L : std::min(L, cu / (4 * p.tiles)), 1, std::min<int64_t>(T, kTile));
  const int64_t adapters = p.tiles == 1 ? p.turns : 1;  // at once
  // Whole lines through LDS pay where a tile's tokens share an adapter: prompts 72 us against 95 straight
  // from memory, with 128 ranks 95 against 194.  One tile is faster without (64 tokens over 40:
  // 31.5 against 28.6; one token 10.1 against 8.7), and a stage of 256 ranks does not fit twice.
  p.staged = p.tiles > 1 && p.row_tiles <= 8;
  // h: workgroups for two a compute unit (prompts 22.0 us, for one 26.7; 64 tokens over 40 alike, 28.6 and
  // 28.8).  With 72 to 128 ranks, whose stages take 96 KB, one is there at a time and the second follows: 1200
  // tokens 15.9 us, for one 17.2, 3500 tokens alike.  Of out's columns for prompts as many as a compute unit
  // holds: three (3500 tokens 44.1 us, for four 45.8), two above 64 ranks (1200 tokens of 128 ranks 25.8 us, for
  // four 30.9); and three in decoding steps, which pay for each with another sum of h's slices (64 tokens:
  // 15.5 us; four 17.3, two 16.3).
  p.slices = within(2 * cu / (p.tiles * adapters), 1, std::min<int64_t>(K / 128, 16));
  p.blocks = p.staged ? within((p.row_tiles > 4 ? 2 : 3) * cu / p.tiles, 1, (N + 127) / 128)
                      : within(3 * cu / (p.tiles * adapters), 1, (N + 255) / 256);
  // A few tiles may hold single tokens of many adapters as well as prompts: a quarter of both (200 tokens
  // over 37 adapters 41 us, 63 with all; a prompt of 116 tokens 18.9 and 22.4).
  if (p.staged && p.tiles < 8) {
    p.slices = std::max(1, p.slices / 4);
    p.blocks = std::max(1, p.blocks / 4);
  }
  // Every block sums h's slices, or a launch before does once: prompts 72 us against 77.5, fewer tiles than
  // eight without it (a launch is 3 us).
  p.join = p.slices > 1 && p.tiles >= 8;
  if (L == 0) {  // no adapter is loaded: there is no h and no workspace for one, and out is y
    p.turns = p.slices = 1;
    p.join = false;
  }
  return p;
}

hipError_t launch_slices_join(const LoraArgs& a, const Layout& p, hipStream_t stream) {
  const int64_t quads = a.T * (4 * p.row_tiles);
  return launch_kernel(lora_join_kernel, dim3((unsigned)((quads + 255) / 256)), dim3(256), stream, a.h,
                       quads, p.slices);
}

template <class E, int RT>
hipError_t launch_tiles(const LoraArgs& a, const Layout& p, hipStream_t stream) {
  hipError_t e = hipSuccess;
  if (a.L > 0)
    e = launch_kernel_lds(lora_shrink_tiles_kernel<E, RT>,
                          dim3((unsigned)(p.turns * p.slices), (unsigned)p.tiles), dim3(64 * kWaves),
                          2 * (kTile + 16 * RT) * 256, stream, a, p.turns, p.slices);
  if (e == hipSuccess && p.join) e = launch_slices_join(a, p, stream);
  if (e != hipSuccess) return e;
  return launch_kernel_lds(lora_expand_tiles_kernel<E, RT>,
                           dim3((unsigned)(p.turns * p.blocks), (unsigned)p.tiles), dim3(64 * kWaves),
                           2 * 128 * 64 * ((RT + 1) / 2), stream, a, p.turns, p.blocks,
                           p.join ? 1 : p.slices);
}

template <class E, int RT>
hipError_t launch(const LoraArgs& a, const Layout& p, hipStream_t stream) {
  if constexpr (RT <= 8)
    if (p.staged) return launch_tiles<E, RT>(a, p, stream);
  hipError_t e = hipSuccess;
  if (a.L > 0)
    e = launch_kernel(lora_shrink_kernel<E, RT>,
                      dim3((unsigned)(p.turns * p.slices), (unsigned)p.tiles), dim3(64 * kWaves),
                      stream, a, p.turns, p.slices);
  if (e == hipSuccess && p.join) e = launch_slices_join(a, p, stream);
  if (e != hipSuccess) return e;
  return launch_kernel(lora_expand_kernel<E, RT>,
                       dim3((unsigned)(p.turns * p.blocks), (unsigned)p.tiles), dim3(64 * kWaves),
                       stream, a, p.turns, p.blocks, p.join ? 1 : p.slices);
}

template <class E>
hipError_t launch_rank(const LoraArgs& a, const Layout& p, hipStream_t stream) {
  switch (p.row_tiles) {
    case 1: return launch<E, 1>(a, p, stream);
    case 2: return launch<E, 2>(a, p, stream);
    case 4: return launch<E, 4>(a, p, stream);
    case 8: return launch<E, 8>(a, p, stream);
    default: return launch<E, 16>(a, p, stream);
  }
}

}  // namespace

size_t lora_workspace_bytes(int64_t T, int64_t N, int64_t K, int64_t R, int64_t L) {
  const Layout p = layout_of(T, N, K, R, L);
  return (size_t)p.slices * T * (16 * p.row_tiles) * sizeof(float);
}

hipError_t launch_lora(const LoraArgs& a, bool bf16, hipStream_t stream) {
  if (a.L == 0 && a.out == a.y) return hipSuccess;
  const Layout p = layout_of(a.T, a.N, a.K, a.R, a.L);
  return bf16 ? launch_rank<Bfloat>(a, p, stream) : launch_rank<Half>(a, p, stream);
}

}  // namespace flexq
