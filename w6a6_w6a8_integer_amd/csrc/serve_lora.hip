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
// h enters the second product as two 16-bit parts, after a power of two that takes a token's largest
// to 2^14 .. 2^15: within 2^-17 of itself, for fp16 2^-22 or 2^-39 of the largest.
#include <algorithm>

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

// The adapter of token t0 + lane, -1 where it has none.
__device__ __forceinline__ int adapter_of(const LoraArgs& a, int64_t t0, int lane) {
  const int id = t0 + lane < a.T ? a.adapters[t0 + lane] : -1;
  return id >= 0 && id < a.L ? id : -1;
}

// The tokens of one adapter in the tile, as this wave sees them: its 16 columns, if it has any, and
// which part of the other axis it takes.
struct Columns {
  int token;        // of the lane's column in the tile; where there is none, the first
  bool in;          // the column exists
  int parts, part;  // waves that share the columns, and which of them this is
  bool idle;
};

__device__ __forceinline__ Columns columns_of(uint64_t members, int lane, int wave) {
  const int n = __builtin_popcountll(members);
  const bool mine = members >> lane & 1;
  // lane i receives the i-th member (behind them the other tokens follow: every lane has a place)
  const int rank = __builtin_popcountll(members & ((1ull << lane) - 1));
  const int list = __builtin_amdgcn_ds_permute((mine ? rank : n + lane - rank) << 2, lane);
  Columns c;
  c.parts = n <= 16 ? 4 : n <= 32 ? 2 : 1;
  c.part = wave & (c.parts - 1);
  const int first = wave / c.parts * 16;
  const int column = first + (lane & 15);
  c.in = column < n;
  c.idle = first >= n;
  c.token = __builtin_amdgcn_ds_bpermute((c.in ? column : 0) << 2, list);
  return c;
}

// f(adapter, tokens that have it) for the adapters of the tile whose first token is turn modulo
// turns.
template <class F>
__device__ __forceinline__ void each_adapter(int id, int turn, int turns, F&& f) {
  const int lane = threadIdx.x & 63;
  uint64_t left = __ballot(id >= 0 && lane % turns == turn);
  while (left != 0) {
    const int first = __builtin_ctzll(left);
    const int cur = __builtin_amdgcn_readlane(id, first);
    const uint64_t members = __ballot(id == cur);
    if (__builtin_ctzll(members) == first) f(cur, members);
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
      const uint16_t* w = a.a + ((int64_t)cur * a.R) * a.K + at;
      int64_t row[RT];  // (rows past the adapter's last are read again, and not used)
#pragma unroll
      for (int i = 0; i < RT; ++i) row[i] = (int64_t)min(16 * i + c, a.R - 1) * a.K;
      constexpr int kUnroll = RT <= 2 ? 8 : RT == 4 ? 4 : 2;
      int k = 0;
      for (; k + 32 * kUnroll <= n; k += 32 * kUnroll) {
        u32x4 xf[kUnroll], wf[kUnroll][RT];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          xf[u] = *reinterpret_cast<const u32x4*>(x + k + 32 * u);
#pragma unroll
          for (int i = 0; i < RT; ++i)
            if (i < tiles) wf[u][i] = *reinterpret_cast<const u32x4*>(w + row[i] + k + 32 * u);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
          for (int i = 0; i < RT; ++i)
            if (i < tiles) h[i] = E::mfma(wf[u][i], xf[u], h[i]);
      }
      for (; k < n; k += 32) {
        const u32x4 xf = *reinterpret_cast<const u32x4*>(x + k);
#pragma unroll
        for (int i = 0; i < RT; ++i)
          if (i < tiles) h[i] = E::mfma(*reinterpret_cast<const u32x4*>(w + row[i] + k), xf, h[i]);
      }
    }
    if (col.parts > 1) {
      __syncthreads();  // the sums of the adapter before have been read
      if (col.part > 0)
#pragma unroll
        for (int i = 0; i < RT; ++i) sums[((wave - wave / col.parts - 1) * RT + i) * 64 + lane] = h[i];
      __syncthreads();
      if (col.part > 0) return;
      for (int q = 1; q < col.parts; ++q)
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const int from = wave + q;
          h[i] += sums[((from - from / col.parts - 1) * RT + i) * 64 + lane];
        }
    }
    if (!col.in) return;
    float* to = a.h + ((int64_t)slice * a.T + t0 + col.token) * (16 * RT) + 4 * p;
#pragma unroll
    for (int i = 0; i < RT; ++i)
      if (i < tiles) *reinterpret_cast<f32x4*>(to + 16 * i) = h[i];
  });
}

// out: one workgroup = a tile's adapters (those of its turn) and `units` times 64 columns of out for each
// wave that shares a token's.  Row r of the MFMA's 16-row tile i is n = 16 (r / 4) + 4 i + r % 4
// of 64, so that a lane ends up with 16 consecutive n of its token.
template <class E, int RT>
__global__ __launch_bounds__(64 * kWaves) void lora_expand_kernel(const LoraArgs a, int turns,
                                                                 int blocks, int slices) {
  constexpr int KS = (RT + 1) / 2;  // 32-deep steps over the rank
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
    const int n0 = 64 * unit0, n1 = min(64 * unit1, a.N);
    for (uint64_t left = __ballot(id < 0 && t0 + lane < a.T); left != 0; left &= left - 1) {
      const int64_t t = t0 + __builtin_ctzll(left);
      for (int n = n0 + 8 * (int)threadIdx.x; n < n1; n += 8 * 64 * kWaves)
        *reinterpret_cast<u32x4*>(a.out + t * a.out_st + n) =
            *reinterpret_cast<const u32x4*>(a.y + t * a.y_st + n);
    }
  }
  each_adapter(id, turn, turns, [&](int cur, uint64_t members) {
    const int rank = a.ranks ? min(max(0, a.ranks[cur]), a.R) : a.R;
    const float by = a.scales ? a.scales[cur] : 1.0f;
    const Columns col = columns_of(members, lane, wave);
    if (col.idle) return;
    const int64_t t = t0 + col.token;
    // this lane's eight of each 32 of h, scaled, their largest, and their two parts
    float h[KS][8];
    float most = 0.0f;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      f32x4 part[2] = {};
      const int r = 32 * s + 8 * p;
      if (r < rank) {
        const float* from = a.h + t * (16 * RT) + r;
        for (int q = 0; q < slices; ++q)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            part[j] += *reinterpret_cast<const f32x4*>(from + (int64_t)q * a.T * (16 * RT) + 4 * j);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[s][e] = r + e < rank ? part[e >> 2][e & 3] * by : 0.0f;
        most = fmaxf(most, fabsf(h[s][e]));
      }
    }
    most = column_max(most);
    const int up = 15 - __builtin_amdgcn_frexp_expf(most);
    u32x4 hi[KS], lo[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v0 = __builtin_amdgcn_ldexpf(h[s][2 * i], up);
        const float v1 = __builtin_amdgcn_ldexpf(h[s][2 * i + 1], up);
        const uint32_t b0 = E::bits(v0), b1 = E::bits(v1);
        // (an infinite or NaN h is its first part alone)
        const float r0 = v0 - E::value((uint16_t)b0), r1 = v1 - E::value((uint16_t)b1);
        hi[s][i] = b0 | b1 << 16;
        lo[s][i] = E::bits(fabsf(r0) < INFINITY ? r0 : 0.0f) |
                   (uint32_t)E::bits(fabsf(r1) < INFINITY ? r1 : 0.0f) << 16;
      }
    const uint16_t* w = a.b + (int64_t)cur * a.N * a.R;
    const int n_of = 16 * (c >> 2) + (c & 3);
    for (int unit = unit0 + col.part; unit < unit1; unit += col.parts) {
      const int n0 = 64 * unit;
      const int mine = n0 + 16 * p;  // the lane's 16 of out
      u32x4 y[2] = {};
      if (col.in && mine < a.N)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          y[j] = *reinterpret_cast<const u32x4*>(a.y + t * a.y_st + mine + 8 * j);
      f32x4 o[4] = {};
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int r = 32 * s + 8 * p;
        if (32 * s >= rank) break;
        u32x4 f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t n = min(n0 + n_of + 4 * i, a.N - 1);
          f[i] = r < rank ? *reinterpret_cast<const u32x4*>(w + n * a.R + r) : u32x4{};
        }
        if (32 * s + 32 > rank)  // what an adapter's rows hold past its rank does not matter
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t keep = (r + 2 * e < rank ? 0xFFFFu : 0u) | (r + 2 * e + 1 < rank ? 0xFFFF0000u : 0u);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i][e] &= keep;
          }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[i] = E::mfma(f[i], hi[s], o[i]);
          o[i] = E::mfma(f[i], lo[s], o[i]);
        }
      }
      if (!col.in || mine >= a.N) continue;
      u32x4 out[2];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          const uint32_t was = y[i >> 1][2 * (i & 1) + k / 2];
          const float v0 = E::value((uint16_t)(was & 0xFFFFu)) + __builtin_amdgcn_ldexpf(o[i][k], -up);
          const float v1 = E::value((uint16_t)(was >> 16)) + __builtin_amdgcn_ldexpf(o[i][k + 1], -up);
          out[i >> 1][2 * (i & 1) + k / 2] = E::bits(v0) | (uint32_t)E::bits(v1) << 16;
        }
#pragma unroll
      for (int j = 0; j < 2; ++j)
        *reinterpret_cast<u32x4*>(a.out + t * a.out_st + mine + 8 * j) = out[j];
    }
  });
}

namespace {

struct Layout {
  int row_tiles, tiles, turns, slices, blocks;
};

Layout layout_of(int64_t T, int64_t N, int64_t K, int64_t R, int64_t L) {
  Layout p;
  const int64_t need = (R + 15) / 16;
  p.row_tiles = need <= 1 ? 1 : need <= 2 ? 2 : need <= 4 ? 4 : need <= 8 ? 8 : 16;
  p.tiles = (int)((T + kTile - 1) / kTile);
  const int64_t target = 2 * device_cu_count();
  // a workgroup an adapter in one tile of a decoding step, where many may occur
  p.turns = (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(T, kTile),
                                                        8 * target / 16 / p.tiles));
  const int64_t adapters = std::max<int64_t>(1, std::min<int64_t>(L, p.turns));
  p.slices = (int)std::max<int64_t>(
      1, std::min<int64_t>(std::min<int64_t>(K / 128, 16), target / (p.tiles * adapters)));
  p.blocks = (int)std::max<int64_t>(
      1, std::min<int64_t>((N + 255) / 256, 2 * target / (p.tiles * adapters)));
  return p;
}

template <class E, int RT>
hipError_t launch(const LoraArgs& a, const Layout& p, hipStream_t stream) {
  const hipError_t e =
      launch_kernel(lora_shrink_kernel<E, RT>, dim3((unsigned)(p.turns * p.slices), (unsigned)p.tiles),
                    dim3(64 * kWaves), stream, a, p.turns, p.slices);
  if (e != hipSuccess) return e;
  return launch_kernel(lora_expand_kernel<E, RT>,
                       dim3((unsigned)(p.turns * p.blocks), (unsigned)p.tiles), dim3(64 * kWaves),
                       stream, a, p.turns, p.blocks, p.slices);
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
  const Layout p = layout_of(a.T, a.N, a.K, a.R, a.L);
  return bf16 ? launch_rank<Bfloat>(a, p, stream) : launch_rank<Half>(a, p, stream);
}

}  // namespace flexq
