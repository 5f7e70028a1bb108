// serve_gemv.hip -- products of a few activation rows with 4-bit group-scaled weights,
// and the packing of those weights.
//
// Y[m][n] = sum_g s[g][n] * sum_{k in g} x[m][k] q[n][k].  A 16-bit activation times a
// code in [-8, 7] is exact in fp32, so the MFMA sums a group's products without an
// earlier rounding and the scale is applied once per group in fp32.
#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "serve_device.h"
#include "serve_kernels.h"

namespace flexq {

namespace {

constexpr uint32_t kRsrcWord3 = 0x00020000u;  // raw 32-bit dword buffer, gfx9 style

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes,
                                           kRsrcWord3);
}

// 16 bytes a lane from memory to LDS: lane l's at `to` + 16 l, zeros past the buffer.
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t from, char* to, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_ptr_t)to, 16, off, 0, 0, 0);
}

// dword of row n, column k = 128 kb + 32 j + 8 p (+ c)
__device__ __forceinline__ int64_t w4_dword(int64_t n, int kb, int j, int p, int64_t kbs) {
  return ((n >> 4) * kbs + kb) * 256 + (p * 16 + (n & 15)) * 4 + j;
}

}  // namespace

// One thread = 8 consecutive codes (one dword); the G / 8 threads of a group are adjacent
// lanes.  blockIdx.x = row (and those gridDim.x apart), blockIdx.y = chunk of 2048 columns.
template <class E, int G>
__global__ __launch_bounds__(256) void pack_w4_kernel(const uint16_t* __restrict__ w, int N,
                                                      int K, uint32_t* __restrict__ w4,
                                                      uint16_t* __restrict__ sw) {
  const int k0 = (blockIdx.y * 256 + threadIdx.x) * 8;
  if (k0 >= K) return;  // whole 16-lane rows drop out together (K % 128 == 0)
  for (int64_t n = blockIdx.x; n < N; n += gridDim.x) {
    const u32x4 h = *reinterpret_cast<const u32x4*>(w + n * K + k0);
    float v[8];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = E::value((uint16_t)(h[i] & 0xFFFFu));
      v[2 * i + 1] = E::value((uint16_t)(h[i] >> 16));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
    for (int o = 1; o < G / 8; o *= 2) amax = fmaxf(amax, __shfl_xor(amax, o));
    const uint16_t s16 = float_to_half_bits(amax / 7.0f);
    const float s = half_bits_to_float(s16);
    uint32_t d = 0;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float r = s != 0.0f ? fminf(fmaxf(rintf(v[c] / s), -7.0f), 7.0f) : 0.0f;
      d |= (uint32_t)((int)r + 8) << (4 * (c >> 1) + 16 * (c & 1));
    }
    w4[w4_dword(n, k0 >> 7, (k0 >> 5) & 3, (k0 >> 3) & 3, K >> 7)] = d;
    if ((k0 & (G - 1)) == 0) sw[(int64_t)(k0 / G) * N + n] = s16;
  }
}

// Both kernels below are bound by HBM (0.5 byte a weight) where the weight is large: one row
// of 57344 x 8192 takes 41 us, 5.9 TB/s, in bfloat16, whose codes take more to convert, 47.
// Smaller weights are latency (4096 x 4096: 5 us, a launch and one load after the other), more
// rows the LDS reads of x and the MFMAs (64 rows of 57344 x 8192: 78 us, 770 TFLOP/s).
//
// Eight codes as the MFMA's 16-bit floats of their own values, so that a sum errs in
// proportion to what it adds: a large activation whose code is 0 adds 0, also where it is
// infinite only NaN, as the definition has it.
template <class E>
struct Codes;

// u = q + 8 as the low mantissa bits of 1024 + u or, four bits further up, 1024 + 16 u; then one
// packed add or fma: nine operations for eight codes.  The constants are held in registers so
// that a pair's bits take one and-or.
template <>
struct Codes<Half> {
  typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
  static constexpr float kScale = 1.0f;  // what the value is still to be multiplied by
  uint32_t low = 0x000F000Fu, high = 0x00F000F0u, base = 0x64006400u;
  __device__ __forceinline__ Codes() {
    asm("" : "+s"(low));
    asm("" : "+s"(high));
    asm("" : "+v"(base));
  }
  __device__ __forceinline__ u32x4 operator()(uint32_t d) const {
    const f16x2 minus1032 = {(_Float16)-1032.0f, (_Float16)-1032.0f};
    const f16x2 by = {(_Float16)0.0625f, (_Float16)0.0625f};
    const f16x2 minus72 = {(_Float16)-72.0f, (_Float16)-72.0f};
    u32x4 a;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t bits = ((i < 2 ? d : d >> 8) & (i % 2 ? high : low)) | base;
      const f16x2 v = __builtin_bit_cast(f16x2, bits);
      a[i] = __builtin_bit_cast(
          uint32_t, i % 2 ? __builtin_elementwise_fma(v, by, minus72) : v + minus1032);
    }
    return a;
  }
};

// Two's complement codes (q + 8 with the top bit turned) go through the conversion that makes
// q / 16 of four bits; packing two is exact.  Fourteen operations for eight codes.
template <>
struct Codes<Bfloat> {
  static constexpr float kScale = 16.0f;
  __device__ __forceinline__ u32x4 operator()(uint32_t d) const {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const uint32_t even = d ^ 0x88888888u;
    uint32_t odd = even >> 4;  // codes in the low halves of the bytes, which the
    asm("" : "+v"(odd));       // conversion can take by itself
    u32x4 a;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t from = i % 2 ? odd : even;
      const f32x2 v = {__builtin_amdgcn_cvt_off_f32_i4((int)((from >> (8 * (i / 2))) & 255u)),
                       __builtin_amdgcn_cvt_off_f32_i4((int)((from >> (8 * (i / 2) + 16)) & 255u))};
      a[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
    }
    return a;
  }
};

// acc += scale * dot, four consecutive weight rows
__device__ __forceinline__ void scale_add(f32x4& acc, f32x4 dot, u32x2 scales) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    acc[i] = fmaf(half_bits_to_float((uint16_t)(scales[i >> 1] >> (16 * (i & 1)))), dot[i], acc[i]);
}

// A k-block's scales of a tile in one load: lane (c, p) has those of rows 4 p to 4 p + 3 and
// group c % (128 / G); group g's are those of lane g of each four.
template <int kGroups>
__device__ __forceinline__ u32x2 group_scales(u32x2 s, int g) {
  if constexpr (kGroups == 1) return s;
  auto of = [&](auto lane) {
    constexpr int kSame = decltype(lane)::value * 0x55;  // that lane's value in all four
    return u32x2{(uint32_t)__builtin_amdgcn_mov_dpp((int)s[0], kSame, 15, 15, true),
                 (uint32_t)__builtin_amdgcn_mov_dpp((int)s[1], kSame, 15, 15, true)};
  };
  switch (g) {
    case 0: return of(std::integral_constant<int, 0>{});
    case 1: return of(std::integral_constant<int, 1>{});
    case 2: return of(std::integral_constant<int, 2>{});
    default: return of(std::integral_constant<int, 3>{});
  }
}

template <class E>
__device__ __forceinline__ void store_four(uint16_t* to, f32x4 v) {
  u32x2 o;
  o[0] = E::bits(v[0]) | (uint32_t)E::bits(v[1]) << 16;
  o[1] = E::bits(v[2]) | (uint32_t)E::bits(v[3]) << 16;
  *reinterpret_cast<u32x2*>(to) = o;
}

// Up to four rows.  A persistent workgroup owns a run of 16-row tiles of the weight, its W
// waves take the 128-deep k-blocks of a tile in turn (1 KB in one piece each), and the waves'
// sums are added in wave order through LDS.  P steps of loads are in flight, on into the next
// tile.
//
// All loads are buffer loads and no branch is around one, so that the waits count exactly
// the steps in flight.  The addresses only ever grow by constants (the scalar unit is
// shared by all waves: address arithmetic was what bound an earlier form).  A step past K
// loads some other weights and zero scales, one past the run nothing that is used.
//
// The activations are in LDS, rows K + 32 elements apart, so that only the weights and
// scales take registers in flight; lanes without a row read the last one's (their columns
// are not stored).
template <class E, int G, int W, int P>
__global__ __launch_bounds__(64 * W, 4) void gemv_w4_kernel(
    const uint16_t* __restrict__ x, int64_t x_stride, const uint32_t* __restrict__ w4,
    const uint16_t* __restrict__ sw, int M, int N, int K, int tiles, uint16_t* __restrict__ y) {
  constexpr int kGroups = 128 / G;  // of a k-block
  constexpr int kSteps = G / 32;    // MFMAs of a group
  extern __shared__ __attribute__((aligned(16))) uint16_t lds_x[];
  __shared__ f32x4 part[2][W][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, p = lane >> 4;
  const int kbs = K >> 7;
  const int rounds = (kbs + W - 1) / W;
  const int first = (int)((int64_t)tiles * blockIdx.x / gridDim.x);
  const int last = (int)((int64_t)tiles * (blockIdx.x + 1) / gridDim.x);

  struct Slot {
    u32x4 w;
    u32x2 s;
  } ring[P];

  // Loads of one wave step: k-block kb of a tile, which the offsets stand for.
  const int64_t run = (int64_t)first * kbs * 1024;
  const auto rw = make_rsrc(reinterpret_cast<const char*>(w4) + run,
                            (uint32_t)((int64_t)last * kbs * 1024 - run));
  const auto rs = make_rsrc(sw + first * 16,
                            (uint32_t)((int64_t)(K / G) * N * 2 - (int64_t)first * 32));
  int kb = wave;
  uint32_t w_off = wave * 1024 + lane * 16;
  uint32_t s_tile = (uint32_t)(wave * kGroups + c % kGroups) * (N * 2) + 8 * p;
  uint32_t s_off = s_tile;
  auto next_load = [&](Slot& r) {
    r.w = __builtin_bit_cast(
        u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, w_off, 0, kNonTemporal));
    r.s = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rs, s_off, 0, 0));
    kb += W;
    w_off += W * 1024;
    s_off += W * kGroups * (N * 2);
    if (kb >= rounds * W) {  // the next tile
      kb = wave;
      w_off += (kbs - rounds * W) * 1024;
      s_tile += 32;
      s_off = s_tile;
    }
  };

  const Codes<E> codes;
  const uint16_t* lds_row = lds_x + min(c, M - 1) * (K + 32) + p * 8;
  const uint16_t* lds_zeros = lds_x + M * (K + 32) + p * 8;

  f32x4 acc = {};
  auto work = [&](const Slot& r, int round) {
    const int kb_now = round * W + wave;  // past K zeros: other activations may be infinite
    const uint16_t* at = kb_now < kbs ? lds_row + kb_now * 128 : lds_zeros;
    u32x4 xf[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) xf[j] = *reinterpret_cast<const u32x4*>(at + j * 32);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      f32x4 dot = {};
#pragma unroll
      for (int j = g * kSteps; j < (g + 1) * kSteps; ++j)
        dot = E::mfma(codes(r.w[j]), xf[j], dot);
      scale_add(acc, dot, group_scales<kGroups>(r.s, g));
    }
  };

  // the waves' sums, in order
  auto finish = [&](int tile) {
    f32x4(*to)[64] = part[tile & 1];
    to[wave][lane] = acc;
    acc = f32x4{};
    lds_barrier();  // (the next tile's sums go to the other half)
    if ((wave + tile) % W != 0) return;
    f32x4 s = to[0][lane];
#pragma unroll
    for (int v = 1; v < W; ++v) {
      const f32x4 o = to[v][lane];
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] += o[k];
    }
    if (c < M) store_four<E>(y + (int64_t)c * N + tile * 16 + 4 * p, s * Codes<E>::kScale);
  };

  const int pieces = K / 8;  // 16 bytes each
  for (int i = threadIdx.x; i < M * pieces; i += 64 * W) {
    const int row = i / pieces, k8 = i % pieces;
    *reinterpret_cast<u32x4*>(lds_x + row * (K + 32) + k8 * 8) =
        *reinterpret_cast<const u32x4*>(x + row * x_stride + k8 * 8);
  }
  if (threadIdx.x < 16) *reinterpret_cast<u32x4*>(lds_x + M * (K + 32) + threadIdx.x * 8) = u32x4{};
#pragma unroll
  for (int i = 0; i < P; ++i) {
    next_load(ring[i]);
    __builtin_amdgcn_sched_barrier(0);  // the waits count on the steps' order
  }
  lds_barrier();  // the activations are there
  int tile = first, round = 0;
  const int steps = (last - first) * rounds;
  for (int step = 0; tile < last; step += P) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (step + i >= steps) break;
      work(ring[i], round);
      __builtin_amdgcn_sched_barrier(0);
      next_load(ring[i]);
      __builtin_amdgcn_sched_barrier(0);
      if (++round == rounds) {
        finish(tile);
        round = 0;
        ++tile;
      }
    }
  }
}

// More rows: a product of 128 T weight rows (T tiles for each of eight waves) and 16 NT rows
// of x over a slice of K.  A few k-blocks of x at a time go to LDS, straight from memory and
// shared by the waves; each wave streams its own weights into registers.  Both are two
// chunks ahead.  Where the weight has too few rows to fill the GPU, K is cut into slices
// whose fp32 sums go to part [slice][M][N], and join_slices_kernel adds them in order.
//
// In LDS a kilobyte block holds eight rows x 128 bytes, loaded as eight whole cache lines;
// the 16-byte pieces are placed so that the 16 lanes of a fragment read (16 rows, one
// piece each) meet 16 different banks: piece k of row r at slot 8 (r ^ h) + (k ^ r), h the
// block's parity.
// k-blocks of a chunk (up to 16 rows, with four: 13 x 5120 x 13824 15.4 us against 13.7, 16 x
// 57344 x 8192 50.8 against 49.1)
constexpr int kChunk = 2;

template <class E, int G, int NT, int T>
__global__ __launch_bounds__(512, NT <= 2 ? 4 : 2) void gemm_w4_kernel(
    const uint16_t* __restrict__ x, int64_t x_stride, const uint32_t* __restrict__ w4,
    const uint16_t* __restrict__ sw, int M, int N, int K, int tiles, int slices,
    float* __restrict__ part, uint16_t* __restrict__ y) {
  constexpr int kGroups = 128 / G, kSteps = G / 32;
  constexpr int kBlocks = 2 * NT;                      // of eight rows
  constexpr int kBytes = kChunk * 2 * kBlocks * 1024;  // of x a chunk
  constexpr int kMine = kChunk * kBlocks / 4;          // kilobytes of it a wave stages
  constexpr int kAhead = 2;
  constexpr uint32_t kNowhere = 0x80000000u;
  __shared__ __attribute__((aligned(1024))) char lds[(kAhead + 1) * kBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, p = lane >> 4;
  const int m0 = blockIdx.y * 64;
  const int kbs = K >> 7, chunks = (kbs + kChunk - 1) / kChunk;
  const int slice = blockIdx.x % slices;
  const int tile0 = (blockIdx.x / slices * 8 + wave) * T;
  const int first = (int)((int64_t)chunks * slice / slices);
  const int last = (int)((int64_t)chunks * (slice + 1) / slices);
  const int rows = min(M - m0, 16 * NT);
  const uint16_t* x0 = x + (int64_t)m0 * x_stride;

  // x: this wave's k-block of a chunk, half of it, and blocks; the lane's row and piece
  const int at = wave * kMine;
  const int my_kb = at / (2 * kBlocks), my_half = at / kBlocks % 2, my_block = at % kBlocks;
  const uint32_t x_bytes = (uint32_t)((rows - 1) * x_stride + K) * 2u;
  uint32_t x_off[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int b = my_block + i;
    const int row8 = (lane >> 3) ^ (b & 1), piece = (lane & 7) ^ row8, row = b * 8 + row8;
    x_off[i] = row < rows ? (uint32_t)(row * x_stride) * 2u + my_half * 128u + piece * 16u
                          : kNowhere;
  }
  auto stage = [&](int chunk) {
    const int kb = chunk * kChunk + my_kb;
    const auto rx = make_rsrc(x0, kb < kbs && chunk < last ? x_bytes : 0u);
    char* to = lds + chunk % (kAhead + 1) * kBytes + at * 1024;
#pragma unroll
    for (int i = 0; i < kMine; ++i)  // (no row: past the buffer still with K added)
      load_to_lds(rx, to + i * 1024, x_off[i] + kb * 256u);
  };

  struct Chunk {
    u32x4 w[kChunk][T];
    u32x2 s[kChunk][T];
  } ring[kAhead];
  const char* w0 = reinterpret_cast<const char*>(w4) + (int64_t)tile0 * kbs * 1024;
  const uint32_t w_bytes = (uint32_t)(max(0, min(T, tiles - tile0)) * kbs) * 1024u;
  const uint32_t s_bytes =
      tile0 < tiles ? (uint32_t)((int64_t)(K / G) * N * 2 - (int64_t)tile0 * 32) : 0u;
  auto load = [&](Chunk& r, int chunk) {
    // (one tile: past K is past the buffer; more: the scales are zero there)
    const auto rw = make_rsrc(w0, chunk < last ? w_bytes : 0u);
    const auto rs = make_rsrc(sw + tile0 * 16, chunk < last ? s_bytes : 0u);
    const uint32_t w_off = chunk * (kChunk * 1024) + lane * 16;
    const uint32_t s_off = (uint32_t)(chunk * (kChunk * kGroups) + c % kGroups) * (N * 2) + 8 * p;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
#pragma unroll
      for (int t = 0; t < T; ++t)
        r.w[i][t] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                  rw, w_off + t * (kbs * 1024) + i * 1024, 0,
                                                  kNonTemporal));
#pragma unroll
      for (int t = 0; t < T; ++t)
        r.s[i][t] = __builtin_bit_cast(
            u32x2, __builtin_amdgcn_raw_buffer_load_b64(
                       rs, s_off + (uint32_t)i * kGroups * (N * 2) + t * 32, 0, 0));
    }
  };

  const Codes<E> codes;
  const int row8 = c & 7, h = c >> 3;
  const int frag_row = h * 1024 + ((row8 ^ h) * 8) * 16;
  f32x4 acc[T][NT] = {};
  auto work = [&](const Chunk& r, int chunk) {
    const char* from = lds + chunk % (kAhead + 1) * kBytes;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        f32x4 dot[T][NT] = {};
#pragma unroll
        for (int j = g * kSteps; j < (g + 1) * kSteps; ++j) {
          u32x4 xf[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n)
            xf[n] = *reinterpret_cast<const u32x4*>(
                from + ((i * 2 + (j >> 1)) * kBlocks + 2 * n) * 1024 + frag_row +
                ((((j & 1) * 4 + p) ^ row8) * 16));
#pragma unroll
          for (int t = 0; t < T; ++t) {
            const u32x4 a = codes(r.w[i][t][j]);
#pragma unroll
            for (int n = 0; n < NT; ++n) dot[t][n] = E::mfma(a, xf[n], dot[t][n]);
          }
        }
#pragma unroll
        for (int t = 0; t < T; ++t) {
          const u32x2 scales = group_scales<kGroups>(r.s[i][t], g);
#pragma unroll
          for (int n = 0; n < NT; ++n) scale_add(acc[t][n], dot[t][n], scales);
        }
      }
    }
  };

  // A chunk's loads: kMine of x, then the weights' and scales'.  Those of chunks past the
  // slice are issued too (the waits count on them) but go nowhere.
  constexpr int kLoads = kMine + kChunk * T * 2;
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    stage(first + i);
    __builtin_amdgcn_sched_barrier(0);
    load(ring[i], first + i);
    __builtin_amdgcn_sched_barrier(0);
  }
  for (int chunk = first; chunk < last; chunk += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      // this wave's part of the chunk has come, then everyone's, and the one before is read
      wait_vm<(kAhead - 1) * kLoads>();
      lds_barrier();
      __builtin_amdgcn_sched_barrier(0);
      stage(chunk + i + kAhead);
      __builtin_amdgcn_sched_barrier(0);
      if (chunk + i < last) work(ring[i], chunk + i);
      __builtin_amdgcn_sched_barrier(0);
      load(ring[i], chunk + i + kAhead);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

#pragma unroll
  for (int t = 0; t < T; ++t) {
    const int tile = tile0 + t;
    if (tile >= tiles) continue;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (n * 16 + c >= rows) continue;
      const int64_t at = (int64_t)(m0 + n * 16 + c) * N + tile * 16 + 4 * p;
      if (slices > 1)
        *reinterpret_cast<f32x4*>(part + (int64_t)slice * M * N + at) = acc[t][n];
      else
        store_four<E>(y + at, acc[t][n] * Codes<E>::kScale);
    }
  }
}

// y = the slices' sums, added in order
template <class E>
__global__ __launch_bounds__(256) void join_slices_kernel(const float* __restrict__ part,
                                                          int64_t quads, int slices,
                                                          uint16_t* __restrict__ y) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= quads) return;
  const f32x4* from = reinterpret_cast<const f32x4*>(part) + i;
  f32x4 s = {};
  for (int v0 = 0; v0 < slices; v0 += 8) {
    f32x4 o[8];  // eight loads at a time
#pragma unroll
    for (int v = 0; v < 8; ++v) o[v] = v0 + v < slices ? from[(v0 + v) * quads] : f32x4{};
#pragma unroll
    for (int v = 0; v < 8; ++v)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] += o[v][k];
  }
  store_four<E>(y + 4 * i, s * Codes<E>::kScale);
}

namespace {

template <class E>
hipError_t pack_any(const uint16_t* w, int64_t N, int64_t K, int group, uint32_t* w4,
                    uint16_t* sw, hipStream_t stream) {
  // (a launch holds fewer than 2^32 threads in a direction)
  const dim3 grid((unsigned)std::min<int64_t>(N, 1 << 23), (unsigned)((K + 2047) / 2048));
  auto* kernel = group == 32   ? pack_w4_kernel<E, 32>
                 : group == 64 ? pack_w4_kernel<E, 64>
                               : pack_w4_kernel<E, 128>;
  return launch_kernel(kernel, grid, dim3(256), stream, w, (int)N, (int)K, w4, sw);
}

// The few-rows kernel, for activations that every workgroup can hold in LDS.  One row of 4096 x 4096 takes 5.4 us with it and 7.8 with
// the other, of 10240 x 8192 11.0 and 13.0, of 57344 x 8192 41 and 47; four of 5120 x 5120 (groups
// of 32) 9.1 and 8.7; one of 8192 x 28672, past the bound on LDS, 25.5 and 24.3.
int64_t x_lds_bytes(int64_t M, int64_t K) { return (M * (K + 32) + 128) * 2; }
bool few_rows(int64_t M, int64_t K) { return M <= 4 && x_lds_bytes(M, K) <= 48 * 1024; }

// The other one: tiles a wave, and slices of K that give every compute unit a workgroup.
// Twice the slices only add sums to join (13 x 5120 x 13824: 15.4 us against 13.7; 64 x 8192 x
// 8192: 31 against 21), half of them leave compute units idle (20 and 28).
struct Cut {
  int tiles_a_wave, slices;
};

Cut cut_of(int64_t M, int64_t N, int64_t K) {
  Cut cut;
  // With more than 32 rows of x its reads from LDS bound a wave; two tiles share them where
  // one tile a wave would take the compute units twice (64 rows, K = 8192: N = 40960 66 us
  // against 86, 57344 78 against 94, 131072 167 against 200; but 8192, 24 against 21, and 48 x
  // 22016 x 4096 29 against 24).
  cut.tiles_a_wave = M > 32 && N / 16 > 8 * device_cu_count() ? 2 : 1;
  const int64_t per = 8 * cut.tiles_a_wave;
  const int64_t units = (N / 16 + per - 1) / per * ((M + 63) / 64);
  const int64_t chunks = (K / 128 + kChunk - 1) / kChunk;
  const int64_t target = device_cu_count();
  cut.slices = (int)std::clamp<int64_t>(target / units, 1, std::min<int64_t>(chunks, 16));
  return cut;
}

template <class E, int G>
hipError_t gemv_launch(const uint16_t* x, int64_t x_stride, const uint32_t* w4,
                       const uint16_t* sw, int64_t M, int64_t N, int64_t K, uint16_t* y,
                       hipStream_t stream) {
  constexpr int W = 8, P = 4;
  const int64_t tiles = N / 16, cus = device_cu_count();
  const int64_t x_bytes = x_lds_bytes(M, K);
  // Two workgroups a compute unit, or three if registers and LDS hold them and the last round
  // of tiles is fuller for it (10240 x 8192, 640 tiles: 11.0 us against 12.3; but 14336 x
  // 4096, 896 tiles: 8.5 against 8.1).  (Two tiles at a time share x's fragments and leave the
  // workgroups' shares less even: 32768 x 4096 14.4 us against 13.6, 57344 x 8192 43.5 against
  // 41.4, 131072 x 4096 46.8 against 47.6.)
  auto cost = [&](int64_t held) { return (tiles + held * cus - 1) / (held * cus) * held; };
  const int64_t held = x_bytes <= 32 * 1024 && cost(3) < cost(2) ? 3 : 2;
  return launch_kernel_lds(gemv_w4_kernel<E, G, W, P>,
                           dim3((unsigned)std::min(tiles, held * cus)), dim3(64 * W), x_bytes,
                           stream, x, x_stride, w4, sw, (int)M, (int)N, (int)K, (int)tiles, y);
}

template <class E, int G, int NT, int T>
hipError_t gemm_launch(const uint16_t* x, int64_t x_stride, const uint32_t* w4,
                       const uint16_t* sw, int64_t M, int64_t N, int64_t K, float* part,
                       uint16_t* y, hipStream_t stream) {
  const Cut cut = cut_of(M, N, K);
  const int64_t tiles = N / 16;
  const dim3 grid((unsigned)((tiles + 8 * T - 1) / (8 * T) * cut.slices),
                  (unsigned)((M + 63) / 64));
  const hipError_t e =
      launch_kernel(gemm_w4_kernel<E, G, NT, T>, grid, dim3(512), stream, x, x_stride, w4, sw,
                    (int)M, (int)N, (int)K, (int)tiles, cut.slices, part, y);
  if (e != hipSuccess || cut.slices == 1) return e;
  const int64_t quads = M * N / 4;
  return launch_kernel(join_slices_kernel<E>, dim3((unsigned)((quads + 255) / 256)), dim3(256),
                       stream, part, quads, cut.slices, y);
}

template <class E, int G>
hipError_t gemv_any(const uint16_t* x, int64_t x_stride, const uint32_t* w4, const uint16_t* sw,
                    int64_t M, int64_t N, int64_t K, float* part, uint16_t* y,
                    hipStream_t stream) {
  if (few_rows(M, K)) return gemv_launch<E, G>(x, x_stride, w4, sw, M, N, K, y, stream);
  if (M <= 16) return gemm_launch<E, G, 1, 1>(x, x_stride, w4, sw, M, N, K, part, y, stream);
  if (M <= 32) return gemm_launch<E, G, 2, 1>(x, x_stride, w4, sw, M, N, K, part, y, stream);
  if (cut_of(M, N, K).tiles_a_wave == 1)
    return gemm_launch<E, G, 4, 1>(x, x_stride, w4, sw, M, N, K, part, y, stream);
  return gemm_launch<E, G, 4, 2>(x, x_stride, w4, sw, M, N, K, part, y, stream);
}

template <class E>
hipError_t gemv_group(const uint16_t* x, int64_t x_stride, const uint32_t* w4,
                      const uint16_t* sw, int64_t M, int64_t N, int64_t K, int group, float* part,
                      uint16_t* y, hipStream_t stream) {
  if (group == 32) return gemv_any<E, 32>(x, x_stride, w4, sw, M, N, K, part, y, stream);
  if (group == 64) return gemv_any<E, 64>(x, x_stride, w4, sw, M, N, K, part, y, stream);
  return gemv_any<E, 128>(x, x_stride, w4, sw, M, N, K, part, y, stream);
}

}  // namespace

size_t gemv_w4_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (few_rows(M, K)) return 0;
  const int slices = cut_of(M, N, K).slices;
  return slices == 1 ? 0 : (size_t)slices * M * N * sizeof(float);
}

hipError_t launch_pack_w4(const uint16_t* w, bool bf16, int64_t N, int64_t K, int group,
                          uint32_t* w4, uint16_t* sw, hipStream_t stream) {
  return bf16 ? pack_any<Bfloat>(w, N, K, group, w4, sw, stream)
              : pack_any<Half>(w, N, K, group, w4, sw, stream);
}

hipError_t launch_gemv_w4(const uint16_t* x, bool bf16, int64_t x_stride, const uint32_t* w4,
                          const uint16_t* sw, int64_t M, int64_t N, int64_t K, int group,
                          void* workspace, uint16_t* y, hipStream_t stream) {
  float* part = static_cast<float*>(workspace);
  return bf16 ? gemv_group<Bfloat>(x, x_stride, w4, sw, M, N, K, group, part, y, stream)
              : gemv_group<Half>(x, x_stride, w4, sw, M, N, K, group, part, y, stream);
}

}  // namespace flexq
