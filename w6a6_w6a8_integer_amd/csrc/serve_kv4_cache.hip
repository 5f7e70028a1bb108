// serve_kv4_cache.hip -- new keys and values into the paged cache of 4-bit codes, and tokens of
// that cache back as 16-bit rows.
#include "kernels.h"
#include "serve_device.h"
#include "serve_kernels.h"

namespace flexq {

namespace {

constexpr int kThreads = 256;

// Threads that share a head row of D elements: two words of eight elements each, word `lane` and word
// `lane + kLanes` (of 96-wide rows the last four have one).
template <int D>
constexpr int kLanes = D == 64 ? 4 : D == 256 ? 16 : 8;

__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("v_min3_f32 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "v"(c));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "v"(c));
  return d;
}

template <int CTRL>
__device__ __forceinline__ float moved(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, false));
}
// smallest and largest over N neighbouring lanes: swap pairs, pairs of pairs, mirror 8, mirror 16
template <int N>
__device__ __forceinline__ void extremes(float& low, float& high) {
  low = fminf(low, moved<0xB1>(low)), high = fmaxf(high, moved<0xB1>(high));
  low = fminf(low, moved<0x4E>(low)), high = fmaxf(high, moved<0x4E>(high));
  if constexpr (N >= 8) low = fminf(low, moved<0x141>(low)), high = fmaxf(high, moved<0x141>(high));
  if constexpr (N >= 16) low = fminf(low, moved<0x140>(low)), high = fmaxf(high, moved<0x140>(high));
}

// x / 15 correctly rounded (the quotient by the rounded reciprocal, and its remainder added).
__device__ __forceinline__ float by_15(float x) {
  const float r = 1.0f / 15.0f, q = x * r;
  return fmaf(fmaf(-15.0f, q, x), r, q);
}

// A lane's two words of a row that N lanes share, as codes (element e of a word at bits 4 e); s and b
// receive the row's scale and offset as fp16.  A row that fp16 scales cannot hold (a NaN in it, or
// s or b not finite) gets NaN for both.  `some`: the second word is there.
//
// rint((x - b) / s): the quotient is first taken as q = (x - b) r with r = 1 / s to within a step, so
// q is within 2^-17 of the correctly rounded quotient where that is below 32 (beyond, both clamp).
// Where some q is that near to a rounding boundary (told with room, 2^-15: one wave in thirty)
// the quotients themselves are formed.  Adding 1.5 2^23 rounds q to a whole number in its low bits.
template <class E, int N>
__device__ __forceinline__ u32x2 quantize_row(const u32x4 (&v)[2], bool some, uint16_t& s, uint16_t& b) {
  float x[2][8];
  float low, high, finite = 0.0f;
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const uint32_t two = v[w][e >> 1];
      x[w][e] = E::value((uint16_t)(two & 0xFFFFu));
      x[w][e + 1] = E::value((uint16_t)(two >> 16));
    }
  low = high = x[0][0];
  finite = x[0][0] * 0.0f;
#pragma unroll
  for (int e = 1; e < 8; ++e) finite = fmaf(x[0][e], 0.0f, finite);
#pragma unroll
  for (int e = 1; e < 7; e += 2) {
    low = min3(low, x[0][e], x[0][e + 1]);
    high = max3(high, x[0][e], x[0][e + 1]);
  }
  low = fminf(low, x[0][7]), high = fmaxf(high, x[0][7]);
  if (some) {
#pragma unroll
    for (int e = 0; e < 8; ++e) finite = fmaf(x[1][e], 0.0f, finite);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      low = min3(low, x[1][e], x[1][e + 1]);
      high = max3(high, x[1][e], x[1][e + 1]);
    }
  }
  if (finite != 0.0f) high = INFINITY;  // (NaN: an infinity or a NaN was there)
  extremes<N>(low, high);
  b = Half::bits(low);
  s = Half::bits(by_15(high - low));
  if ((b & 0x7C00u) == 0x7C00u || (s & 0x7C00u) == 0x7C00u) b = s = 0x7E00u;
  const float sf = Half::value(s), bf = Half::value(b);
  if (!(sf > 0.0f)) return u32x2{0, 0};
  const float r = __builtin_amdgcn_rcpf(sf);
  constexpr float kRound = 12582912.0f;
  constexpr uint32_t kRounds = 0x4B400000u * 0x111u;  // its bits, eight times over (mod 2^32 three)
  u32x2 codes;
  float near = 0.0f;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint32_t sum = 0;
#pragma unroll
    for (int e = 7; e >= 0; --e) {
      const float q = __builtin_amdgcn_fmed3f((x[w][e] - bf) * r, 0.0f, 15.0f), m = q + kRound;
      near = fmaxf(near, fabsf(q - (m - kRound)));
      sum = (sum << 4) + __float_as_uint(m);
    }
    codes[w] = sum - kRounds;
  }
  if (near > 0.5f - 0x1p-15f) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint32_t sum = 0;
#pragma unroll
      for (int e = 7; e >= 0; --e) {
        const float q = __builtin_amdgcn_fmed3f((x[w][e] - bf) / sf, 0.0f, 15.0f);
        sum = (sum << 4) + __float_as_uint(q + kRound);
      }
      codes[w] = sum - kRounds;
    }
  }
  return codes;
}

// codes of elements e at bits 4 e -> at bits 4 (e / 2) + 16 (e % 2), the order of the keys' dwords
__device__ __forceinline__ uint32_t key_order(uint32_t w) {
  uint32_t even = w & 0x0F0F0F0Fu, odd = (w >> 4) & 0x0F0F0F0Fu;
  even = (even | even >> 4) & 0x00FF00FFu;
  odd = (odd | odd >> 4) & 0x00FF00FFu;
  even = (even | even >> 8) & 0xFFFFu;
  odd = (odd | odd >> 8) & 0xFFFFu;
  return even | odd << 16;
}
// and back
__device__ __forceinline__ uint32_t element_order(uint32_t w) {
  uint32_t even = w & 0xFFFFu, odd = w >> 16;
  even = (even | even << 8) & 0x00FF00FFu;
  odd = (odd | odd << 8) & 0x00FF00FFu;
  even = (even | even << 4) & 0x0F0F0F0Fu;
  odd = (odd | odd << 4) & 0x0F0F0F0Fu;
  return even | odd << 4;
}

// the byte of a value dword that token r % 4 has: 0, 2, 1, 3
__device__ __forceinline__ int byte_of(int r) { return (r >> 1 & 1) | (r & 1) << 1; }

}  // namespace

// Four dwords' bytes as four dwords of one byte of each, in the order 0, 2, 1, 3 of the tokens.
__device__ __forceinline__ void turn(const uint32_t (&c)[4], uint32_t (&o)[4]) {
  const uint32_t low02 = __builtin_amdgcn_perm(c[2], c[0], 0x05010400u);
  const uint32_t high02 = __builtin_amdgcn_perm(c[2], c[0], 0x07030602u);
  const uint32_t low13 = __builtin_amdgcn_perm(c[3], c[1], 0x05010400u);
  const uint32_t high13 = __builtin_amdgcn_perm(c[3], c[1], 0x07030602u);
  o[0] = __builtin_amdgcn_perm(low13, low02, 0x05040100u);
  o[1] = __builtin_amdgcn_perm(low13, low02, 0x07060302u);
  o[2] = __builtin_amdgcn_perm(high13, high02, 0x05040100u);
  o[3] = __builtin_amdgcn_perm(high13, high02, 0x07060302u);
}

// One workgroup = TOKENS tokens of one head.  kLanes lanes a row find its extremes and form its codes;
// the keys' go to the cache at once, the values' and the scales through LDS, where eight
// tokens of consecutive slots from a multiple of eight become whole 32-byte pieces of four pairs
// of d and 16-byte pieces of scales.  Other tokens are written byte by byte (scales half by half),
// so that no token's codes are read to write another's.  Prompts of 21 900 tokens of 8 heads of
// 128 take 32 us for 114 MB, 3.6 TB/s (a copy reaches 4.9): forming the codes, eleven operations an
// element, does not quite hide behind the loads.
template <class E, int D, int TOKENS>
__global__ __launch_bounds__(kThreads) void kv4_cache_write_kernel(
    const uint16_t* __restrict__ k, int64_t k_st, int64_t k_sh, const uint16_t* __restrict__ v,
    int64_t v_st, int64_t v_sh, const int* __restrict__ slots, int T, int Hkv, int64_t num_slots,
    int shift, uint32_t* __restrict__ kc, uint32_t* __restrict__ vc, uint16_t* __restrict__ sc) {
  constexpr int N = kLanes<D>, kWords = D / 8;
  __shared__ uint32_t tile[TOKENS * kWords];  // value codes, element e at bits 4 e
  __shared__ __attribute__((aligned(16))) uint16_t scales[4][TOKENS];
  __shared__ int slot_of[TOKENS + 8];         // -1 where a token is dropped
  __shared__ int eights[TOKENS / 8 + 1], singles[TOKENS];  // tokens that begin eight slots; alone
  __shared__ int num_eights, num_singles;
  static_assert(TOKENS <= 64, "one lane a token");
  const int h = blockIdx.y, t0 = blockIdx.x * TOKENS, tid = threadIdx.x;
  if (tid < TOKENS + 8) {
    const int64_t slot = tid < TOKENS && t0 + tid < T ? slots[t0 + tid] : -1;
    slot_of[tid] = slot >= 0 && slot < num_slots ? (int)slot : -1;
  }
  __syncthreads();
  // rows of this thread's turns: the keys, then the values
  const int lane = tid % N;
  const bool some = lane + N < kWords;
  constexpr int kTurns = 2 * TOKENS * N / kThreads > 0 ? 2 * TOKENS * N / kThreads : 1;
  u32x4 x[kTurns][2];
#pragma unroll
  for (int u = 0; u < kTurns; ++u) {
    const int row = tid / N + u * (kThreads / N), i = row % TOKENS;
    const bool value = row >= TOKENS;
    x[u][0] = x[u][1] = u32x4{};
    if (row < 2 * TOKENS && slot_of[i] >= 0) {
      const uint16_t* from = value ? v + (int64_t)(t0 + i) * v_st + h * v_sh
                                   : k + (int64_t)(t0 + i) * k_st + h * k_sh;
      x[u][0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(from + 8 * lane));
      if (some) x[u][1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(from + 8 * (lane + N)));
    }
  }
  if (tid < 64) {  // (while the rows are on their way)
    const int slot = tid < TOKENS ? slot_of[tid] : -1;
    bool leads = slot >= 0 && (slot & 7) == 0;
    for (int i = 1; leads && i < 8; ++i) leads = slot_of[tid + i] == slot + i;
    const uint64_t all = __ballot(leads);
    // alone: kept, and no token up to seven before begins eight that hold this one
    const bool alone = slot >= 0 && (all & (tid >= 7 ? 0xFFull << (tid - 7) : 0xFFull >> (7 - tid))) == 0;
    const uint64_t some_alone = __ballot(alone);
    const uint64_t below = (1ull << tid) - 1;
    if (leads) eights[__builtin_popcountll(all & below)] = tid;
    if (alone) singles[__builtin_popcountll(some_alone & below)] = tid;
    if (tid == 0) {
      num_eights = __builtin_popcountll(all);
      num_singles = __builtin_popcountll(some_alone);
    }
  }
  auto block_of = [&](int slot) {
    const int r = slot & ((1 << shift) - 1);
    return ((int64_t)(slot >> shift) * Hkv + h) * (1 << (shift - 4)) + (r >> 4);
  };
#pragma unroll
  for (int u = 0; u < kTurns; ++u) {
    const int row = tid / N + u * (kThreads / N), i = row % TOKENS;
    const bool value = row >= TOKENS;
    uint16_t s, b;
    const u32x2 codes = quantize_row<E, N>(x[u], some, s, b);
    const int slot = row < 2 * TOKENS ? slot_of[i] : -1;
    if (slot < 0) continue;
    if (lane == 0) {
      scales[value ? 2 : 0][i] = s;
      scales[value ? 3 : 1][i] = b;
    }
    if (value) {
      tile[i * kWords + lane] = codes[0];
      if (some) tile[i * kWords + lane + N] = codes[1];
    } else {
      uint32_t* to = kc + block_of(slot) * (2 * D) + (slot & 15) * kWords + lane;
      to[0] = key_order(codes[0]);
      if (some) to[N] = key_order(codes[1]);
    }
  }
  __syncthreads();
  for (int i = tid; i < num_eights * kWords; i += kThreads) {
    const int t = eights[i / kWords], w = i % kWords, slot = slot_of[t];
    uint32_t* const to = vc + block_of(slot) * (2 * D) + (slot >> 3 & 1) * D + 8 * w;
    uint32_t c[2][4], o[2][4];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
      for (int j = 0; j < 4; ++j) c[q][j] = tile[(t + 4 * q + j) * kWords + w];
      turn(c[q], o[q]);
    }
    reinterpret_cast<u32x4*>(to)[0] = u32x4{o[0][0], o[1][0], o[0][1], o[1][1]};
    reinterpret_cast<u32x4*>(to)[1] = u32x4{o[0][2], o[1][2], o[0][3], o[1][3]};
    if (w < 4) {
      u32x4 eight;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        eight[j] = scales[w][t + 2 * j] | (uint32_t)scales[w][t + 2 * j + 1] << 16;
      *reinterpret_cast<u32x4*>(sc + block_of(slot) * 64 + 16 * w + (slot & 8)) = eight;
    }
  }
  for (int i = tid; i < num_singles * kWords; i += kThreads) {
    const int t = singles[i / kWords], w = i % kWords, slot = slot_of[t];
    uint8_t* to = reinterpret_cast<uint8_t*>(vc + block_of(slot) * (2 * D) + (slot >> 3 & 1) * D + 8 * w +
                                             (slot >> 2 & 1)) + byte_of(slot);
    const uint32_t c = tile[t * kWords + w];
#pragma unroll
    for (int pair = 0; pair < 4; ++pair) to[8 * pair] = (uint8_t)(c >> (8 * pair));
    if (w < 4) sc[block_of(slot) * 64 + 16 * w + (slot & 15)] = scales[w][t];
  }
}

// A lane a word of eight elements of a token and head: x = b + s c, rounded once.  A token outside the
// cache reads as 0.  Few loads an element: the four scales are one load of four neighbouring lanes, and
// a word's value pairs come whole, with the four tokens that are not asked for (24 MB of codes to 90
// MB of rows: 29 us with a load for each scale and pair, 25 so).
template <class E, int D>
__global__ __launch_bounds__(kThreads) void kv4_cache_read_kernel(
    const uint32_t* __restrict__ kc, const uint32_t* __restrict__ vc,
    const uint16_t* __restrict__ sc, const int* __restrict__ slots, int64_t rows, int Hkv,
    int64_t num_slots, int shift, uint16_t* __restrict__ k, uint16_t* __restrict__ v) {
  constexpr int N = D == 96 ? 16 : D / 8, kWords = D / 8;
  const int lane = threadIdx.x % N;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / N) + threadIdx.x / N;  // (token, head)
  const bool in_rows = row < rows;
  const uint32_t token = in_rows ? (uint32_t)row / (uint32_t)Hkv : 0;
  const int h = (int)((uint32_t)row - token * Hkv);
  const int64_t slot = in_rows ? slots[token] : -1;
  const bool in = slot >= 0 && slot < num_slots;
  const int r = in ? (int)slot & ((1 << shift) - 1) : 0;
  const int64_t block = in ? ((slot >> shift) * Hkv + h) * (1 << (shift - 4)) + (r >> 4) : 0;
  uint32_t by = 0, kw = 0;
  u32x4 vw[2] = {};
  if (in) {
    by = sc[block * 64 + 16 * (lane & 3) + (r & 15)];
    const int w = lane < kWords ? lane : 0;
    kw = kc[block * (2 * D) + (r & 15) * kWords + w];
    const u32x4* from = reinterpret_cast<const u32x4*>(vc + block * (2 * D) + (r >> 3 & 1) * D + 8 * w);
    vw[0] = from[0];
    vw[1] = from[1];
  }
  // (every lane of four takes part)
  const float ks = Half::value((uint16_t)__builtin_amdgcn_update_dpp(0, (int)by, 0x00, 0xF, 0xF, false));
  const float kb = Half::value((uint16_t)__builtin_amdgcn_update_dpp(0, (int)by, 0x55, 0xF, 0xF, false));
  const float vs = Half::value((uint16_t)__builtin_amdgcn_update_dpp(0, (int)by, 0xAA, 0xF, 0xF, false));
  const float vb = Half::value((uint16_t)__builtin_amdgcn_update_dpp(0, (int)by, 0xFF, 0xF, 0xF, false));
  if (!in_rows || lane >= kWords) return;
  u32x4 ko = {}, vo = {};
  if (in) {
    kw = element_order(kw);
    const int at = 8 * byte_of(r), quad = r >> 2 & 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t pair = (quad ? vw[i >> 1][2 * (i & 1) + 1] : vw[i >> 1][2 * (i & 1)]) >> at;
      ko[i] = E::bits(fmaf(ks, (float)(kw >> (8 * i) & 15u), kb)) |
              (uint32_t)E::bits(fmaf(ks, (float)(kw >> (8 * i + 4) & 15u), kb)) << 16;
      vo[i] = E::bits(fmaf(vs, (float)(pair & 15u), vb)) |
              (uint32_t)E::bits(fmaf(vs, (float)(pair >> 4 & 15u), vb)) << 16;
    }
  }
  __builtin_nontemporal_store(ko, reinterpret_cast<u32x4*>(k + row * D + 8 * lane));
  __builtin_nontemporal_store(vo, reinterpret_cast<u32x4*>(v + row * D + 8 * lane));
}

namespace {

template <class E, int TOKENS>
auto* write_kernel(int64_t D) {
  return D == 64    ? kv4_cache_write_kernel<E, 64, TOKENS>
         : D == 96  ? kv4_cache_write_kernel<E, 96, TOKENS>
         : D == 128 ? kv4_cache_write_kernel<E, 128, TOKENS>
                    : kv4_cache_write_kernel<E, 256, TOKENS>;
}

template <class E>
auto* read_kernel(int64_t D) {
  return D == 64    ? kv4_cache_read_kernel<E, 64>
         : D == 96  ? kv4_cache_read_kernel<E, 96>
         : D == 128 ? kv4_cache_read_kernel<E, 128>
                    : kv4_cache_read_kernel<E, 256>;
}

}  // namespace

hipError_t launch_kv4_cache_write(const uint16_t* k, int64_t k_st, int64_t k_sh,
                                  const uint16_t* v, int64_t v_st, int64_t v_sh, bool bf16,
                                  const int32_t* slots, int64_t T, int64_t Hkv, int64_t D,
                                  int64_t num_pages, int page_size, uint32_t* kc, uint32_t* vc,
                                  uint16_t* scales, hipStream_t stream) {
  // 32 tokens a workgroup where there are four such for every compute unit (prompts of 21 900 tokens, 8
  // heads: 32.3 us, with 64 33.9; 16 tokens: 4.6 us)
  const int tokens = (T + 31) / 32 * Hkv >= 4 * device_cu_count() ? 32 : 16;
  const dim3 grid((unsigned)((T + tokens - 1) / tokens), (unsigned)Hkv);
  auto* kernel = tokens == 32 ? (bf16 ? write_kernel<Bfloat, 32>(D) : write_kernel<Half, 32>(D))
                              : (bf16 ? write_kernel<Bfloat, 16>(D) : write_kernel<Half, 16>(D));
  return launch_kernel(kernel, grid, dim3(kThreads), stream, k, k_st, k_sh, v, v_st, v_sh, slots,
                       (int)T, (int)Hkv, num_pages * page_size,
                       __builtin_ctz((unsigned)page_size), kc, vc, scales);
}

hipError_t launch_kv4_cache_read(const uint32_t* kc, const uint32_t* vc, const uint16_t* scales,
                                 const int32_t* slots, int64_t T, int64_t Hkv, int64_t D,
                                 int64_t num_pages, int page_size, bool bf16, uint16_t* k,
                                 uint16_t* v, hipStream_t stream) {
  const int64_t rows = T * Hkv, per = kThreads / (D == 96 ? 16 : D / 8);
  auto* kernel = bf16 ? read_kernel<Bfloat>(D) : read_kernel<Half>(D);
  return launch_kernel(kernel, dim3((unsigned)((rows + per - 1) / per)), dim3(kThreads), stream, kc,
                       vc, scales, slots, rows, (int)Hkv, num_pages * page_size,
                       __builtin_ctz((unsigned)page_size), k, v);
}

}  // namespace flexq
