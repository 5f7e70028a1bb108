// serve_kv4_cache.hip -- new keys and values into the paged cache of 4-bit codes, and tokens of
// that cache back as 16-bit rows.
#include "kernels.h"
#include "serve_device.h"
#include "serve_kernels.h"

namespace flexq {

namespace {

constexpr int kThreads = 256;

// Threads that share a head row of D elements, eight each (16 with four that have none for
// D = 96), all in one wave.
template <int D>
constexpr int kLanes = D == 96 ? 16 : D / 8;

// extremes over N neighbouring lanes
template <int N>
__device__ __forceinline__ float lanes_min(float x) {
#pragma unroll
  for (int o = 1; o < N; o *= 2) x = fminf(x, __shfl_xor(x, o));
  return x;
}
template <int N>
__device__ __forceinline__ float lanes_max(float x) {
#pragma unroll
  for (int o = 1; o < N; o *= 2) x = fmaxf(x, __shfl_xor(x, o));
  return x;
}

// rint((x - b) / s) clamped to 0 .. 15, s > 0, r = 1 / s.  The quotient is first taken as
// q = (x - b) r, within 2^-18 of the correctly rounded one where that is below 32 (beyond, both
// clamp); only where q is that near to a rounding boundary (told with room, 2^-15) is the
// quotient itself formed.
__device__ __forceinline__ uint32_t code_of(float x, float b, float s, float r) {
  const float d = x - b, q = d * r;
  float k = rintf(q);
  if (fabsf(fabsf(q - k) - 0.5f) < 0x1p-15f) k = rintf(d / s);
  return (uint32_t)fminf(fmaxf(k, 0.0f), 15.0f);
}

// A lane's eight elements of a row that N lanes share, as codes (element e at bits 4 e); s and b
// receive the row's scale and offset as fp16.  A row that fp16 scales cannot hold (a NaN in it, or
// s or b not finite) gets NaN for both.  Every lane of the row takes part; `some`: it has
// elements.
template <class E, int N>
__device__ __forceinline__ uint32_t quantize_row(const u32x4 v, bool some, uint16_t& s, uint16_t& b) {
  float x[8];
  float low = INFINITY, high = -INFINITY, nan = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] = E::value((uint16_t)(e & 1 ? v[e >> 1] >> 16 : v[e >> 1] & 0xFFFFu));
    if (some) {
      low = fminf(low, x[e]);
      high = fmaxf(high, x[e]);
      nan = x[e] != x[e] ? 1.0f : nan;
    }
  }
  low = lanes_min<N>(low);
  high = lanes_max<N>(high);
  nan = lanes_max<N>(nan);
  b = Half::bits(low);
  s = Half::bits((high - low) / 15.0f);
  if (nan != 0.0f || (b & 0x7C00u) == 0x7C00u || (s & 0x7C00u) == 0x7C00u) {
    b = s = 0x7E00u;
    return 0;
  }
  const float sf = Half::value(s), bf = Half::value(b);
  if (sf == 0.0f) return 0;
  const float r = 1.0f / sf;
  uint32_t codes = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) codes |= code_of(x[e], bf, sf, r) << (4 * e);
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

// One workgroup = TOKENS tokens of one head.  kLanes lanes a row find its extremes and form its codes;
// the keys' go to the cache at once, the values' through LDS, where eight tokens of consecutive
// slots from a multiple of eight become whole 32-byte pieces of four pairs of d.  Other
// tokens are written byte by byte, so that no token's codes are read to write another's.
template <class E, int D, int TOKENS>
__global__ __launch_bounds__(kThreads) void kv4_cache_write_kernel(
    const uint16_t* __restrict__ k, int64_t k_st, int64_t k_sh, const uint16_t* __restrict__ v,
    int64_t v_st, int64_t v_sh, const int* __restrict__ slots, int T, int Hkv, int64_t num_slots,
    int shift, uint32_t* __restrict__ kc, uint32_t* __restrict__ vc, uint16_t* __restrict__ sc) {
  constexpr int N = kLanes<D>, kWords = D / 8;
  __shared__ uint32_t tile[TOKENS * kWords];  // value codes, element e at bits 4 e
  __shared__ int slot_of[TOKENS + 8];         // -1 where a token is dropped
  __shared__ uint64_t led;                    // tokens that begin eight consecutive slots
  static_assert(TOKENS <= 64, "one bit a token");
  const int h = blockIdx.y, t0 = blockIdx.x * TOKENS, tid = threadIdx.x;
  if (tid < TOKENS + 8) {
    const int64_t slot = tid < TOKENS && t0 + tid < T ? slots[t0 + tid] : -1;
    slot_of[tid] = slot >= 0 && slot < num_slots ? (int)slot : -1;
  }
  __syncthreads();
  if (tid < 64) {
    bool leads = tid < TOKENS && slot_of[tid] >= 0 && (slot_of[tid] & 7) == 0;
    for (int i = 1; leads && i < 8; ++i) leads = slot_of[tid + i] == slot_of[tid] + i;
    const uint64_t all = __ballot(leads);
    if (tid == 0) led = all;
  }
  auto block_of = [&](int slot) {
    const int r = slot & ((1 << shift) - 1);
    return ((int64_t)(slot >> shift) * Hkv + h) * (1 << (shift - 4)) + (r >> 4);
  };
  // rows of this turn's lanes: the keys, then the values
  const int lane = tid % N;
  const bool some = lane < kWords;
  constexpr int kTurns = (2 * TOKENS * N + kThreads - 1) / kThreads;
  u32x4 x[kTurns];
#pragma unroll
  for (int u = 0; u < kTurns; ++u) {
    const int row = tid / N + u * (kThreads / N), i = row % TOKENS;
    const bool value = row >= TOKENS;
    x[u] = u32x4{};
    if (row < 2 * TOKENS && some && slot_of[i] >= 0) {
      const uint16_t* from = value ? v + (int64_t)(t0 + i) * v_st + h * v_sh
                                   : k + (int64_t)(t0 + i) * k_st + h * k_sh;
      x[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(from + 8 * lane));
    }
  }
#pragma unroll
  for (int u = 0; u < kTurns; ++u) {
    const int row = tid / N + u * (kThreads / N), i = row % TOKENS;
    const bool value = row >= TOKENS;
    uint16_t s, b;
    const uint32_t codes = quantize_row<E, N>(x[u], some, s, b);
    const int slot = row < 2 * TOKENS ? slot_of[i] : -1;
    if (slot < 0) continue;
    const int64_t block = block_of(slot);
    const int r = slot & 15;
    if (lane == 0) {
      uint16_t* to = sc + block * 64 + (value ? 32 : 0) + r;
      to[0] = s;
      to[16] = b;
    }
    if (!some) continue;
    if (value)
      tile[i * kWords + lane] = codes;
    else
      kc[block * (2 * D) + r * kWords + lane] = key_order(codes);
  }
  __syncthreads();
  const uint64_t leads = led;
  for (int i = tid; i < TOKENS * kWords; i += kThreads) {
    const int t = i / kWords, w = i % kWords;
    const int slot = slot_of[t];
    if (slot < 0) continue;
    // whether a token up to seven before leads eight that hold this one
    if ((leads >> t & 1) != 0) {
      uint32_t c[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = tile[(t + j) * kWords + w];
      u32x4 out[2];
#pragma unroll
      for (int pair = 0; pair < 4; ++pair)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t o = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            o |= (c[4 * q + j] >> (8 * pair) & 0xFFu) << (8 * (j >> 1 | (j & 1) << 1));
          out[pair >> 1][2 * (pair & 1) + q] = o;
        }
      u32x4* to = reinterpret_cast<u32x4*>(vc + block_of(slot) * (2 * D) + (slot >> 3 & 1) * D + 8 * w);
      to[0] = out[0];
      to[1] = out[1];
    } else if ((leads & (t >= 7 ? 0x7Full << (t - 7) : 0x7Full >> (7 - t))) == 0) {
      uint8_t* to = reinterpret_cast<uint8_t*>(vc + block_of(slot) * (2 * D) + (slot >> 3 & 1) * D +
                                               8 * w + (slot >> 2 & 1)) +
                    byte_of(slot);
      const uint32_t c = tile[t * kWords + w];
#pragma unroll
      for (int pair = 0; pair < 4; ++pair) to[8 * pair] = (uint8_t)(c >> (8 * pair));
    }
  }
}

// kLanes lanes a token and head: x = b + s c, rounded once.  A token outside the cache reads as 0.
template <class E, int D>
__global__ __launch_bounds__(kThreads) void kv4_cache_read_kernel(
    const uint32_t* __restrict__ kc, const uint32_t* __restrict__ vc,
    const uint16_t* __restrict__ sc, const int* __restrict__ slots, int64_t rows, int Hkv,
    int64_t num_slots, int shift, uint16_t* __restrict__ k, uint16_t* __restrict__ v) {
  constexpr int N = kLanes<D>, kWords = D / 8;
  const int lane = threadIdx.x % N;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / N) + threadIdx.x / N;  // (token, head)
  if (row >= rows || lane >= kWords) return;
  const int h = (int)(row % Hkv);
  const int64_t slot = slots[row / Hkv];
  u32x4 ko = {}, vo = {};
  if (slot >= 0 && slot < num_slots) {
    const int r = (int)slot & ((1 << shift) - 1);
    const int64_t block = ((slot >> shift) * Hkv + h) * (1 << (shift - 4)) + (r >> 4);
    const uint16_t* by = sc + block * 64 + (r & 15);
    const float ks = Half::value(by[0]), kb = Half::value(by[16]);
    const float vs = Half::value(by[32]), vb = Half::value(by[48]);
    const uint32_t kw = element_order(kc[block * (2 * D) + (r & 15) * kWords + lane]);
    const uint32_t* from = vc + block * (2 * D) + (r >> 3 & 1) * D + 8 * lane + (r >> 2 & 1);
    uint32_t vw = 0;
#pragma unroll
    for (int pair = 0; pair < 4; ++pair)
      vw |= (from[2 * pair] >> (8 * byte_of(r)) & 0xFFu) << (8 * pair);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ko[i] = E::bits(fmaf(ks, (float)(kw >> (8 * i) & 15u), kb)) |
              (uint32_t)E::bits(fmaf(ks, (float)(kw >> (8 * i + 4) & 15u), kb)) << 16;
      vo[i] = E::bits(fmaf(vs, (float)(vw >> (8 * i) & 15u), vb)) |
              (uint32_t)E::bits(fmaf(vs, (float)(vw >> (8 * i + 4) & 15u), vb)) << 16;
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
  const int tokens = (T + 63) / 64 * Hkv >= 2 * device_cu_count() ? 64 : 16;
  const dim3 grid((unsigned)((T + tokens - 1) / tokens), (unsigned)Hkv);
  auto* kernel = tokens == 64 ? (bf16 ? write_kernel<Bfloat, 64>(D) : write_kernel<Half, 64>(D))
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
