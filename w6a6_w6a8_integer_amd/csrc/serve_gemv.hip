// serve_gemv.hip -- products of a few activation rows with 4-bit group-scaled weights,
// and the packing of those weights.
//
// Y[m][n] = sum_g s[g][n] * sum_{k in g} x[m][k] q[n][k].  A 16-bit activation times a
// code in [-8, 7] is exact in fp32, so the MFMA sums a group's products without an
// earlier rounding and the scale is applied once per group in fp32.
#include "kernels.h"
#include "serve_device.h"
#include "serve_kernels.h"

namespace flexq {

namespace {

// dword of row n, column k = 128 kb + 32 j + 8 p (+ c)
__device__ __forceinline__ int64_t w4_dword(int64_t n, int kb, int j, int p, int64_t kbs) {
  return ((n >> 4) * kbs + kb) * 256 + (p * 16 + (n & 15)) * 4 + j;
}

}  // namespace

// One thread = 8 consecutive codes (one dword); the G / 8 threads of a group are adjacent
// lanes.  blockIdx.x = row, blockIdx.y = chunk of 2048 columns.
template <class E, int G>
__global__ __launch_bounds__(256) void pack_w4_kernel(const uint16_t* __restrict__ w, int N,
                                                      int K, uint32_t* __restrict__ w4,
                                                      uint16_t* __restrict__ sw) {
  const int64_t n = blockIdx.x;
  const int k0 = (blockIdx.y * 256 + threadIdx.x) * 8;
  if (k0 >= K) return;  // whole 16-lane rows drop out together (K % 128 == 0)
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

// One workgroup = one 16-row tile of the weight x up to 16 NT activation rows; its W waves
// take the 128-deep k-blocks in turn and their sums are added in wave order at the end.
// D of the MFMA: column = activation row, rows = weight rows 4 (lane / 16) + i.
template <class E, int G, int NT, int W>
__global__ __launch_bounds__(64 * W) void gemv_w4_kernel(
    const uint16_t* __restrict__ x, int64_t x_stride, const uint32_t* __restrict__ w4,
    const uint16_t* __restrict__ sw, int M, int N, int K, uint16_t* __restrict__ y) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 15, p = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int m0 = blockIdx.y * 64;
  const int kbs = K >> 7;
  const u32x4* wt = reinterpret_cast<const u32x4*>(w4) + blockIdx.x * (int64_t)kbs * 64 + lane;
  f32x4 acc[NT] = {};
  for (int kb = wave; kb < kbs; kb += W) {
    const u32x4 d = wt[(int64_t)kb * 64];
#pragma unroll
    for (int g = 0; g < 128 / G; ++g) {
      const uint16_t* sp = sw + (int64_t)(kb * (128 / G) + g) * N + n0 + 4 * p;
      f32x4 dot[NT] = {};
#pragma unroll
      for (int jj = 0; jj < G / 32; ++jj) {
        const int j = g * (G / 32) + jj;
        u32x4 a;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int lo = (int)((d[j] >> (4 * i)) & 15u) - 8;
          const int hi = (int)((d[j] >> (4 * i + 16)) & 15u) - 8;
          a[i] = E::bits((float)lo) | (uint32_t)E::bits((float)hi) << 16;
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int m = m0 + t * 16 + c;
          u32x4 b = {};
          if (m < M)
            b = *reinterpret_cast<const u32x4*>(x + m * x_stride + kb * 128 + j * 32 + p * 8);
          dot[t] = E::mfma(a, b, dot[t]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float s = half_bits_to_float(sp[i]);
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t][i] = fmaf(s, dot[t][i], acc[t][i]);
      }
    }
  }
  __shared__ f32x4 part[W][NT][64];
#pragma unroll
  for (int t = 0; t < NT; ++t) part[wave][t][lane] = acc[t];
  __syncthreads();
  for (int t = wave; t < NT; t += W) {
    f32x4 s = part[0][t][lane];
#pragma unroll
    for (int v = 1; v < W; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] += part[v][t][lane][i];
    const int m = m0 + t * 16 + c;
    if (m < M) {
      u32x2 o;
      o[0] = E::bits(s[0]) | (uint32_t)E::bits(s[1]) << 16;
      o[1] = E::bits(s[2]) | (uint32_t)E::bits(s[3]) << 16;
      *reinterpret_cast<u32x2*>(y + (int64_t)m * N + n0 + 4 * p) = o;
    }
  }
}

namespace {

template <class E>
hipError_t pack_any(const uint16_t* w, int64_t N, int64_t K, int group, uint32_t* w4,
                    uint16_t* sw, hipStream_t stream) {
  const dim3 grid((unsigned)N, (unsigned)((K + 2047) / 2048));
  auto* kernel = group == 32   ? pack_w4_kernel<E, 32>
                 : group == 64 ? pack_w4_kernel<E, 64>
                               : pack_w4_kernel<E, 128>;
  return launch_kernel(kernel, grid, dim3(256), stream, w, (int)N, (int)K, w4, sw);
}

template <class E, int G>
hipError_t gemv_any(const uint16_t* x, int64_t x_stride, const uint32_t* w4, const uint16_t* sw,
                    int64_t M, int64_t N, int64_t K, uint16_t* y, hipStream_t stream) {
  constexpr int W = 4;
  const int64_t rows = M < 64 ? M : 64;
  const dim3 grid((unsigned)(N / 16), (unsigned)((M + 63) / 64));
  auto* kernel = rows <= 16   ? gemv_w4_kernel<E, G, 1, W>
                 : rows <= 32 ? gemv_w4_kernel<E, G, 2, W>
                              : gemv_w4_kernel<E, G, 4, W>;
  return launch_kernel(kernel, grid, dim3(64 * W), stream, x, x_stride, w4, sw, (int)M, (int)N,
                       (int)K, y);
}

template <class E>
hipError_t gemv_group(const uint16_t* x, int64_t x_stride, const uint32_t* w4,
                      const uint16_t* sw, int64_t M, int64_t N, int64_t K, int group, uint16_t* y,
                      hipStream_t stream) {
  if (group == 32) return gemv_any<E, 32>(x, x_stride, w4, sw, M, N, K, y, stream);
  if (group == 64) return gemv_any<E, 64>(x, x_stride, w4, sw, M, N, K, y, stream);
  return gemv_any<E, 128>(x, x_stride, w4, sw, M, N, K, y, stream);
}

}  // namespace

hipError_t launch_pack_w4(const uint16_t* w, bool bf16, int64_t N, int64_t K, int group,
                          uint32_t* w4, uint16_t* sw, hipStream_t stream) {
  return bf16 ? pack_any<Bfloat>(w, N, K, group, w4, sw, stream)
              : pack_any<Half>(w, N, K, group, w4, sw, stream);
}

hipError_t launch_gemv_w4(const uint16_t* x, bool bf16, int64_t x_stride, const uint32_t* w4,
                          const uint16_t* sw, int64_t M, int64_t N, int64_t K, int group,
                          uint16_t* y, hipStream_t stream) {
  return bf16 ? gemv_group<Bfloat>(x, x_stride, w4, sw, M, N, K, group, y, stream)
              : gemv_group<Half>(x, x_stride, w4, sw, M, N, K, group, y, stream);
}

}  // namespace flexq
