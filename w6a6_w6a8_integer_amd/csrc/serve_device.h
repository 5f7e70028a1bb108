// serve_device.h -- gfx950 device helpers of the decoding-step kernels: 16-bit element
// types and their MFMAs, waits and barriers.
#pragma once
#include "w6_device.h"

namespace flexq {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kNonTemporal = 2;  // cache-policy bit of loads

typedef __attribute__((address_space(3))) void* lds_ptr_t;

// s_waitcnt vmcnt(N) alone (gfx9 encoding: vmcnt[3:0], expcnt[6:4], lgkmcnt[11:8],
// vmcnt[5:4] in [15:14]).
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

// A barrier that the wave's own LDS accesses have come before (a stage may be overwritten
// behind it).  Loads from memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// 16x16x32 MFMA on 16-bit elements: lane l supplies A row l % 16 and B column l % 16, the
// eight elements of k-slots 8 (l / 16) ..; D lane l holds column l % 16, rows
// 4 (l / 16) + 0 .. 3, in fp32.  A and B agree on what k each slot stands for; the
// kernels use that freedom to take fragments in the order memory holds them.
//
// 32x32x16: row and column l % 32, k-slots 8 (l / 32) ..; D lane l holds column l % 32 and, in
// register r, row 8 (r / 4) + 4 (l / 32) + r % 4.
struct Half {
  static __device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint16_t bits(float f) { return float_to_half_bits(f); }
  static __device__ __forceinline__ float value(uint16_t h) { return half_bits_to_float(h); }
  // Two fp32 values in [0, 2^15] each as the sum of two halves: cut, then what was cut off.  The
  // sum is less than 2^-20 of the value, or 2^-24 (half's least step), below it.
  static __device__ __forceinline__ u32x2 split(float x, float y) {
    const auto h = __builtin_amdgcn_cvt_pkrtz(x, y);
    const auto l = __builtin_amdgcn_cvt_pkrtz(fmaf(-(float)h[0], 1.0f, x), fmaf(-(float)h[1], 1.0f, y));
    return u32x2{__builtin_bit_cast(uint32_t, h), __builtin_bit_cast(uint32_t, l)};
  }
  static constexpr uint32_t kExponent = 0x7C00u;  // all ones: infinity or NaN
  static constexpr uint32_t kOne = 0x3C00u;
  // A row's largest probability is held as 2^(kTop - 1) to 2^(kTop + kLag): half's range reaches
  // no further up, and down to 2^-24, so that small ones keep their bits.
  static constexpr float kTop = 11.0f, kLag = 4.0f;
};

struct Bfloat {
  static __device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint16_t bits(float f) {
    return __builtin_bit_cast(uint16_t, (__bf16)f);
  }
  static __device__ __forceinline__ float value(uint16_t h) {
    return __builtin_bit_cast(float, (uint32_t)h << 16);
  }
  // Two fp32 values each as the sum of two parts, both rounded to nearest: within 2^-17 of the
  // value and to either side of it.  (Cut to 16 bits instead they are up to 2^-15 too small,
  // all to one side, which an average over many keys keeps.)
  static __device__ __forceinline__ u32x2 split(float x, float y) {
    typedef float pair __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const uint32_t h =
        __builtin_bit_cast(uint32_t, __builtin_convertvector((pair{x, y}), bf16x2));
    const pair left = {x - __builtin_bit_cast(float, h << 16),
                       y - __builtin_bit_cast(float, h & 0xFFFF0000u)};
    return u32x2{h, __builtin_bit_cast(uint32_t, __builtin_convertvector(left, bf16x2))};
  }
  static constexpr uint32_t kExponent = 0x7F80u;
  static constexpr uint32_t kOne = 0x3F80u;
  static constexpr float kTop = 0.0f, kLag = 8.0f;  // (fp32's exponents: any will do)
};

}  // namespace flexq
