// serve_plan.h -- what the attention kernels over a paged cache share: how a call's cache is
// cut into shares of equal work on the GPU, where a share keeps what others join, and the
// kernel that joins it.  A is the kernel's argument struct (AttentionArgs or one that extends
// it) with its tuning: A::kHead, what starting on a request costs in 32-key steps,
// A::least_share(), the least share of a workgroup, A::kWindowed, whether keys between the
// first tokens and a sliding window are passed over, and A::kScaledReference, whether a row's
// reference follows its values' scales.
#pragma once
#include <algorithm>

#include "kernels.h"
#include "serve_device.h"
#include "serve_kernels.h"

namespace flexq {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

typedef __attribute__((address_space(4))) const int32_t* scalar_ptr_t;

// (max, sum) over the lanes that hold one of RW rows (l ^ 32, and of 16 rows l ^ 16 too).  A
// swap of x with itself gives both halves of the exchange, each in every lane.
template <int RW>
__device__ __forceinline__ float row_max(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(u, u, false, false));
  const uint32_t a0 = a[0], a1 = a[1];
  const float y = fmaxf(__builtin_bit_cast(float, a0), __builtin_bit_cast(float, a1));
  if constexpr (RW == 32) return y;
  const uint32_t v = __builtin_bit_cast(uint32_t, y);
  const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(v, v, false, false));
  const uint32_t b0 = b[0], b1 = b[1];
  return fmaxf(__builtin_bit_cast(float, b0), __builtin_bit_cast(float, b1));
}
template <int RW>
__device__ __forceinline__ float row_sum(float x) {
  if constexpr (RW == 16) {
    const uint32_t v = __builtin_bit_cast(uint32_t, x);
    const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(v, v, false, false));
    const uint32_t b0 = b[0], b1 = b[1];
    x = __builtin_bit_cast(float, b0) + __builtin_bit_cast(float, b1);
  }
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(u, u, false, false));
  const uint32_t a0 = a[0], a1 = a[1];
  return __builtin_bit_cast(float, a0) + __builtin_bit_cast(float, a1);
}

// the low n bits, n clamped to 0 .. 8
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : (n >= 8 ? 0xFFu : (1u << n) - 1u);
}

// The plan.  Request b weighs A::kHead + steps_b, steps_b = ceil((ctx + new) / 32) its 32-key
// steps, without those that no window reaches (0 without new tokens); the weights laid end to end are cut into G shares that
// differ by one unit at most: equal work whatever the lengths.  A share holds the end of
// one request, whole ones, and the beginning of another.  Whole ones are written out; of
// the others each share keeps statistics and sums in the workspace (place 2 i the end,
// 2 i + 1 the beginning), and a second kernel joins them in order.  The lengths live on the
// GPU, so every wave forms the plan itself.
struct Plan {
  uint32_t shares, size, longer;  // G; `longer` shares of size + 1 come first
  __device__ uint32_t start(uint32_t i) const { return i * size + min(i, longer); }
  // the share that holds unit x
  __device__ uint32_t share_of(uint32_t x) const {
    const uint32_t in_longer = longer * (size + 1);
    return x < in_longer ? x / (size + 1) : longer + (x - in_longer) / size;
  }
};

struct Request {
  int cu, n_new, ctx, len;
  int gap = 0;  // 32-key steps between the first tokens and the window
  __device__ uint32_t steps() const { return max(1, ((len + 31) >> 5) - gap); }  // rows without a key too
  template <class A>
  __device__ uint32_t weight() const { return n_new == 0 ? 0 : A::kHead + steps(); }
};

template <class A>
__device__ __forceinline__ Request make_request(const A& a, int cu, int cu1, int ctx) {
  Request r;
  const int most = a.max_blocks << a.page_shift;
  r.cu = cu;
  r.n_new = min(max(0, cu1 - cu), a.max_new);
  r.ctx = min(max(0, ctx), most);
  r.len = min(r.ctx + r.n_new, most);
  if constexpr (A::kWindowed) r.gap = window_gap(a, r);
  return r;
}

template <class A>
__device__ __forceinline__ Request load_request(const A& a, int b) {
  return b < a.B ? make_request(a, a.cu[b], a.cu[b + 1], a.ctx[b]) : Request{};
}

// Sums over the lanes up to each, by DPP moves (a move through LDS takes ten times as long): within rows
// of 16, then a row's last lane into the next row, and the first half's into the second.
__device__ __forceinline__ uint32_t inclusive_sum(uint32_t v) {
#define FLEXQ_SCAN_STEP(ctrl, rows) \
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xF, false)
  FLEXQ_SCAN_STEP(0x111, 0xF);  // row_shr:1, 2, 4, 8
  FLEXQ_SCAN_STEP(0x112, 0xF);
  FLEXQ_SCAN_STEP(0x114, 0xF);
  FLEXQ_SCAN_STEP(0x118, 0xF);
  FLEXQ_SCAN_STEP(0x142, 0xA);  // row_bcast:15 into rows 1 and 3
  FLEXQ_SCAN_STEP(0x143, 0xC);  // row_bcast:31 into rows 2 and 3
#undef FLEXQ_SCAN_STEP
  return v;
}

// 64 consecutive requests, one a lane.
struct Window {
  int base;
  Request mine;
  template <class A>
  __device__ Request at(int b) const {
    const int i = b - base;
    Request r;
    r.cu = __builtin_amdgcn_readlane(mine.cu, i);
    r.n_new = __builtin_amdgcn_readlane(mine.n_new, i);
    r.ctx = __builtin_amdgcn_readlane(mine.ctx, i);
    r.len = __builtin_amdgcn_readlane(mine.len, i);
    if constexpr (A::kWindowed) r.gap = __builtin_amdgcn_readlane(mine.gap, i);
    return r;
  }
};

// The plan, and the request that holds the first unit of share i with the units before
// that request (b = B where there is no such share) and a window that begins at or before
// it.  Two levels of 64 lanes: kMaxRequests.
template <class A>
__device__ __forceinline__ Plan make_plan(const A& a, uint32_t shares, uint32_t i,
                                          int& b, uint32_t& before, Window& window) {
  static_assert(kMaxRequests <= 64 * 64, "two levels of 64 lanes");
  const int lane = threadIdx.x & 63;
  const int per = (a.B + 63) / 64;
  uint32_t sum = 0;
  window.base = 0;
  window.mine = load_request(a, lane * per);
  if (lane * per < a.B) sum = window.mine.template weight<A>();
#pragma unroll 4
  for (int j = 1; j < per; ++j) sum += load_request(a, lane * per + j).template weight<A>();
  const uint32_t inc = inclusive_sum(sum);
  const uint32_t total = __builtin_amdgcn_readlane(inc, 63);
  Plan plan;
  plan.shares = min(shares, max(1u, total / a.least_share()));
  plan.size = total / plan.shares;
  plan.longer = total - plan.size * plan.shares;
  b = a.B;
  before = 0;
  if (i >= plan.shares || total == 0) return plan;
  const uint32_t x = plan.start(i);
  const int at = __builtin_ctzll(__ballot(inc > x));
  before = __builtin_amdgcn_readlane(inc - sum, at);
  b = at * per;
  if (per > 1) {
    window.base = b;
    window.mine = load_request(a, b + lane);
    const uint32_t w = lane < per ? window.mine.template weight<A>() : 0;
    const uint32_t in = inclusive_sum(w);
    const int k = __builtin_ctzll(__ballot(before + in > x));
    before += __builtin_amdgcn_readlane(in - w, k);
    b += k;
  }
  return plan;
}

// Where the workspace keeps what: (first, last) share of every request, then for every
// place, key head and row the maximum and sum, then the unnormalized output.
struct Parts {
  int2* plan;
  float2* stat;
  f32x4* out;
};

__host__ __device__ __forceinline__ size_t round16(size_t n) { return (n + 15) / 16 * 16; }

__device__ __forceinline__ Parts parts_of(const AttentionArgs& a, int shares, int rows) {
  char* p = static_cast<char*>(a.workspace);
  Parts w;
  w.plan = reinterpret_cast<int2*>(p);
  p += round16(sizeof(int2) * a.B);
  w.stat = reinterpret_cast<float2*>(p);
  p += round16(sizeof(float2) * 2 * shares * a.Hkv * rows);
  w.out = reinterpret_cast<f32x4*>(p);
  return w;
}

// 2^n x for a whole n of any size: an infinite x stays.
__device__ __forceinline__ float scaled(float x, float n) {
  return __builtin_ldexpf(x, (int)fminf(fmaxf(n, -1e4f), 1e4f));
}

// Four elements of a row of out, and its lse.  With A::kScaledReference, where the reference
// follows more than the row's scores, total's exponent goes to the whole ref first, so that lse is
// rounded alike whatever the reference is.
template <class E, class A>
__device__ __forceinline__ void write_row(const A& a, int64_t t, int h, int d4, f32x4 acc, float ref,
                                          float total) {
  const float by = total != 0.0f ? 1.0f / total : 0.0f;
  u32x2 v;
#pragma unroll
  for (int k = 0; k < 2; ++k)
    v[k] = E::bits(acc[2 * k] * by) | (uint32_t)E::bits(acc[2 * k + 1] * by) << 16;
  *reinterpret_cast<u32x2*>(a.out + (t * a.H + h) * a.D + 4 * d4) = v;
  if (a.lse && d4 == 0) {
    if constexpr (A::kScaledReference) {
      ref += (float)__builtin_amdgcn_frexp_expf(total);
      total = __builtin_amdgcn_frexp_mantf(total);
    }
    a.lse[t * a.H + h] = total != 0.0f ? (ref + log2f(total)) * kLn2 : -INFINITY;
  }
}

// Joins the parts of requests that several shares hold, in a fixed order: D / 4 threads (four
// elements each) take a row's parts SLICES at a time, and the slices' sums are joined
// through LDS.
template <class A, class E, int DT, int SLICES>
__global__ __launch_bounds__(256) void join_parts_kernel(const A a, int shares) {
  constexpr int D = 32 * DT;
  constexpr int kLanes = D / 4, kRows = 256 / kLanes / SLICES;
  __shared__ f32x4 sums[SLICES > 1 ? 256 : 1];
  __shared__ float2 stats[SLICES > 1 ? 256 : 1];
  const int b = blockIdx.z, hk = blockIdx.y;
  const int group = a.H / a.Hkv;
  const int slot = threadIdx.x / kLanes, d4 = threadIdx.x % kLanes;
  const int slice = slot % SLICES;
  const int row = blockIdx.x * kRows + slot / SLICES;
  const Parts parts = parts_of(a, shares, a.max_new * group);
  const int2 plan = parts.plan[b];  // not set for a request without new tokens
  const Request request = load_request(a, b);
  const int rows = request.n_new * group;
  if ((int)blockIdx.x * kRows >= rows || plan.x == plan.y) return;  // the whole workgroup
  const bool in = slot < kRows * SLICES && row < rows;
  const int64_t stride = (int64_t)a.Hkv * (a.max_new * group);
  // the first share's place is 2 i + 1, the others' 2 i
  const int64_t at0 = 2 * (int64_t)plan.x * stride + (int64_t)hk * (a.max_new * group) + row;
  const int n = in ? plan.y - plan.x + 1 : 0;
  float top = -INFINITY, total = 0.0f;
  f32x4 acc = {};
#pragma unroll 4
  for (int i = slice; i < n; i += SLICES) {
    const int64_t at = at0 + (i == 0 ? 1 : 2 * (int64_t)i) * stride;
    const float2 s = parts.stat[at];
    const f32x4 o = parts.out[at * (D / 4) + d4];
    const float to = fmaxf(top, s.x), ref = to == -INFINITY ? 0.0f : to;
    const float old = top - ref, by = s.x - ref;
    top = to;
    total = scaled(s.y, by) + scaled(total, old);
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = scaled(o[k], by) + scaled(acc[k], old);
  }
  if constexpr (SLICES > 1) {
    sums[threadIdx.x] = acc;
    stats[threadIdx.x] = {top, total};
    __syncthreads();
    if (slice != 0 || !in) return;
    for (int j = 1; j < SLICES; ++j) top = fmaxf(top, stats[threadIdx.x + j * kLanes].x);
    const float ref = top == -INFINITY ? 0.0f : top;
    total = 0.0f;
    acc = f32x4{};
#pragma unroll
    for (int j = 0; j < SLICES; ++j) {
      const float2 s = stats[threadIdx.x + j * kLanes];
      const f32x4 o = sums[threadIdx.x + j * kLanes];
      const float by = s.x - ref;
      total += scaled(s.y, by);
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[k] += scaled(o[k], by);
    }
  }
  const int64_t t = (int64_t)request.cu + row / group;
  if (in && t >= 0 && t < a.T)
    write_row<E>(a, t, hk * group + row % group, d4, acc, top == -INFINITY ? 0.0f : top, total);
}

// The join where a call has more than one share.
template <class A, class E, int DT>
hipError_t launch_join(const A& a, int shares, hipStream_t stream) {
  // a row's parts number about shares / B: few are taken by one thread after the other
  constexpr int kSlots = 256 / (8 * DT);
  const bool many = shares >= 8 * a.B;
  const int rows = a.max_new * (a.H / a.Hkv), per = many ? 1 : kSlots;
  return launch_kernel(
      many ? join_parts_kernel<A, E, DT, kSlots> : join_parts_kernel<A, E, DT, 1>,
      dim3((unsigned)((rows + per - 1) / per), (unsigned)a.Hkv, (unsigned)a.B), dim3(256), stream,
      a, shares);
}

// Bytes of workspace for `shares` shares.
inline size_t parts_bytes(int64_t B, int64_t max_new, int64_t H, int64_t D, int shares) {
  const size_t places = shares == 1 ? 0 : (size_t)2 * shares * H * max_new;
  return round16(sizeof(int2) * B) + round16(sizeof(float2) * places) + sizeof(float) * places * D;
}

}  // namespace flexq
