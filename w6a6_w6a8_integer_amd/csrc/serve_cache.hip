// serve_cache.hip -- the paged cache's bookkeeping on the GPU: block tables and slot maps
// from request lengths, and the writing of new keys and values.
#include <algorithm>

#include "kernels.h"
#include "serve_device.h"
#include "serve_kernels.h"

namespace flexq {

namespace {

constexpr int kScanThreads = 256;

// Exclusive prefix sums of the two numbers of every thread over the workgroup's
// threads; tot receives the sums.
__device__ __forceinline__ int2 scan2(int2 v, int2* wave_sums, int2& tot) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int2 inc = v;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const int a = __shfl_up(inc.x, o), b = __shfl_up(inc.y, o);
    if (lane >= o) {
      inc.x += a;
      inc.y += b;
    }
  }
  if (lane == 63) wave_sums[wave] = inc;
  __syncthreads();
  int2 before = {0, 0}, all = {0, 0};
#pragma unroll
  for (int w = 0; w < kScanThreads / 64; ++w) {
    if (w == wave) before = all;
    all.x += wave_sums[w].x;
    all.y += wave_sums[w].y;
  }
  __syncthreads();
  tot = all;
  return {before.x + inc.x - v.x, before.y + inc.y - v.y};
}

// The last i in [0, n) with start[i] <= v, for start ascending from start[0] = 0.
__device__ __forceinline__ int find(const int* start, int n, int v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= v)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

}  // namespace

// Every workgroup forms the prefix sums of all requests in LDS (at most 32 KB, from
// L2), then takes its share of the new pages and of the slot map; a slot
// on a new page reads the free list, not the table another workgroup may be writing, so
// one launch does.
__global__ __launch_bounds__(kScanThreads) void block_tables_kernel(
    const int* __restrict__ ctx_lens, const int* __restrict__ new_lens, int B,
    const int* __restrict__ free_pages, int num_free, const int* __restrict__ free_head, int shift,
    int* __restrict__ table, int max_blocks, int max_tokens, int* __restrict__ slots,
    int* __restrict__ cu_new, int* __restrict__ counts) {
  extern __shared__ int sums[];
  int* cu = sums;           // [B + 1] tokens before request b
  int* off = sums + B + 1;  // [B + 1] new pages before request b
  __shared__ int2 wave_sums[kScanThreads / 64];
  const int page = 1 << shift;
  const int head = free_head ? *free_head : 0;
  int2 base = {0, 0};
  for (int b0 = 0; b0 < B; b0 += kScanThreads) {
    const int b = b0 + threadIdx.x;
    int2 v = {0, 0};
    if (b < B) {
      const int64_t c = max(0, ctx_lens[b]), n = max(0, new_lens[b]);
      v.x = (int)n;
      v.y = (int)(((c + n + page - 1) >> shift) - ((c + page - 1) >> shift));
    }
    int2 tot;
    const int2 e = scan2(v, wave_sums, tot);
    if (b < B) {
      cu[b] = base.x + e.x;
      off[b] = base.y + e.y;
    }
    base.x += tot.x;
    base.y += tot.y;
  }
  if (threadIdx.x == 0) {
    cu[B] = base.x;
    off[B] = base.y;
  }
  __syncthreads();

  const int stride = gridDim.x * kScanThreads, first = blockIdx.x * kScanThreads + threadIdx.x;
  for (int b = first; b <= B; b += stride) cu_new[b] = cu[b];
  if (first == 0) {
    counts[0] = base.x;
    counts[1] = base.y;
    counts[2] = head + base.y;
  }
  for (int64_t i = first; i < base.y; i += stride) {
    const int b = find(off, B, (int)i);
    const int64_t have = ((int64_t)max(0, ctx_lens[b]) + page - 1) >> shift;
    const int64_t col = have + (i - off[b]);
    const int64_t f = (int64_t)head + i;
    if (col >= 0 && col < max_blocks)
      table[(int64_t)b * max_blocks + col] = f >= 0 && f < num_free ? free_pages[f] : -1;
  }
  for (int64_t t = first; t < max_tokens; t += stride) {
    int slot = -1;
    if (t < base.x) {
      const int b = find(cu, B, (int)t);
      const int64_t c = max(0, ctx_lens[b]);
      const int64_t pos = c + (t - cu[b]);
      const int64_t have = (c + page - 1) >> shift;
      const int64_t col = pos >> shift;
      int id = -1;
      if (col >= 0 && col < max_blocks) {
        const int64_t f = (int64_t)head + off[b] + (col - have);
        if (col < have)
          id = table[(int64_t)b * max_blocks + col];
        else if (f >= 0 && f < num_free)
          id = free_pages[f];
      }
      if (id >= 0) slot = (int)(((int64_t)id << shift) + (pos & (page - 1)));
    }
    slots[t] = slot;
  }
}

// One thread = 8 consecutive elements of one head of one token: a 16-byte piece of the
// keys' row, or 8 elements of the values that go to 8 places 32 bytes apart.
__global__ __launch_bounds__(256) void kv_cache_write_kernel(
    const uint16_t* __restrict__ k, int64_t k_st, int64_t k_sh, const uint16_t* __restrict__ v,
    int64_t v_st, int64_t v_sh, const int* __restrict__ slots, int64_t items, int Hkv, int D,
    int64_t num_slots, int shift, uint16_t* __restrict__ kc, uint16_t* __restrict__ vc) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= items) return;
  const int per_row = D / 8;
  const int d = (int)(i % per_row) * 8;
  const int64_t th = i / per_row;
  const int h = (int)(th % Hkv);
  const int64_t t = th / Hkv;
  const int64_t slot = slots[t];
  if (slot < 0 || slot >= num_slots) return;
  const int64_t r = slot & ((1 << shift) - 1);
  const int64_t block = ((slot >> shift) * Hkv + h) * (1 << (shift - 4)) + (r >> 4);
  const u32x4 ke = *reinterpret_cast<const u32x4*>(k + t * k_st + h * k_sh + d);
  *reinterpret_cast<u32x4*>(kc + block * 16 * D + (d >> 5) * 512 + (r & 15) * 32 + (d & 31)) = ke;
  const u32x4 ve = *reinterpret_cast<const u32x4*>(v + t * v_st + h * v_sh + d);
  uint16_t* dst = vc + block * 16 * D + d * 16 + (r & 15);
#pragma unroll
  for (int e = 0; e < 8; ++e) dst[e * 16] = (uint16_t)(ve[e >> 1] >> (16 * (e & 1)));
}

hipError_t launch_block_tables(const int32_t* ctx, const int32_t* add, int64_t B,
                               const int32_t* free_pages, int64_t num_free, const int32_t* head,
                               int page_size, int32_t* table, int64_t max_blocks,
                               int64_t max_tokens, int32_t* slots, int32_t* cu, int32_t* counts,
                               hipStream_t stream) {
  const int64_t work = std::max<int64_t>(max_tokens, B);
  const int64_t grid = std::min<int64_t>(work / kScanThreads + 1, 4 * device_cu_count());
  const size_t lds = (size_t)(B + 1) * 2 * sizeof(int);
  return launch_kernel_lds(block_tables_kernel, dim3((unsigned)grid), dim3(kScanThreads), lds,
                           stream, ctx, add, (int)B, free_pages, (int)num_free, head,
                           __builtin_ctz((unsigned)page_size), table, (int)max_blocks,
                           (int)max_tokens, slots, cu, counts);
}

hipError_t launch_kv_cache_write(const uint16_t* k, int64_t k_st, int64_t k_sh,
                                 const uint16_t* v, int64_t v_st, int64_t v_sh,
                                 const int32_t* slots, int64_t T, int64_t Hkv, int64_t D,
                                 int64_t num_pages, int page_size, uint16_t* kc, uint16_t* vc,
                                 hipStream_t stream) {
  const int64_t items = T * Hkv * (D / 8);
  return launch_kernel(kv_cache_write_kernel, dim3((unsigned)((items + 255) / 256)), dim3(256),
                       stream, k, k_st, k_sh, v, v_st, v_sh, slots, items, (int)Hkv, (int)D,
                       num_pages * page_size, __builtin_ctz((unsigned)page_size), kc, vc);
}

}  // namespace flexq
