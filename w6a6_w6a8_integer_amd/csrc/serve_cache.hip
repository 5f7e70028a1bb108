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
// one launch does.  Bound by its latencies (launch, the lengths, the scan, the page looked up,
// each after the other): 4.5 us for 16 requests, 9.3 for 512 prompts and 8.7 MB.
template <int PER>
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

  const bool wide = (reinterpret_cast<uintptr_t>(slots) & 15) == 0;
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
  // PER slots a thread: one search, then on from token to token.
  for (int64_t t0 = PER * (int64_t)first; t0 < max_tokens; t0 += PER * (int64_t)stride) {
    int slot[PER];
    int b = 0, next = 0, id = -1;  // request, its last token + 1, page of column `col`
    int64_t c = 0, col = -1;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int64_t t = t0 + j;
      slot[j] = -1;
      if (t >= base.x) continue;
      if (j == 0 || t >= next) {
        b = j == 0 ? find(cu, B, (int)t) : b + 1;
        while (t >= cu[b + 1]) ++b;  // (requests without new tokens)
        next = cu[b + 1];
        c = max(0, ctx_lens[b]);
        col = -1;
      }
      const int64_t pos = c + (t - cu[b]), now = pos >> shift;
      if (now != col) {
        col = now;
        const int64_t have = (c + page - 1) >> shift, f = (int64_t)head + off[b] + (col - have);
        id = -1;
        if (col < max_blocks) {
          if (col < have)
            id = table[(int64_t)b * max_blocks + col];
          else if (f >= 0 && f < num_free)
            id = free_pages[f];
        }
        if (id > INT32_MAX >> shift) id = -1;  // its slots are no int32
      }
      if (id >= 0) slot[j] = (id << shift) + (int)(pos & (page - 1));
    }
    if constexpr (PER % 4 == 0) {
      if (t0 + PER <= max_tokens && wide) {
#pragma unroll
        for (int j = 0; j < PER; j += 4)
          *reinterpret_cast<int4*>(slots + t0 + j) =
              make_int4(slot[j], slot[j + 1], slot[j + 2], slot[j + 3]);
        continue;
      }
    }
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (t0 + j < max_tokens) slots[t0 + j] = slot[j];
  }
}

// New keys and values into the cache, a copy bound by HBM (read and written once): prompts of
// 180 MB take 36 to 37 us, 4.9 TB/s, what a plain copy reaches; the loads and stores are not
// kept in the caches (43 us when they were).
//
// In the cache the keys of a token are 64-byte pieces and the values have the token
// innermost, eight tokens of one d in 16 bytes (half a 16-token block).  So tokens whose
// slots run on through the same half block form a group: its values go through LDS and
// come out as columns, a whole group (eight tokens) in 16-byte stores, a shorter one (the
// ends of a prompt, single tokens, scattered slots) element by element.  A workgroup owns
// the groups that begin among its kTokens tokens, for one head; the last may reach seven
// tokens further.
template <int D, int kTokens>
__global__ __launch_bounds__(256) void kv_cache_write_kernel(
    const uint16_t* __restrict__ k, int64_t k_st, int64_t k_sh, const uint16_t* __restrict__ v,
    int64_t v_st, int64_t v_sh, const int* __restrict__ slots, int T, int Hkv, int64_t num_slots,
    int shift, uint16_t* __restrict__ kc, uint16_t* __restrict__ vc) {
  constexpr int kPieces = D / 8;       // 16-byte pieces of a row
  constexpr int kPitch = D + 8;        // of a token's row in LDS, elements
  constexpr int kMost = kTokens + 7;
  __shared__ __attribute__((aligned(16))) uint16_t tile[kMost * kPitch];
  __shared__ int slot_of[kMost + 1];   // of token t0 - 1 + i, -1 where it is dropped
  __shared__ int begin[kTokens], length[kTokens];  // of the groups, begin from t0
  __shared__ int groups, first, end;       // and the tokens they hold, from t0
  const int h = blockIdx.y, t0 = blockIdx.x * kTokens, tid = threadIdx.x;
  if (tid <= kMost) {
    const int t = t0 - 1 + tid;
    const int64_t slot = t >= 0 && t < T ? slots[t] : -1;
    slot_of[tid] = slot >= 0 && slot < num_slots ? (int)slot : -1;
  }
  __syncthreads();
  if (tid < kTokens) {  // one wave
    const int* s = slot_of + 1 + tid;
    const bool kept = s[0] >= 0;
    const bool leads = kept && ((s[0] & 7) == 0 || s[-1] != s[0] - 1);
    int n = 1;
    while (leads && (s[0] + n & 7) != 0 && s[n] == s[0] + n) ++n;
    const uint64_t mask = __ballot(leads);
    if (leads) {
      const int at = __builtin_popcountll(mask & ((1ull << tid) - 1));
      begin[at] = tid;
      length[at] = n;
      if ((mask >> tid) >> 1 == 0) end = tid + n;
    }
    if (tid == 0) {
      groups = __builtin_popcountll(mask);
      first = mask ? __builtin_ctzll(mask) : 0;
      if (!mask) end = 0;
    }
  }
  __syncthreads();
  const int at0 = first, n = end - first;
  // every load of the workgroup before its first store, and none kept in the caches (18 %)
  constexpr int kTurns = (kMost * kPieces + 255) / 256;
  u32x4 ke[kTurns], ve[kTurns];
#pragma unroll
  for (int u = 0; u < kTurns; ++u) {
    const int i = tid + u * 256, t = i / kPieces, d = i % kPieces * 8;
    if (i >= n * kPieces) break;
    const int64_t from = t0 + at0 + t;
    ke[u] = __builtin_nontemporal_load(
        reinterpret_cast<const u32x4*>(k + from * k_st + h * k_sh + d));
    ve[u] = __builtin_nontemporal_load(
        reinterpret_cast<const u32x4*>(v + from * v_st + h * v_sh + d));
  }
#pragma unroll
  for (int u = 0; u < kTurns; ++u) {
    const int i = tid + u * 256, t = i / kPieces, d = i % kPieces * 8;
    if (i >= n * kPieces) break;
    const int slot = slot_of[1 + at0 + t];
    if (slot < 0) continue;  // dropped
    *reinterpret_cast<u32x4*>(tile + t * kPitch + d) = ve[u];
    const int r = slot & ((1 << shift) - 1);
    const int64_t block = ((int64_t)(slot >> shift) * Hkv + h) * (1 << (shift - 4)) + (r >> 4);
    *reinterpret_cast<u32x4*>(kc + block * (16 * D) + (d >> 5) * 512 + (r & 15) * 32 + (d & 31)) =
        ke[u];
  }
  __syncthreads();
  for (int i = tid; i < groups * D; i += 256) {
    const int g = i / D, d = i % D;
    const int len = length[g], slot = slot_of[1 + begin[g]];
    const uint16_t* from = tile + (begin[g] - at0) * kPitch + d;
    const int r = slot & ((1 << shift) - 1);
    const int64_t block = ((int64_t)(slot >> shift) * Hkv + h) * (1 << (shift - 4)) + (r >> 4);
    uint16_t* to = vc + block * (16 * D) + d * 16 + (r & 15);
    if (len == 8) {
      u32x4 out;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        out[j] = from[2 * j * kPitch] | (uint32_t)from[(2 * j + 1) * kPitch] << 16;
      *reinterpret_cast<u32x4*>(to) = out;
    } else {
      for (int j = 0; j < len; ++j) to[j] = from[j * kPitch];
    }
  }
}

hipError_t launch_block_tables(const int32_t* ctx, const int32_t* add, int64_t B,
                               const int32_t* free_pages, int64_t num_free, const int32_t* head,
                               int page_size, int32_t* table, int64_t max_blocks,
                               int64_t max_tokens, int32_t* slots, int32_t* cu, int32_t* counts,
                               hipStream_t stream) {
  // One slot a thread while those threads fit the GPU twice over; then eight, which share
  // the search and most page lookups (16 requests of a token: 4.5 us against 7.0 with eight;
  // 2.1 million slots: 9.3 against 13.9 with one).
  const int64_t most = 8 * device_cu_count();
  const int per = max_tokens <= most * kScanThreads / 4 ? 1 : 8;
  const int64_t work = std::max<int64_t>((max_tokens + per - 1) / per, B);
  const int64_t grid = std::min<int64_t>(work / kScanThreads + 1, most);
  const size_t lds = (size_t)(B + 1) * 2 * sizeof(int);
  auto* kernel = per == 1 ? block_tables_kernel<1> : block_tables_kernel<8>;
  return launch_kernel_lds(kernel, dim3((unsigned)grid), dim3(kScanThreads), lds, stream, ctx,
                           add, (int)B, free_pages, (int)num_free, head,
                           __builtin_ctz((unsigned)page_size), table, (int)max_blocks,
                           (int)max_tokens, slots, cu, counts);
}

hipError_t launch_kv_cache_write(const uint16_t* k, int64_t k_st, int64_t k_sh,
                                 const uint16_t* v, int64_t v_st, int64_t v_sh,
                                 const int32_t* slots, int64_t T, int64_t Hkv, int64_t D,
                                 int64_t num_pages, int page_size, uint16_t* kc, uint16_t* vc,
                                 hipStream_t stream) {
  // sixteen tokens a workgroup where that is what it takes to have two for a compute unit
  // (80 tokens: 4.8 us against 8.5 with 64; prompts: 40 us with 16 against 37 with 64)
  const int tokens = (T + 63) / 64 * Hkv >= 2 * device_cu_count() ? 64 : 16;
  const dim3 grid((unsigned)((T + tokens - 1) / tokens), (unsigned)Hkv);
  auto* kernel = tokens == 64 ? (D == 64    ? kv_cache_write_kernel<64, 64>
                                 : D == 96  ? kv_cache_write_kernel<96, 64>
                                 : D == 128 ? kv_cache_write_kernel<128, 64>
                                            : kv_cache_write_kernel<256, 64>)
                              : (D == 64    ? kv_cache_write_kernel<64, 16>
                                 : D == 96  ? kv_cache_write_kernel<96, 16>
                                 : D == 128 ? kv_cache_write_kernel<128, 16>
                                            : kv_cache_write_kernel<256, 16>);
  return launch_kernel(kernel, grid, dim3(256), stream, k, k_st, k_sh, v, v_st, v_sh, slots,
                       (int)T, (int)Hkv, num_pages * page_size,
                       __builtin_ctz((unsigned)page_size), kc, vc);
}

}  // namespace flexq
