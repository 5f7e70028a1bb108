// serve_api.hip -- the C ABI of the decoding-step operators (declared in
// include/flexq_serve.h).  As in api.hip: every argument is checked on the host before any
// HIP call, and nothing is allocated.
#include <cmath>
#include <initializer_list>

#include "../../include/flexq_serve.h"
#include "abi_checks.h"
#include "serve_kernels.h"

namespace {

using flexq::aligned;
using flexq::launched;
using flexq::overlap;
using flexq::Range;
using flexq::range_of;

constexpr int64_t kMaxM = 65535LL * 16;
constexpr int64_t kMaxN = 1LL << 24;
constexpr int64_t kMaxK = 1LL << 22;

inline bool any_overlap(Range out, std::initializer_list<Range> others) {
  for (const Range& r : others)
    if (overlap(out, r)) return true;
  return false;
}

// bytes from the first element to the last of a [n0][n1][n2] tensor of `size`-byte
// elements with strides st0, st1 >= 0 and 1
inline uint64_t span(int64_t n0, int64_t st0, int64_t n1, int64_t st1, int64_t n2, int size) {
  return ((uint64_t)(n0 - 1) * st0 + (uint64_t)(n1 - 1) * st1 + n2) * size;
}

inline flexq_status check_dtype(int32_t dtype) {
  return dtype == FLEXQ_FP16 || dtype == FLEXQ_BF16 ? FLEXQ_SUCCESS : FLEXQ_ERROR_INVALID_VALUE;
}

flexq_status check_w4(int64_t N, int64_t K, int32_t group_size) {
  if (N < 0 || K <= 0) return FLEXQ_ERROR_INVALID_VALUE;
  if (group_size != 32 && group_size != 64 && group_size != 128) return FLEXQ_ERROR_UNSUPPORTED;
  if (N % 16 != 0 || N > kMaxN || K % 128 != 0 || K > kMaxK) return FLEXQ_ERROR_UNSUPPORTED;
  if (N * (K / group_size) >= (1LL << 29)) return FLEXQ_ERROR_UNSUPPORTED;  // 32-bit offsets
  return FLEXQ_SUCCESS;
}

inline bool cache_page(int32_t page) {
  return page == 16 || page == 32 || page == 64 || page == 128 || page == 256;
}

inline bool head_width(int64_t D) { return D == 64 || D == 96 || D == 128 || D == 256; }

// a paged cache's sizes: 16-token blocks are counted in 31 bits
flexq_status check_cache(int64_t num_pages, int64_t Hkv, int64_t D, int32_t page_size) {
  if (num_pages < 0 || Hkv <= 0 || D <= 0 || page_size <= 0) return FLEXQ_ERROR_INVALID_VALUE;
  if (!cache_page(page_size) || !head_width(D)) return FLEXQ_ERROR_UNSUPPORTED;
  if (Hkv >= (1LL << 31) || num_pages >= (1LL << 31) / Hkv / (page_size / 16) + 1 ||
      num_pages * Hkv * (page_size / 16) >= (1LL << 31))
    return FLEXQ_ERROR_UNSUPPORTED;
  return FLEXQ_SUCCESS;
}

inline uint64_t cache_bytes(int64_t num_pages, int64_t Hkv, int64_t D, int32_t page_size) {
  return (uint64_t)num_pages * Hkv * page_size * D * 2;
}

constexpr int64_t kMaxStride = 1LL << 40;

flexq_status check_attention_sizes(int64_t B, int64_t max_new, int64_t H, int64_t Hkv, int64_t D) {
  if (B < 0 || max_new < 0 || H <= 0 || Hkv <= 0 || D <= 0 || H % Hkv != 0)
    return FLEXQ_ERROR_INVALID_VALUE;
  if (!head_width(D) || H > 4096 || B > flexq::kMaxRequests || max_new > 65536)
    return FLEXQ_ERROR_UNSUPPORTED;
  return FLEXQ_SUCCESS;
}

}  // namespace

extern "C" {

size_t flexq_packed_w4_bytes(int64_t N, int64_t K) {
  if (N <= 0 || K <= 0 || K % 128 != 0) return 0;
  return (size_t)N * (size_t)K / 2;
}

flexq_status flexq_pack_w4(const uint16_t* w, int32_t dtype, int64_t N, int64_t K,
                           int32_t group_size, uint32_t* w4, uint16_t* s_w_fp16, void* stream) {
  FLEXQ_TRY(check_dtype(dtype));
  FLEXQ_TRY(check_w4(N, K, group_size));
  if (N == 0) return FLEXQ_SUCCESS;
  if (!w || !w4 || !s_w_fp16) return FLEXQ_ERROR_INVALID_VALUE;
  if (!aligned(w, 16) || !aligned(w4, 16) || !aligned(s_w_fp16, 2)) return FLEXQ_ERROR_UNSUPPORTED;
  const Range in = range_of(w, (uint64_t)N * K * 2);
  const Range ow = range_of(w4, flexq_packed_w4_bytes(N, K));
  const Range os = range_of(s_w_fp16, (uint64_t)N * (K / group_size) * 2);
  if (overlap(in, ow) || overlap(in, os) || overlap(ow, os)) return FLEXQ_ERROR_INVALID_VALUE;
  return launched(flexq::launch_pack_w4(w, dtype == FLEXQ_BF16, N, K, group_size, w4, s_w_fp16,
                                        (hipStream_t)stream));
}

size_t flexq_gemv_w4_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || M > kMaxM || N <= 0 || check_w4(N, K, 128) != FLEXQ_SUCCESS) return 0;
  return flexq::gemv_w4_workspace_bytes(M, N, K);
}

flexq_status flexq_gemv_w4(const uint16_t* x, int32_t dtype, int64_t x_stride,
                           const uint32_t* w4, const uint16_t* s_w_fp16, int64_t M, int64_t N,
                           int64_t K, int32_t group_size, void* workspace,
                           size_t workspace_bytes, uint16_t* y, void* stream) {
  FLEXQ_TRY(check_dtype(dtype));
  if (M < 0) return FLEXQ_ERROR_INVALID_VALUE;
  FLEXQ_TRY(check_w4(N, K, group_size));
  if (M > kMaxM) return FLEXQ_ERROR_UNSUPPORTED;
  if (M == 0 || N == 0) return FLEXQ_SUCCESS;
  if (!x || !w4 || !s_w_fp16 || !y) return FLEXQ_ERROR_INVALID_VALUE;
  if (M > 1) {
    if (x_stride < K) return FLEXQ_ERROR_INVALID_VALUE;
    if (x_stride % 8 != 0 || x_stride > (1LL << 24)) return FLEXQ_ERROR_UNSUPPORTED;
  } else {
    x_stride = K;
  }
  const size_t need = flexq::gemv_w4_workspace_bytes(M, N, K);
  if (need > 0 && (!workspace || workspace_bytes < need)) return FLEXQ_ERROR_INVALID_VALUE;
  if (!aligned(x, 16) || !aligned(w4, 16) || !aligned(s_w_fp16, 8) || !aligned(y, 8) ||
      !aligned(workspace, 16))
    return FLEXQ_ERROR_UNSUPPORTED;
  const Range in[3] = {range_of(x, span(1, 0, M, x_stride, K, 2)),
                       range_of(w4, flexq_packed_w4_bytes(N, K)),
                       range_of(s_w_fp16, (uint64_t)N * (K / group_size) * 2)};
  const Range ry = range_of(y, (uint64_t)M * N * 2), ws = range_of(workspace, need);
  if (any_overlap(ry, {in[0], in[1], in[2], ws}) || any_overlap(ws, {in[0], in[1], in[2]}))
    return FLEXQ_ERROR_INVALID_VALUE;
  return launched(flexq::launch_gemv_w4(x, dtype == FLEXQ_BF16, x_stride, w4, s_w_fp16, M, N, K,
                                        group_size, workspace, y, (hipStream_t)stream));
}

flexq_status flexq_block_tables(const int32_t* ctx_lens, const int32_t* new_lens, int64_t B,
                                const int32_t* free_pages, int64_t num_free,
                                const int32_t* free_head, int32_t page_size,
                                int32_t* block_table, int64_t max_blocks, int64_t max_tokens,
                                int32_t* slot_map, int32_t* cu_new, int32_t* counts,
                                void* stream) {
  if (B < 0 || num_free < 0 || max_blocks < 0 || max_tokens < 0 || page_size <= 0)
    return FLEXQ_ERROR_INVALID_VALUE;
  if ((page_size & (page_size - 1)) != 0 || page_size > 65536 || B > flexq::kMaxRequests ||
      num_free > (1LL << 30) || max_blocks > (1LL << 30) || max_tokens > (1LL << 30))
    return FLEXQ_ERROR_UNSUPPORTED;
  if (!cu_new || !counts || (B > 0 && (!ctx_lens || !new_lens)) || (num_free > 0 && !free_pages) ||
      (B * max_blocks > 0 && !block_table) || (max_tokens > 0 && !slot_map))
    return FLEXQ_ERROR_INVALID_VALUE;
  if (!aligned(ctx_lens, 4) || !aligned(new_lens, 4) || !aligned(free_pages, 4) ||
      !aligned(free_head, 4) || !aligned(block_table, 4) || !aligned(slot_map, 4) ||
      !aligned(cu_new, 4) || !aligned(counts, 4))
    return FLEXQ_ERROR_UNSUPPORTED;
  const Range in[4] = {range_of(ctx_lens, 4 * B), range_of(new_lens, 4 * B),
                       range_of(free_pages, 4 * num_free), range_of(free_head, free_head ? 4 : 0)};
  const Range out[4] = {range_of(block_table, 4 * B * max_blocks),
                        range_of(slot_map, 4 * max_tokens), range_of(cu_new, 4 * (B + 1)),
                        range_of(counts, 12)};
  for (int i = 0; i < 4; ++i) {
    if (any_overlap(out[i], {in[0], in[1], in[2], in[3]})) return FLEXQ_ERROR_INVALID_VALUE;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return FLEXQ_ERROR_INVALID_VALUE;
  }
  return launched(flexq::launch_block_tables(ctx_lens, new_lens, B, free_pages, num_free,
                                             free_head, page_size, block_table, max_blocks,
                                             max_tokens, slot_map, cu_new, counts,
                                             (hipStream_t)stream));
}

flexq_status flexq_kv_cache_write(const uint16_t* k, int64_t k_stride_t, int64_t k_stride_h,
                                  const uint16_t* v, int64_t v_stride_t, int64_t v_stride_h,
                                  const int32_t* slot_map, int64_t T, int64_t Hkv, int64_t D,
                                  int64_t num_pages, int32_t page_size, uint16_t* k_cache,
                                  uint16_t* v_cache, void* stream) {
  if (T < 0 || k_stride_t < 0 || k_stride_h < 0 || v_stride_t < 0 || v_stride_h < 0)
    return FLEXQ_ERROR_INVALID_VALUE;
  FLEXQ_TRY(check_cache(num_pages, Hkv, D, page_size));
  if (Hkv > 65535 || T >= (1LL << 34) / D / Hkv + 1 || T * Hkv * D >= (1LL << 34))
    return FLEXQ_ERROR_UNSUPPORTED;
  if (T == 0) return FLEXQ_SUCCESS;
  if (!k || !v || !slot_map || (num_pages > 0 && (!k_cache || !v_cache)))
    return FLEXQ_ERROR_INVALID_VALUE;
  if (T == 1) k_stride_t = v_stride_t = 0;  // (never used)
  if (Hkv == 1) k_stride_h = v_stride_h = 0;
  if (k_stride_t % 8 || k_stride_h % 8 || v_stride_t % 8 || v_stride_h % 8 ||
      k_stride_t > kMaxStride || k_stride_h > kMaxStride || v_stride_t > kMaxStride ||
      v_stride_h > kMaxStride)
    return FLEXQ_ERROR_UNSUPPORTED;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slot_map, 4) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16))
    return FLEXQ_ERROR_UNSUPPORTED;
  const Range rk = range_of(k_cache, cache_bytes(num_pages, Hkv, D, page_size));
  const Range rv = range_of(v_cache, cache_bytes(num_pages, Hkv, D, page_size));
  const Range ik = range_of(k, span(T, k_stride_t, Hkv, k_stride_h, D, 2));
  const Range iv = range_of(v, span(T, v_stride_t, Hkv, v_stride_h, D, 2));
  const Range is = range_of(slot_map, 4 * T);
  if (any_overlap(rk, {rv, ik, iv, is}) || any_overlap(rv, {ik, iv, is}))
    return FLEXQ_ERROR_INVALID_VALUE;
  return launched(flexq::launch_kv_cache_write(k, k_stride_t, k_stride_h, v, v_stride_t,
                                               v_stride_h, slot_map, T, Hkv, D, num_pages,
                                               page_size, k_cache, v_cache, (hipStream_t)stream));
}

size_t flexq_tree_attention_workspace_bytes(int64_t B, int64_t max_new, int64_t H, int64_t Hkv,
                                            int64_t D) {
  if (check_attention_sizes(B, max_new, H, Hkv, D) != FLEXQ_SUCCESS || B == 0 || max_new == 0)
    return 0;
  return flexq::attention_workspace_bytes(B, max_new, H, Hkv, D);
}

flexq_status flexq_tree_attention(const uint16_t* q, int32_t dtype, int64_t q_stride_t,
                                  int64_t q_stride_h, const uint16_t* k_cache,
                                  const uint16_t* v_cache, int64_t num_pages, int32_t page_size,
                                  const int32_t* block_table, int64_t max_blocks,
                                  const int32_t* ctx_lens, const int32_t* cu_new, int64_t B,
                                  int64_t T, int64_t max_new, int64_t H, int64_t Hkv, int64_t D,
                                  const int32_t* tree_mask, int64_t mask_words, float scale,
                                  void* workspace, size_t workspace_bytes, uint16_t* out,
                                  float* lse, void* stream) {
  FLEXQ_TRY(check_dtype(dtype));
  if (T < 0 || q_stride_t < 0 || q_stride_h < 0 || max_blocks < 0 || mask_words < 0 ||
      !std::isfinite(scale))
    return FLEXQ_ERROR_INVALID_VALUE;
  FLEXQ_TRY(check_attention_sizes(B, max_new, H, Hkv, D));
  FLEXQ_TRY(check_cache(num_pages, Hkv, D, page_size));
  if (max_blocks > (1LL << 24) / page_size || T > (1LL << 24)) return FLEXQ_ERROR_UNSUPPORTED;
  if (tree_mask && max_new > 32 * mask_words) return FLEXQ_ERROR_INVALID_VALUE;
  if (mask_words > (1LL << 24)) return FLEXQ_ERROR_UNSUPPORTED;
  if (B == 0 || T == 0 || max_new == 0) return FLEXQ_SUCCESS;
  if (!q || !ctx_lens || !cu_new || !out || !workspace || (max_blocks > 0 && !block_table) ||
      num_pages == 0 || !k_cache || !v_cache)
    return FLEXQ_ERROR_INVALID_VALUE;
  if (workspace_bytes < flexq::attention_workspace_bytes(B, max_new, H, Hkv, D))
    return FLEXQ_ERROR_INVALID_VALUE;
  if (T == 1) q_stride_t = 0;  // (never used)
  if (H == 1) q_stride_h = 0;
  if (q_stride_t % 8 || q_stride_h % 8 || q_stride_t > kMaxStride || q_stride_h > kMaxStride)
    return FLEXQ_ERROR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(block_table, 4) || !aligned(ctx_lens, 4) || !aligned(cu_new, 4) ||
      !aligned(tree_mask, 4) || !aligned(workspace, 16) || !aligned(out, 16) || !aligned(lse, 4))
    return FLEXQ_ERROR_UNSUPPORTED;
  const uint64_t cache = cache_bytes(num_pages, Hkv, D, page_size);
  const Range in[7] = {range_of(q, span(T, q_stride_t, H, q_stride_h, D, 2)),
                       range_of(k_cache, cache),
                       range_of(v_cache, cache),
                       range_of(block_table, 4 * B * max_blocks),
                       range_of(ctx_lens, 4 * B),
                       range_of(cu_new, 4 * (B + 1)),
                       range_of(tree_mask, tree_mask ? 4 * T * mask_words : 0)};
  const Range ws = range_of(workspace, workspace_bytes);
  const Range ro = range_of(out, (uint64_t)T * H * D * 2);
  const Range rl = range_of(lse, lse ? (uint64_t)T * H * 4 : 0);
  for (const Range& r : in)
    if (any_overlap(r, {ws, ro, rl})) return FLEXQ_ERROR_INVALID_VALUE;
  if (overlap(ws, ro) || overlap(ws, rl) || overlap(ro, rl)) return FLEXQ_ERROR_INVALID_VALUE;
  flexq::AttentionArgs a;
  a.q = q;
  a.q_st = q_stride_t;
  a.q_sh = q_stride_h;
  a.kc = k_cache;
  a.vc = v_cache;
  a.num_pages = (int32_t)num_pages;
  a.page_shift = __builtin_ctz((unsigned)page_size);
  a.table = block_table;
  a.max_blocks = (int32_t)max_blocks;
  a.ctx = ctx_lens;
  a.cu = cu_new;
  a.B = (int32_t)B;
  a.T = (int32_t)T;
  a.max_new = (int32_t)max_new;
  a.H = (int32_t)H;
  a.Hkv = (int32_t)Hkv;
  a.D = (int32_t)D;
  a.mask = tree_mask;
  a.mask_words = (int32_t)mask_words;
  a.scale = scale;
  a.workspace = workspace;
  a.out = out;
  a.lse = lse;
  return launched(flexq::launch_tree_attention(a, dtype == FLEXQ_BF16, (hipStream_t)stream));
}

}  // extern "C"
