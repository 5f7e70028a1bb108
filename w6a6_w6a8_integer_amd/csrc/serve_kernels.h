// serve_kernels.h -- host-side launchers of the decoding-step kernels (internal to
// libflexq).  Arguments are already validated by the C ABI layer (serve_api.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace flexq {

hipError_t launch_pack_w4(const uint16_t* w, bool bf16, int64_t N, int64_t K, int group,
                          uint32_t* w4, uint16_t* sw, hipStream_t stream);

hipError_t launch_gemv_w4(const uint16_t* x, bool bf16, int64_t x_stride, const uint32_t* w4,
                          const uint16_t* sw, int64_t M, int64_t N, int64_t K, int group,
                          void* workspace, uint16_t* y, hipStream_t stream);
size_t gemv_w4_workspace_bytes(int64_t M, int64_t N, int64_t K);

// most requests a step holds (their prefix sums sit in LDS)
constexpr int64_t kMaxRequests = 4096;

hipError_t launch_block_tables(const int32_t* ctx, const int32_t* add, int64_t B,
                               const int32_t* free_pages, int64_t num_free, const int32_t* head,
                               int page_size, int32_t* table, int64_t max_blocks,
                               int64_t max_tokens, int32_t* slots, int32_t* cu, int32_t* counts,
                               hipStream_t stream);

hipError_t launch_kv_cache_write(const uint16_t* k, int64_t k_st, int64_t k_sh,
                                 const uint16_t* v, int64_t v_st, int64_t v_sh,
                                 const int32_t* slots, int64_t T, int64_t Hkv, int64_t D,
                                 int64_t num_pages, int page_size, uint16_t* kc, uint16_t* vc,
                                 hipStream_t stream);

// What a tree attention call works on (flexq_serve.h has the meaning of each).
struct AttentionArgs {
  const uint16_t* q;
  int64_t q_st, q_sh;
  const uint16_t* kc;
  const uint16_t* vc;
  int32_t num_pages, page_shift;
  const int32_t* table;
  int32_t max_blocks;
  const int32_t* ctx;
  const int32_t* cu;
  int32_t B, T, max_new, H, Hkv, D;
  const int32_t* mask;
  int32_t mask_words;
  float scale;
  void* workspace;
  uint16_t* out;
  float* lse;
};

size_t attention_workspace_bytes(int64_t B, int64_t max_new, int64_t H, int64_t Hkv, int64_t D);
hipError_t launch_tree_attention(const AttentionArgs& a, bool bf16, hipStream_t stream);

}  // namespace flexq
