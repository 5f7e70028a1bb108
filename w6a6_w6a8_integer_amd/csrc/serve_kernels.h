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
  // What starting on a request costs, in 32-key steps, and the least share of a workgroup
  // (counting no start: 32 single tokens over 4k 57 us against 54; shares down to one step: a
  // single token over 37 10.1 us, as then there is a join, against 8.2).
  static constexpr uint32_t kHead = 5, kMinShare = 8;
  static constexpr bool kWindowed = false, kScaledReference = false;
  __host__ __device__ static constexpr uint32_t least_share() { return kMinShare; }
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

// The same over a 4-bit cache: kc and vc hold codes, and keys of the context before the last
// `window` of a token's positions are left out, but for the first `sinks` (window 0: none are).
struct Kv4AttentionArgs : AttentionArgs {
  // (steps of a quarter of the bytes: 32 single tokens over 4k 24.0 us, a window of 4k on eight requests
  // 38.7, trees of seven over 8k 80.0; with 5 and 8 as above 25.5, 39.8, 81.7, with 3 and 8 28.3, 40.7, 81.0)
  static constexpr uint32_t kHead = 16;
  uint32_t key_waves;  // waves that take a share's steps in turn, four each at the least
  __host__ __device__ uint32_t least_share() const { return 4 * key_waves; }
  static constexpr bool kWindowed = true, kScaledReference = true;
  uint32_t group, group_inverse;  // H / Hkv, floor(2^32 / group) (less one for a group of one)
  const uint16_t* scales;
  int32_t window, sinks;
};

size_t kv4_attention_workspace_bytes(int64_t B, int64_t max_new, int64_t H, int64_t Hkv,
                                     int64_t D);
hipError_t launch_kv4_attention(const Kv4AttentionArgs& a, bool bf16, hipStream_t stream);

hipError_t launch_kv4_cache_write(const uint16_t* k, int64_t k_st, int64_t k_sh,
                                  const uint16_t* v, int64_t v_st, int64_t v_sh, bool bf16,
                                  const int32_t* slots, int64_t T, int64_t Hkv, int64_t D,
                                  int64_t num_pages, int page_size, uint32_t* kc, uint32_t* vc,
                                  uint16_t* scales, hipStream_t stream);
hipError_t launch_kv4_cache_read(const uint32_t* kc, const uint32_t* vc, const uint16_t* scales,
                                 const int32_t* slots, int64_t T, int64_t Hkv, int64_t D,
                                 int64_t num_pages, int page_size, bool bf16, uint16_t* k,
                                 uint16_t* v, hipStream_t stream);

// What a lora_add call works on; h is the workspace, fp32 [slices][T][R padded].
struct LoraArgs {
  const uint16_t* x;
  int64_t x_st;
  const uint16_t* y;
  int64_t y_st;
  const int32_t* adapters;
  const uint16_t* a;
  const uint16_t* b;
  const int32_t* ranks;
  const float* scales;
  int64_t T;
  int32_t N, K, R, L;
  float* h;
  uint16_t* out;
  int64_t out_st;
};

size_t lora_workspace_bytes(int64_t T, int64_t N, int64_t K, int64_t R, int64_t L);
hipError_t launch_lora(const LoraArgs& a, bool bf16, hipStream_t stream);

}  // namespace flexq
