// serve_attention.hip -- attention of drafted tokens over the paged cache.
//
// For the rows of one request and key head (new tokens x query heads of the group), with
// K and V of up to ctx + new tokens: S = scale K Q^T, P = 2^(S log2 e - m + c) with a running
// maximum m per row and a constant c, O = V^T P, l = sum P; out = O / l.  One pass over the cache.
//
// Both products are MFMAs with the rows as columns, so a lane owns one row's statistics: a
// wave holds 16 rows (16x16x32) or, where there are many, 32 (32x32x16: half the
// instructions for the same rows).  D of K Q^T gives a lane the scores of its row at some
// keys, and the fragment of P that V^T P takes wants eight consecutive keys of that row.
// The keys of a 32-key step are dealt to the score tiles' rows so that they are the same
// eight, and no exchange between lanes is needed:
//   16 rows: row r of score tile t holds key 8 (r / 4) + 4 t + r % 4; lane l ends up with
//            keys 8 (l / 16) .. + 7;
//   32 rows: row r holds the key with bits 2 and 3 of r swapped; lane l ends up with keys
//            16 j + 8 (l / 32) .. + 7, j = 0, 1.
//
// Bound by HBM's reads of the cache, for many rows nearly as much by the MFMAs and the
// exponentials beside them.  Measured (8 key heads of 128, 64 heads): 32 single tokens over
// up to 4k tokens 54 us, 5.3 TB/s; 24 requests of up to 13 over 8k 95 us, 4.9 TB/s; 2 of up to
// 9 over 128k 184 us, 5.0 TB/s and 344 TFLOP/s.
#include "serve_plan.h"

namespace flexq {

namespace {

constexpr int kWaves = 4;
// Workgroups a compute unit holds: two by LDS (4 stages of 2 D 64 bytes, 2 where D = 256),
// on 64-wide heads as many as registers allow (48 rows of 40 heads: 30 us against 32 with two;
// 110 rows, three: 45 against 49, and 55 with a fourth that waits for the others).
constexpr int units_per_cu(int64_t D, int rows) { return D > 64 ? 2 : rows == 16 ? 4 : 3; }

typedef __attribute__((address_space(1))) const void* global_ptr_t;

}  // namespace

// 0xFFFF in each 16-bit half of v that is infinite or NaN.
template <class E>
__device__ __forceinline__ uint32_t not_finite(uint32_t v) {
  return ((v & E::kExponent) == E::kExponent ? 0xFFFFu : 0u) |
         (((v >> 16) & E::kExponent) == E::kExponent ? 0xFFFF0000u : 0u);
}

// A wave's products for RW rows and one 32-key step of 2 DT fragments of keys and values.
template <class E, int DT, int RW>
struct Products;

// 16 rows: key fragments [tile t][32-wide slice of D], value fragments [16-wide slice]
template <class E, int DT>
struct Products<E, DT, 16> {
  static constexpr int kGroups = 1;  // of eight keys, a lane's
  typedef f32x4 Out;
  static constexpr int kOuts = 2 * DT;   // tiles of O, four consecutive d a lane and quad
  // first key of a lane's group in the step
  static __device__ __forceinline__ int key(int lane, int) { return 8 * (lane >> 4); }
  // the lane (of row c) and the group that hold key k
  static __device__ __forceinline__ int lane_of(int k, int c) { return (k >> 3) * 16 + c; }
  static __device__ __forceinline__ int group_of(int) { return 0; }
  // first d of a lane's slice of Q for k-step i
  static __device__ __forceinline__ int slice(int lane, int i) { return 32 * i + 8 * (lane >> 4); }
  static constexpr int kSlices = DT;
  // index of four consecutive d: quad g of tile t
  static __device__ __forceinline__ int d4(int lane, int t, int) { return 4 * t + (lane >> 4); }
  static constexpr int kQuads = 1;
  // half of the step whose block a staged fragment's lane reads, and where in the block
  static __device__ __forceinline__ int half(int lane, int wave) {
    return wave < 2 ? (lane >> 3) & 1 : lane >> 5;
  }
  static __device__ __forceinline__ int offset(int lane, int wave) {
    const int c = lane & 15, p = lane >> 4;
    return wave < 2 ? (8 * ((c >> 2) & 1) + 4 * wave + (c & 3)) * 32 + 8 * p
                    : (wave - 2) * DT * 256 + c * 16 + 8 * (p & 1);
  }
  static constexpr int kValueStep = 256;  // elements between a value wave's fragments
  static __device__ __forceinline__ void scores(const u32x4* k, const u32x4 (&q)[kSlices],
                                                float (&x)[8]) {
    const int lane = threadIdx.x & 63;
    u32x4 f[2 * DT];
#pragma unroll
    for (int i = 0; i < 2 * DT; ++i) f[i] = k[i * 64 + lane];
    f32x4 s[2] = {};
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int t = 0; t < 2; ++t) s[t] = E::mfma(f[t * DT + i], q[i], s[t]);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = s[e >> 2][e & 3];
  }
  // O += V^T P for one fragment; `group` is 0 and `t` the tile of O
  static constexpr int kValues = 2 * DT;
  static __device__ __forceinline__ constexpr int tile(int i) { return i; }
  static __device__ __forceinline__ constexpr int group(int) { return 0; }
  static __device__ __forceinline__ Out mfma(u32x4 v, u32x4 p, Out o) { return E::mfma(v, p, o); }
};

// 32 rows: keys as they lie in their two 16-token blocks (the 16-byte pieces of a
// kilobyte placed so that a fragment's rows meet different banks: piece q of row r at slot
// 4 r + (q ^ r / 4)), value fragments [block][32-wide slice]
template <class E, int DT>
struct Products<E, DT, 32> {
  static constexpr int kGroups = 2;
  typedef f32x16 Out;
  static constexpr int kOuts = DT;
  static __device__ __forceinline__ int key(int lane, int j) { return 16 * j + 8 * (lane >> 5); }
  static __device__ __forceinline__ int lane_of(int k, int c) { return ((k >> 3) & 1) * 32 + c; }
  static __device__ __forceinline__ int group_of(int k) { return k >> 4; }
  static __device__ __forceinline__ int slice(int lane, int i) { return 16 * i + 8 * (lane >> 5); }
  static constexpr int kSlices = 2 * DT;
  static __device__ __forceinline__ int d4(int lane, int t, int g) {
    return 8 * t + 2 * g + (lane >> 5);
  }
  static constexpr int kQuads = 4;
  static __device__ __forceinline__ int half(int, int wave) { return wave & 1; }
  static __device__ __forceinline__ int offset(int lane, int wave) {
    const int r = lane >> 2;
    return wave < 2 ? r * 32 + ((lane & 3) ^ (r >> 2)) * 8 : (lane & 31) * 16 + 8 * (lane >> 5);
  }
  static constexpr int kValueStep = 512;
  static __device__ __forceinline__ void scores(const u32x4* k, const u32x4 (&q)[kSlices],
                                                float (&x)[16]) {
    const int lane = threadIdx.x & 63, c = lane & 31, h = lane >> 5;
    const int key = (c & 19) | (c & 4) << 1 | (c & 8) >> 1, r = key & 15;
    const u32x4* row = k + (key >> 4) * (DT * 64) + 4 * r;
    u32x4 f[2 * DT];
#pragma unroll
    for (int i = 0; i < 2 * DT; ++i)
      f[i] = row[(i >> 1) * 64 + (((i & 1) * 2 + h) ^ (r >> 2))];
    f32x16 s = {};
#pragma unroll
    for (int i = 0; i < 2 * DT; ++i) s = E::mfma32(f[i], q[i], s);
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = s[e];
  }
  static constexpr int kValues = 2 * DT;
  static __device__ __forceinline__ constexpr int tile(int i) { return i % DT; }
  static __device__ __forceinline__ constexpr int group(int i) { return i / DT; }
  static __device__ __forceinline__ Out mfma(u32x4 v, u32x4 p, Out o) {
    return E::mfma32(v, p, o);
  }
};

// One workgroup = one share of the cache, key head and block of 4 RW rows, RW a wave.
//
// The four waves stage the fragments of a 32-key step in LDS (a quarter each, straight
// from memory) and every wave reads all of them for its own rows.  S stages: the loads
// of S - 1 steps are on their way while one is worked on, and one barrier a step tells
// that a step has come and that the one before has been read.
//
// ONE: there is one row block, nobody reads the cache's lines again, and they are not kept
// (32 single tokens over 4k: 54 us against 62 when they are, 24 of 13 over 8k 96 and 110, 2 of 9
// over 128k 189 and 193; but 8 of 48 over 2k, 40 heads of 64, 29.6 and 28.1).
template <class E, int DT, int RW, int S, bool ONE>
__global__ __launch_bounds__(64 * kWaves, 2) void tree_attention_kernel(const AttentionArgs a,
                                                                        int shares,
                                                                        int row_blocks) {
  using P = Products<E, DT, RW>;
  constexpr int D = 32 * DT;
  constexpr int kStage = 4 * DT * 1024;  // bytes: 2 DT fragments of keys, 2 DT of values
  constexpr int kKeys = 8 * P::kGroups;  // scores a lane holds
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  int& again = *reinterpret_cast<int*>(lds + S * kStage);  // (behind the stages)
  if (threadIdx.x == 0) again = 0;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & (RW - 1);
  // Workgroups 8 apart share an XCD: the row blocks that read the same keys do.
  const int id = blockIdx.x;
  const int unit = id / (8 * row_blocks) * 8 + id % 8;
  const int hk = unit % a.Hkv;
  const uint32_t share = unit / a.Hkv;
  const int block_row0 = id / 8 % row_blocks * (kWaves * RW);
  int b;
  uint32_t before;
  Window window;
  const Plan plan = make_plan(a, shares, share, b, before, window);
  if (b >= a.B) return;
  const uint32_t share_begin = plan.start(share), share_end = plan.start(share + 1);
  const int group = a.H / a.Hkv;
  const Parts parts = parts_of(a, shares, a.max_new * group);
  const int per_page = 1 << (a.page_shift - 4);  // 16-token blocks of a page
  // A negative scale goes into the queries' signs and a zero one into the queries, so that
  // the scores' order is the scaled ones'.  A row's reference m is a whole number, the
  // scores' maximum rounded up, and raised only where a score exceeds it by E::kLag: l and O are
  // in proportion to 2^(E::kTop - m) whatever m is, and change by powers of 2.
  const float scale = a.scale != 0.0f ? fabsf(a.scale) * kLog2e : 1.0f;
  // what is added to a row's scaled scores (m = -inf: nothing attended yet)
  auto reference = [&](float m) { return m == -INFINITY ? 0.0f : E::kTop - m; };
  const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
  const uint32_t keep_q = a.scale != 0.0f ? 0xFFFFFFFFu : 0u;

  // what a lane takes of a step's fragments: half of the step, and where in a block
  const bool key_wave = wave < 2;
  const int half = P::half(lane, wave);
  const uint16_t* src = (key_wave ? a.kc : a.vc) + P::offset(lane, wave);

  // Once; and where some sum is not finite a second time, with infinite and NaN values taken
  // out of every step and given to the rows that attend them.  (The first time they meet both
  // parts of a probability, and where one is 0 an infinity makes NaN.)
  const int first_b = b;
  const uint32_t first_before = before;
  for (bool careful = false;; careful = true) {
    for (b = first_b, before = first_before; b < a.B && before < share_end; ++b) {
      if ((uint32_t)(b - window.base) >= 64u) {
        window.base = b;
        window.mine = load_request(a, b + lane);
      }
      const Request r = window.at<AttentionArgs>(b);
      const uint32_t weight = r.weight<AttentionArgs>();
      if (weight == 0) continue;
      const int cu = r.cu, n_new = r.n_new, ctx = r.ctx, len = r.len, steps = (int)r.steps();
      // this share's steps of the request
      const uint32_t first_step = before + a.kHead;
      const int begin = share_begin > first_step ? (int)(share_begin - first_step) : 0;
      const int own_end = min(steps, (int)(share_end - first_step));
      before += weight;
      if (own_end <= begin) continue;
      const uint32_t s0 = plan.share_of(first_step), s1 = plan.share_of(first_step + steps - 1);
      if (threadIdx.x == 0 && hk == 0 && block_row0 == 0 && share == s0)
        parts.plan[b] = {(int)s0, (int)s1};
      const int rows = n_new * group;
      if (block_row0 >= rows) continue;
      int end = own_end;
      if (!a.mask) {  // a chain: nothing past the last row's token
        const int last = min(block_row0 + kWaves * RW, rows) - 1;
        end = min(end, (ctx + last / group + 32) >> 5);
      }
      // where the last waves have fewer rows, a compute unit's next workgroup turns them round
      const int row0 = block_row0 + (id >> 8 & 1 ? kWaves - 1 - wave : wave) * RW;
      const bool idle = row0 >= rows;  // a wave that only stages

      const int row = row0 + c, tok = row / group;  // the lane's row, its token in the request
      const int64_t tok_at = (int64_t)cu + tok;     // and that token's place in q
      const bool in = row < rows && tok_at >= 0 && tok_at < a.T;
      u32x4 qf[P::kSlices];
      const uint16_t* q = a.q + tok_at * a.q_st + (int64_t)(hk * group + row % group) * a.q_sh;
#pragma unroll
      for (int i = 0; i < P::kSlices; ++i)
        qf[i] = in ? *reinterpret_cast<const u32x4*>(q + P::slice(lane, i)) : u32x4{};

      // Table entry of the 16 tokens at 32 step + 16 half (-1 past the request's tokens), and
      // the 16-token block of the cache it stands for (-1 where there is none).
      const scalar_ptr_t table = (scalar_ptr_t)(a.table + (int64_t)b * a.max_blocks);
      auto page_of = [&](int step, int half) {
        const int pos = min(step, end - 1) * 32 + half * 16;
        return pos < len ? table[pos >> a.page_shift] : -1;
      };
      auto block_of = [&](int id, int step, int half) {
        if ((unsigned)id >= (unsigned)a.num_pages) return -1;
        return (id * a.Hkv + hk) * per_page + ((step * 2 + half) & (per_page - 1));
      };
      // Stages a step whose table entries are in id0, id1, and fetches the next step's.
      // holes: bit 2 (step % 32) + half where there is no block.
      int id0 = page_of(begin, 0), id1 = page_of(begin, 1);
      uint64_t holes = 0;
      auto stage = [&](int step) {
        const int b0 = block_of(id0, step, 0), b1 = block_of(id1, step, 1);
        const int at = 2 * (step & 31);
        holes = (holes & ~(3ull << at)) | (uint64_t)((b0 < 0 ? 1 : 0) | (b1 < 0 ? 2 : 0)) << at;
        const uint16_t* from = src + (int64_t)max(half ? b1 : b0, 0) * (16 * D);
        char* to = lds + (step % S) * kStage + wave * (DT * 1024);
#pragma unroll
        for (int i = 0; i < DT; ++i)
          __builtin_amdgcn_global_load_lds(
              (global_ptr_t)(from + i * (key_wave ? 512 : P::kValueStep)),
              (lds_ptr_t)(to + i * 1024), 16, 0, ONE ? kNonTemporal : 0);
        id0 = page_of(step + 1, 0);
        id1 = page_of(step + 1, 1);
      };

      typename P::Out o[P::kOuts] = {};
      float m = -INFINITY, l = 0.0f;

      lds_barrier();  // the stages of the request before have been read
      // S - 1 steps, the last again where there are fewer: with a fixed number of loads behind
      // it the wait for q (before the loop, not in it) leaves them in flight.
#pragma unroll
      for (int i = 0; i < S - 1; ++i) stage(begin + i);
      wait_vm<(S - 1) * DT>();
#pragma unroll
      for (int i = 0; i < P::kSlices; ++i) {
        asm volatile("" : "+v"(qf[i]));
        qf[i] = (qf[i] & keep_q) ^ flip;
      }
      for (int step = begin; step < end; ++step) {
        if (end - step >= S - 1)
          wait_vm<(S - 2) * DT>();
        else
          wait_vm<0>();
        lds_barrier();
        if (step + S - 1 < end) stage(step + S - 1);
        if (idle) continue;
        const u32x4* kf = reinterpret_cast<const u32x4*>(lds + (step % S) * kStage);
        const u32x4* vf = kf + 2 * DT * 64 + lane;

        // S = K Q^T; then the values' fragments are on their way while P is formed
        float x[kKeys];
        P::scores(kf, qf, x);
        __builtin_amdgcn_sched_barrier(0);
        u32x4 f[P::kValues];
#pragma unroll
        for (int i = 0; i < P::kValues; ++i) f[i] = vf[i * 64];
        __builtin_amdgcn_sched_barrier(0);

        // Keys that are no context (drafted, or none at all) or on no page: the wave masks.
        const uint32_t hole = (uint32_t)(holes >> (2 * (step & 31))) & 3u;
        const bool masked = careful || hole != 0 || step * 32 + 32 > ctx;
        uint32_t seen[P::kGroups];   // attended keys among each eight of this lane's
        uint32_t there[P::kGroups];  // keys that exist
        bool poison = false;         // a value is infinite or NaN
        if (masked) {
#pragma unroll
          for (int j = 0; j < P::kGroups; ++j) {
            const int key0 = P::key(lane, j);          // the group's first key in the step
            const int j0 = step * 32 + key0 - ctx;     // its drafted index (may be negative)
            there[j] = (hole >> (key0 >> 4)) & 1u ? 0u : low_bits(len - step * 32 - key0);
            if (a.mask) {  // the context, then the tree's bits
              seen[j] = low_bits(-j0);
              if (j0 > -8 && in) {
                const int32_t* words = a.mask + tok_at * a.mask_words;
                const int w = j0 >> 5;
                const uint32_t w0 = w >= 0 && w < a.mask_words ? (uint32_t)words[w] : 0u;
                const uint32_t w1 = w + 1 < a.mask_words ? (uint32_t)words[w + 1] : 0u;
                seen[j] |= (uint32_t)(((uint64_t)w1 << 32 | w0) >> (j0 & 31)) & 0xFFu;
              }
            } else {  // a chain: the tokens up to the row's own
              seen[j] = low_bits(tok + 1 - j0);
            }
            seen[j] &= there[j];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (!((seen[j] >> e) & 1u)) x[8 * j + e] = -INFINITY;
          }
          // values of keys that do not exist are zeroed, and infinite and NaN ones for now
          bool bad = false;
#pragma unroll
          for (int i = 0; i < P::kValues; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t t = there[P::group(i)] >> (2 * k);
              const uint32_t w = f[i][k] & ((t & 1u) * 0xFFFFu | (t >> 1 & 1u) * 0xFFFF0000u);
              const uint32_t ex = not_finite<E>(w);
              bad |= ex != 0;
              f[i][k] = w & ~ex;
            }
          poison = __ballot(bad) != 0;
        }

        float top = x[0];
#pragma unroll
        for (int e = 1; e < kKeys; ++e) top = fmaxf(top, x[e]);
        top = row_max<RW>(top);
        top *= scale;
        if (__ballot(top > m + E::kLag)) {  // rare after a request's first step
          top = fmaxf(m, ceilf(top));
          const float by = m - (top == -INFINITY ? 0.0f : top);
          m = top;
          l = scaled(l, by);
#pragma unroll
          for (int t = 0; t < P::kOuts; ++t)
#pragma unroll
            for (int i = 0; i < 4 * P::kQuads; ++i) o[t][i] = scaled(o[t][i], by);
        }
        const float ref = reference(m);
        u32x4 hi[P::kGroups], lo[P::kGroups];
#pragma unroll
        for (int j = 0; j < P::kGroups; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float v0 = __builtin_amdgcn_exp2f(fmaf(x[8 * j + 2 * i], scale, ref));
            const float v1 = __builtin_amdgcn_exp2f(fmaf(x[8 * j + 2 * i + 1], scale, ref));
            l += v0 + v1;
            const u32x2 both = E::split(v0, v1);
            hi[j][i] = both[0];
            lo[j][i] = both[1];
          }

#pragma unroll
        for (int i = 0; i < P::kValues; ++i) {
          auto& to = o[P::tile(i)];
          to = P::mfma(f[i], hi[P::group(i)], to);
        }
#pragma unroll
        for (int i = 0; i < P::kValues; ++i) {
          auto& to = o[P::tile(i)];
          to = P::mfma(f[i], lo[P::group(i)], to);
        }
        if (!poison) continue;
        // Infinite and NaN values reach only the rows that attend their keys: one key at a
        // time, and a row that does not attend it keeps its sum.
#pragma unroll 1
        for (int k = 0; k < 32; ++k) {
          const int e = k & 7, from = P::lane_of(k, c);
#pragma unroll
          for (int j = 0; j < P::kGroups; ++j) {
            if (P::group_of(k) != j) continue;
            const bool mine = lane == from && ((there[j] >> e) & 1u);
            // (any attended key's probability is positive, also one too small for fp32)
            const u32x4 one_p = {mine ? E::kOne : 0u, 0u, 0u, 0u};
            const bool attends = (__shfl((int)seen[j], from) >> e) & 1;
#pragma unroll
            for (int i = 0; i < P::kValues; ++i) {
              if (P::group(i) != j) continue;
              const uint32_t v = mine ? reinterpret_cast<const uint16_t*>(vf + i * 64)[e] : 0u;
              const u32x4 one_v = {v & not_finite<E>(v), 0u, 0u, 0u};
              auto& to = o[P::tile(i)];
              const auto with = P::mfma(one_v, one_p, to);
#pragma unroll
              for (int t = 0; t < 4 * P::kQuads; ++t) to[t] = attends ? with[t] : to[t];
            }
          }
        }
      }
      f32x4 finite = {};  // or NaN
#pragma unroll
      for (int t = 0; t < P::kOuts; ++t)
#pragma unroll
        for (int i = 0; i < 4 * P::kQuads; ++i)
          finite[i & 3] = fmaf(o[t][i], 0.0f, finite[i & 3]);
      if (__ballot(finite[0] + finite[1] + finite[2] + finite[3] != 0.0f)) again = 1;

      const float sum = row_sum<RW>(l);
      const float top = m == -INFINITY ? m : -reference(m);
      if (row >= rows) continue;
#pragma unroll
      for (int t = 0; t < P::kOuts; ++t)
#pragma unroll
        for (int g = 0; g < P::kQuads; ++g) {
          const int d4 = P::d4(lane, t, g);
          const f32x4 v = {o[t][4 * g], o[t][4 * g + 1], o[t][4 * g + 2], o[t][4 * g + 3]};
          if (s0 != s1) {
            const int64_t place = 2 * (int64_t)share + (share == s0 ? 1 : 0);
            const int64_t at = (place * a.Hkv + hk) * (a.max_new * group) + row;
            parts.out[at * (D / 4) + d4] = v;
            if (d4 == 0) parts.stat[at] = {top, sum};
          } else if (in) {
            write_row<E>(a, tok_at, hk * group + row % group, d4, v, top == -INFINITY ? 0.0f : top,
                         sum);
          }
        }
    }
    lds_barrier();
    if (careful || again == 0) break;
  }
}

namespace {

// How a call is laid out: rows a wave holds, row blocks, shares of the cache
struct Layout {
  int rows, row_blocks, shares;
};

Layout layout_of(int64_t max_new, int64_t H, int64_t Hkv, int64_t D) {
  Layout p;
  const int64_t rows = max_new * (H / Hkv);
  // 32 rows a wave halve the LDS reads and MFMAs for many rows, and are half empty for few (up
  // to 104 rows: 97 us against 126 with 16; 72 rows over 128k: 189 against 227; but 48 rows:
  // 32 us against 30, one row 9.0 against 8.2).  256-wide heads have no registers for them.
  p.rows = rows <= 4 * 16 || D > 128 ? 16 : 32;
  p.row_blocks = (int)((rows + kWaves * p.rows - 1) / (kWaves * p.rows));
  const int64_t target = units_per_cu(D, p.rows) * device_cu_count();
  const int64_t units = Hkv * p.row_blocks;
  p.shares = (int)std::max<int64_t>(1, target / units);
  return p;
}

template <class E, int DT>
hipError_t launch_rows(const AttentionArgs& a, hipStream_t stream) {
  // stages: what two workgroups' share of a compute unit's LDS holds
  constexpr int S = DT <= 4 ? 4 : 2;
  Layout p = layout_of(a.max_new, a.H, a.Hkv, a.D);
  // no more shares than the tables' room can fill (short contexts: one, and no join)
  const int64_t room = a.kHead + (((int64_t)a.max_blocks << a.page_shift) + 31) / 32;
  p.shares = (int)std::min<int64_t>(p.shares, std::max<int64_t>(1, a.B * room / a.kMinShare));
  const int64_t units = (int64_t)p.shares * a.Hkv;
  const dim3 grid((unsigned)((units + 7) / 8 * 8 * p.row_blocks));
  const bool one = p.row_blocks == 1;
  auto* kernel = tree_attention_kernel<E, DT, 16, S, true>;
  if constexpr (DT > 4) {
    if (!one) kernel = tree_attention_kernel<E, DT, 16, S, false>;
  } else if (p.rows == 32) {  // (16 rows a wave are one row block)
    kernel = one ? tree_attention_kernel<E, DT, 32, S, true>
                 : tree_attention_kernel<E, DT, 32, S, false>;
  }
  const hipError_t e = launch_kernel_lds(kernel, grid, dim3(64 * kWaves), S * 4 * DT * 1024 + 16,
                                         stream, a, p.shares, p.row_blocks);
  if (e != hipSuccess || p.shares == 1) return e;
  return launch_join<AttentionArgs, E, DT>(a, p.shares, stream);
}

template <class E>
hipError_t launch_width(const AttentionArgs& a, hipStream_t stream) {
  switch (a.D) {
    case 64: return launch_rows<E, 2>(a, stream);
    case 96: return launch_rows<E, 3>(a, stream);
    case 128: return launch_rows<E, 4>(a, stream);
    default: return launch_rows<E, 8>(a, stream);
  }
}

}  // namespace

size_t attention_workspace_bytes(int64_t B, int64_t max_new, int64_t H, int64_t Hkv, int64_t D) {
  return parts_bytes(B, max_new, H, D, layout_of(max_new, H, Hkv, D).shares);
}

hipError_t launch_tree_attention(const AttentionArgs& a, bool bf16, hipStream_t stream) {
  return bf16 ? launch_width<Bfloat>(a, stream) : launch_width<Half>(a, stream);
}

}  // namespace flexq
