// serve_kv4_attention.hip -- attention of drafted tokens over a paged cache of 4-bit codes, with
// an optional sliding window whose first tokens stay visible.
//
// A key is k = b + s c with codes c = 0 .. 15 and a scale and an offset for its token and head, a
// value likewise.  For a row with queries q, Q = sum q, and w_j = p_j s_j, W = sum w_j:
//   q.k = s (q.(64 + c) - 64 Q) + b Q
//   sum_j p_j v_j = sum_j w_j (c_j - 8) + 8 W + sum_j p_j b_j
// so both products are MFMAs on whole numbers that fp16 holds, whatever the tensors' type, and the
// scales meet scores and probabilities.  A key's code enters as 64 + c (its bits under 64's exponent: one
// and-or a pair) with -64 Q as what the MFMAs begin from; that errs by D / 32 roundings of at
// most (64 + 79) sum|q|, less than sums of q.(c - 8) and 8 Q are allowed.  A value's enters as c - 8 (or
// 16 (c - 8), of the next four bits), an and-or and an addition a pair: sums over a long context of
// codes of one sign would err with their size, not with their result's.
//
// In how many bits: scores, statistics and sums are fp32.  The queries enter as fp16 after a row's power of
// two, whole down to 2^-24 of the row's largest and below within 2^-34 of it.  w_j enters as the sum of two
// fp16 parts, within 2^-22 of itself or 2^-35 of the row's largest, whichever is more, for bfloat16 rows
// too: values that cancel leave what a weight errs by alone in the output, where one part's 2^-11 is
// no longer under the rounding's 2^-8.  W sums the very parts that meet the codes, so that what a weight
// errs by meets its value's s c alone.
//
// A wave stages its own 32-key steps in LDS straight from memory, S - 1 of them on their way while one
// is worked on, and needs no barrier until a request's end.  Rows are
// columns of the MFMAs (16 a group), so a lane owns one row's statistics, and the keys are
// dealt to the score tiles' rows so that a lane's scores are those that its fragment of P takes:
// row r of score tile t holds key 8 (r / 4) + 4 t + r % 4, lane l keys 8 (l / 16) .. + 7.  Waves
// that the rows leave over take the steps in turn and add up in LDS; columns that they leave over
// hold the same rows again, each for a part of a step's keys, so that few rows do not pay for 16.
//
// What bounds it: two contexts of 128k, 64 heads on 8, 52 us (4.7 TB/s of the cache's bytes; its loads
// alone 41, its arithmetic alone 42); a window of 4k on eight requests of 40 heads 39 (4.6; 33 and 35).  Many
// short requests and trees of many rows wait for chains of latencies (a step's LDS reads, MFMAs, exponentials,
// the look for what leaves fp16's range) with two or three waves a SIMD: 32 single tokens over 4k 24 us (3.2
// TB/s; loads 18, arithmetic 22), trees of seven over 8k 80 (loads 36, arithmetic 79: vector units busy half of
// the time, MFMAs a fifth).
#include <type_traits>

#include "serve_plan.h"

namespace flexq {

namespace {

constexpr int kWaves = 4;
typedef __attribute__((address_space(1))) const void* global_ptr_t;
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// A row's largest w is held as 2^(kTop - 1) to 2^(kTop + kLag): fp16 reaches no further up, and
// down to 2^-24, so that small ones keep their bits.
constexpr float kTop = 11.0f, kLag = 4.0f;
constexpr uint16_t kMostBits = (15 + 11 + 4) << 10;  // 2^(kTop + kLag) in fp16

// Workgroups a compute unit holds.
constexpr int units_per_cu(int64_t D, int groups) { return groups == 1 && D <= 128 ? 3 : 2; }

// (by value: a bit cast of a vector's element takes the whole vector's first bits)
__device__ __forceinline__ f16x2 pair_of(uint32_t v) { return __builtin_bit_cast(f16x2, v); }

// Eight codes of a dword as four pairs of halves.  The constants sit in registers: as literals they
// would take an and and an or.
struct Codes {
  uint32_t base64 = 0x54005400u, base1024 = 0x64006400u;
  uint32_t low_bits = 0x000F000Fu, high_bits = 0x00F000F0u;
  __device__ __forceinline__ Codes() {
    asm("" : "+v"(base64));
    asm("" : "+v"(base1024));
    asm("" : "+s"(low_bits));
    asm("" : "+s"(high_bits));
  }
  // 64 + c, pairs in the order of a key's dword: the bits below 64's exponent are the halves' bits
  // 4 to 7, so three shifts and four and-ors
  __device__ __forceinline__ u32x4 key(uint32_t w) const {
    return u32x4{(w << 4 & high_bits) | base64, (w & high_bits) | base64,
                 (w >> 4 & high_bits) | base64, (w >> 8 & high_bits) | base64};
  }
  // c - 8 from the low four bits of the bytes, 16 (c - 8) from the high ones: (1024 + c) - 1032 and
  // (1024 + 16 c) - 1152
  __device__ __forceinline__ uint32_t low(uint32_t w) const {
    return __builtin_bit_cast(uint32_t,
                              pair_of((w & low_bits) | base1024) - f16x2{1032.0f16, 1032.0f16});
  }
  __device__ __forceinline__ uint32_t high(uint32_t w) const {
    return __builtin_bit_cast(uint32_t,
                              pair_of((w & high_bits) | base1024) - f16x2{1152.0f16, 1152.0f16});
  }
};

// the value of the lane N places on, round the 16 of a DPP row
template <int N>
__device__ __forceinline__ uint32_t from_lane(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + 16 - N, 0xF, 0xF, false);
}
template <int N>
__device__ __forceinline__ float from_lane(float v) {
  return __builtin_bit_cast(float, from_lane<N>(__builtin_bit_cast(uint32_t, v)));
}

// The 16 lanes of a group of rows hold 16 / FOLD rows FOLD times over, each 1 / FOLD of the row's keys.
// Maximum and sum over the lanes that hold a row:
template <int FOLD>
__device__ __forceinline__ float fold_max(float x) {
  if constexpr (FOLD >= 2) x = fmaxf(x, from_lane<8>(x));
  if constexpr (FOLD >= 4) x = fmaxf(x, from_lane<4>(x));
  return row_max<16>(x);
}
template <int FOLD>
__device__ __forceinline__ float fold_sum(float x) {
  if constexpr (FOLD >= 2) x += from_lane<8>(x);
  if constexpr (FOLD >= 4) x += from_lane<4>(x);
  return row_sum<16>(x);
}
__device__ __forceinline__ float half_at(const uint32_t* v, int e) {
  return half_bits_to_float((uint16_t)(e & 1 ? v[e >> 1] >> 16 : v[e >> 1] & 0xFFFFu));
}

__device__ __forceinline__ u32x4 all_halves(float f) {
  const uint32_t h = Half::bits(f) * 0x10001u;
  return u32x4{h, h, h, h};
}

// A 32-key step as a wave stages it in LDS: the codes of the keys' two 16-token blocks, of the
// values', and both blocks' scales, in 16-byte pieces as they lie in memory, but for the key rows of
// 64 and 128 bytes, whose pieces change places by their row so that the eight rows that
// eight lanes read at once meet different banks.
template <int DT>
struct Stage {
  static constexpr int D = 32 * DT;
  static constexpr int kBytes = 32 * D + 256;
  static constexpr int kLoads = DT + 1;  // that a wave issues for a step
  static __device__ __forceinline__ int swizzle(int row) {
    return DT == 4 ? (row >> 1 & 1) | (row >> 3 & 1) << 1 : DT == 8 ? (row & 3) | (row >> 3 & 1) << 2 : 0;
  }
};

// A lane's queries (consecutive eights of its quarter of D) as fp16 times the power of 2 that takes the
// row's largest to 2^14 .. 2^15 (for fp16 2^30 at most), a negative scale in their sign, a zero one
// in the queries themselves.  Returns what takes raw scores to exponents of 2.
template <class E, int DT>
__device__ __forceinline__ float scaled_queries(u32x4 (&q)[DT], float scale) {
  u16x2 most = {0, 0};
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t two = q[i][e] & 0x7FFF7FFFu;
      most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, two));
    }
  int up = 15 - __builtin_amdgcn_frexp_expf(row_max<16>(E::value(most[0] > most[1] ? most[0] : most[1])));
  const float sign = scale == 0.0f ? 0.0f : scale < 0.0f ? -1.0f : 1.0f;
  if constexpr (std::is_same_v<E, Half>) {
    up = min(up, 30);
    const _Float16 f0 = (_Float16)(__builtin_amdgcn_ldexpf(sign, min(up, 15)));
    const _Float16 f1 = (_Float16)(__builtin_amdgcn_ldexpf(1.0f, max(up - 15, 0)));
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t two = q[i][e];
        q[i][e] = __builtin_bit_cast(uint32_t, pair_of(two) * f16x2{f0, f0} * f16x2{f1, f1});
      }
  } else {
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t two = q[i][e];
        const float v0 = __builtin_amdgcn_ldexpf(E::value((uint16_t)(two & 0xFFFFu)) * sign, up);
        const float v1 = __builtin_amdgcn_ldexpf(E::value((uint16_t)(two >> 16)) * sign, up);
        q[i][e] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(v0, v1));
      }
  }
  // (neither 0 nor infinite: a masked score's -inf and a score of 0 keep their products)
  return fminf(fmaxf(__builtin_amdgcn_ldexpf(scale != 0.0f ? fabsf(scale) * kLog2e : 1.0f, -up), 0x1p-126f),
               0x1.fffffep+127f);
}

// The pairs of the lanes that hold a row's other keys, behind the lane's own.  (Only the first 16 / FOLD
// lanes of 16 get them in order; the others' columns are nobody's rows.)
template <int FOLD>
__device__ __forceinline__ void gather(u32x4& v) {
  if constexpr (FOLD == 2) {
    const uint32_t v0 = v[0], v1 = v[1];
    v[2] = from_lane<8>(v0);
    v[3] = from_lane<8>(v1);
  } else {
    const uint32_t v0 = v[0];
    v[1] = from_lane<4>(v0);
    v[2] = from_lane<8>(v0);
    v[3] = from_lane<12>(v0);
  }
}

}  // namespace

// 32-key steps between the first tokens and the earliest key that any row's window holds.
__device__ __forceinline__ int window_gap(const Kv4AttentionArgs& a, const Request& r) {
  if (a.window <= 0) return 0;
  // (a tree's row that attends no drafted token has the window that ends before them)
  const int low = max(0, r.ctx + (a.mask ? 0 : 1) - a.window) >> 5;
  return max(0, min(low, (r.len + 31) >> 5) - ((a.sinks + 31) >> 5));
}

// One workgroup = one share of the cache, key head and block of rows: KW of its waves take the steps in
// turn, 4 / KW the rows, RG groups of 16 each.
template <class E, int DT, int RG, int FOLD, int S>
__global__ __launch_bounds__(64 * kWaves, units_per_cu(32 * DT, RG)) void kv4_attention_kernel(
    const Kv4AttentionArgs a, int shares, int row_blocks, int key_waves) {
  static_assert(FOLD == 1 || RG == 1, "few rows are one group");
  constexpr int D = 32 * DT;
  constexpr int kRows = 16 / FOLD;  // of a group
  constexpr int kKeys = 8 / FOLD;   // whose scores a lane holds
  // Two groups of rows are often two waves that read the same keys: the second finds them in L2 (trees of
  // seven on 24 contexts of 8k 80 us, passed by 82; one wave's keys, two contexts of 128k, passed by 52, kept 55).
  constexpr int kKept = RG == 2 ? 0 : kNonTemporal;
  constexpr int kTiles = 2 * DT;  // of O, and quads of consecutive d that a lane ends up with
  extern __shared__ __attribute__((aligned(1024))) char lds[];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, p = lane >> 4;
  const int key_wave = wave & (key_waves - 1), row_wave = wave >> __builtin_ctz(key_waves);
  const int block_rows = (kWaves >> __builtin_ctz(key_waves)) * (16 * RG);
  // Workgroups 8 apart share an XCD: the row blocks that read the same keys do.
  int hk = blockIdx.x, block_row0 = 0;
  uint32_t share = blockIdx.y;
  if (row_blocks > 1) {
    const int id = blockIdx.x;
    const int unit = id / (8 * row_blocks) * 8 + id % 8;
    hk = unit % a.Hkv;
    share = unit / a.Hkv;
    block_row0 = id / 8 % row_blocks * block_rows;
  }
  int b;
  uint32_t before;
  Window window;
  const Plan plan = make_plan(a, shares, share, b, before, window);
  if (b >= a.B) return;
  const uint32_t share_begin = plan.start(share), share_end = plan.start(share + 1);
  const int group = a.group;
  const Parts parts = parts_of(a, shares, a.max_new * group);
  // row / group
  auto token_of = [&](int row) {
    const int t = __umulhi(row, a.group_inverse);
    return t + (row - t * group >= group ? 1 : 0);
  };
  const int per_page = 1 << (a.page_shift - 4);  // 16-token blocks of a page

  // This wave's stages, and the lane's places in one: its first key's quarter row (the other
  // key's is four rows on), its eight keys' value pairs, their scales.
  using Staged = Stage<DT>;
  char* const ring = lds + wave * (S * Staged::kBytes);
  const int key_row = 8 * (c >> 2 & 1) + (c & 3);
  const int key_at = (c >> 3) * 8 * D + key_row * (D / 2);
  const int value_at = 16 * D + (p >> 1) * 8 * D + (p & 1) * 4 * D;
  const int part = c / kRows * kKeys;  // the first of the lane's keys among those eight
  const int scale_at = 32 * D + (p >> 1) * 128 + (p & 1) * 16 + 2 * part;
  uint32_t key_from[DT < 4 ? 1 : DT / 4];  // the piece of a block's keys that the lane fetches
#pragma unroll
  for (int u = 0; u < DT / 4; ++u) {
    const int i = 64 * u + lane, row = i / DT;
    key_from[u] = (row * DT + (i % DT ^ Staged::swizzle(row))) * 16;
  }
  const Codes codes;
  float zero = 0.0f;  // the compiler's own zero would keep p s from being one instruction
  asm("" : "+v"(zero));

  for (; b < a.B && before < share_end; ++b) {
    if ((uint32_t)(b - window.base) >= 64u) {
      window.base = b;
      window.mine = load_request(a, b + lane);
    }
    const Request r = window.at<Kv4AttentionArgs>(b);
    const uint32_t weight = r.weight<Kv4AttentionArgs>();
    if (weight == 0) continue;
    const int cu = r.cu, n_new = r.n_new, ctx = r.ctx, len = r.len, steps = (int)r.steps();
    // this share's steps of the request
    const uint32_t first_step = before + a.kHead;
    const int begin = share_begin > first_step ? (int)(share_begin - first_step) : 0;
    int end = min(steps, (int)(share_end - first_step));
    before += weight;
    if (end <= begin) continue;
    // whether the request begins in this share, and whether all of it is there
    const bool begins = first_step >= share_begin;
    const bool whole = begins && first_step + steps <= share_end;
    if (threadIdx.x == 0 && hk == 0 && block_row0 == 0 && begins)
      parts.plan[b] = {(int)share, whole ? (int)share : (int)plan.share_of(first_step + steps - 1)};
    const int rows = n_new * group;
    if (block_row0 >= rows) continue;
    // Steps count without the gap: step v is the request's step v, or v + gap behind the sinks.
    const int sink_steps = r.gap > 0 ? (a.sinks + 31) >> 5 : 0;
    int gap = r.gap, skip = 0;  // of this row block: what its own window passes over besides
    if (!a.mask) {  // a chain: nothing past the last row's token, or before the first's window
      const int last = min(block_row0 + block_rows, rows) - 1;
      const int to = (ctx + token_of(last) + 32) >> 5;
      end = min(end, to <= sink_steps ? to : max(sink_steps, to - gap));
      if (gap > 0) skip = max(0, ((ctx + token_of(block_row0) + 1 - a.window) >> 5) - gap - sink_steps);
    }
    auto actual = [&](int v) { return v < sink_steps ? v : v + gap; };
    auto following = [&](int v) { return v >= sink_steps && v < sink_steps + skip ? sink_steps + skip : v; };

    const int row0 = block_row0 + row_wave * (16 * RG);
    // the lane's rows, their tokens in the request, and those tokens' places in q
    int tok[RG];
    bool in[RG];
    float Q[RG], by[RG];       // sum of the fp16 queries; from raw scores to exponents of 2
    f32x4 minus64[RG];         // - 64 Q
    u32x4 q[RG][DT];
    int since[RG];             // first key of the row's window
#pragma unroll
    for (int g = 0; g < RG; ++g) {
      const int row = row0 + 16 * g + c % kRows;
      tok[g] = token_of(row);
      const int64_t at = (int64_t)cu + tok[g];
      in[g] = row < rows && at >= 0 && at < a.T;
      const uint16_t* from = a.q + at * a.q_st + (int64_t)(hk * group + row - tok[g] * group) * a.q_sh + p * 8 * DT;
#pragma unroll
      for (int i = 0; i < DT; ++i)
        q[g][i] = in[g] ? *reinterpret_cast<const u32x4*>(from + 8 * i) : u32x4{};
    }

    const scalar_ptr_t table = (scalar_ptr_t)(a.table + (int64_t)b * a.max_blocks);
    auto page_of = [&](int step, int half) {
      const int pos = step * 32 + half * 16;
      return pos < len ? table[pos >> a.page_shift] : -1;
    };
    auto block_of = [&](int page, int step, int half) {
      if ((unsigned)page >= (unsigned)a.num_pages) return -1;
      return (page * a.Hkv + hk) * per_page + ((step * 2 + half) & (per_page - 1));
    };
    auto next = [&](int v) { return following(v + key_waves); };
    const int first = following(begin + key_wave);
    const bool works = row0 < rows && first < end;
    int ahead = min(first, end - 1);  // the next step to be staged, and its pages
    int page0 = page_of(actual(ahead), 0), page1 = page_of(actual(ahead), 1);
    uint32_t holes = 0;  // bit 2 slot + h: no page behind the staged step's keys 16 h ..
    // Stages the step `ahead`, and fetches the pages of the one after it.
    auto stage = [&](int slot) {
      const int step = actual(ahead);
      const int b0 = block_of(page0, step, 0), b1 = block_of(page1, step, 1);
      holes = (holes & ~(3u << 2 * slot)) | ((b0 < 0 ? 1u : 0u) | (b1 < 0 ? 2u : 0u)) << 2 * slot;
      const int64_t at0 = (int64_t)max(b0, 0) * (8 * D), at1 = (int64_t)max(b1, 0) * (8 * D);
      const char* keys = reinterpret_cast<const char*>(a.kc);
      const char* values = reinterpret_cast<const char*>(a.vc);
      char* const to = ring + slot * Staged::kBytes;
#pragma unroll
      for (int u = 0; u < DT; ++u) {
        const char* from;
        if constexpr (DT % 4 == 0) {  // whole kilobytes of one block
          constexpr int kEach = DT / 4;
          from = (u < DT / 2 ? keys : values) + (u / kEach % 2 ? at1 : at0) +
                 (u < DT / 2 ? key_from[u % kEach] : lane * 16u + u % kEach * 1024u);
        } else {
          const int i = 64 * u + lane, j = i % D;
          from = (i < D ? keys : values) + (j < D / 2 ? at0 : at1) + j % (D / 2) * 16;
        }
        __builtin_amdgcn_global_load_lds((global_ptr_t)from, (lds_ptr_t)(to + u * 1024), 16, 0,
                                         kKept);
      }
      const char* from = reinterpret_cast<const char*>(a.scales) +
                         (int64_t)max(lane < 32 ? b0 : b1, 0) * 128 + (lane & 31) * 4;
      __builtin_amdgcn_global_load_lds((global_ptr_t)from, (lds_ptr_t)(to + 32 * D), 4, 0,
                                       kKept);
      const int after = next(ahead);
      ahead = after;
      const int then = actual(min(after, end - 1));
      page0 = page_of(then, 0);
      page1 = page_of(then, 1);
    };
    // S - 1 steps, the last again where there are fewer: with a fixed number of loads behind it the
    // wait for q leaves them in flight.
    if (works)
#pragma unroll
      for (int i = 0; i < S - 1; ++i) {
        const int v = ahead;
        stage(i);
        if (ahead >= end && i < S - 2) ahead = v;
      }
#pragma unroll
    for (int g = 0; g < RG; ++g) {
#pragma unroll
      for (int i = 0; i < DT; ++i)
        asm volatile("" : "+v"(q[g][i]));  // (not before the first steps are on their way)
      by[g] = scaled_queries<E, DT>(q[g], a.scale);
      // the sums that take the codes' 64 off, by the MFMAs that will add it
      minus64[g] = f32x4{};
      const u32x4 m64 = all_halves(-64.0f);
#pragma unroll
      for (int i = 0; i < DT; ++i) minus64[g] = Half::mfma(m64, q[g][i], minus64[g]);
      Q[g] = minus64[g][0] * -0.015625f;
      since[g] = -(1 << 30);
      if (a.window > 0) {
        int drafted = tok[g] + 1;
        if (a.mask) {
          drafted = 0;
          if (in[g]) {
            const int32_t* words = a.mask + ((int64_t)cu + tok[g]) * a.mask_words;
            for (int w = 0; w < a.mask_words && 32 * w < n_new; ++w) {
              const int bits = n_new - 32 * w;
              drafted += __builtin_popcount((uint32_t)words[w] & (bits >= 32 ? ~0u : (1u << bits) - 1u));
            }
          }
        }
        since[g] = ctx + drafted - a.window;
      }
    }
    f32x4 o[RG][kTiles] = {};
    f32x4 W[RG] = {};           // sum of w, of all keys in every lane of a column
    float m[RG], l[RG], B[RG];  // reference, and the lane's share of the sums of p and p b
    const u32x4 ones = all_halves(1.0f);
#pragma unroll
    for (int g = 0; g < RG; ++g) m[g] = -INFINITY, l[g] = B[g] = 0.0f;

    auto work = [&](int slot, int index) __attribute__((always_inline)) {
      const char* const from = ring + slot * Staged::kBytes;
      auto scales_at = [&](int which, uint32_t* to) {
        const uint32_t* at = reinterpret_cast<const uint32_t*>(from + scale_at + 32 * which);
#pragma unroll
        for (int i = 0; i < kKeys / 2; ++i) to[i] = at[i];
      };
      uint32_t kd[2][DT];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const char* row = from + key_at + t * (2 * D);
#pragma unroll
        for (int i = 0; i < DT; ++i) {
          if constexpr (DT % 4 == 0) {
            const int piece = (p * (DT / 4) + i / 4) ^ Staged::swizzle(key_row);
            const u32x4 v = *reinterpret_cast<const u32x4*>(row + piece * 16);
            kd[t][i] = v[i & 3];
          } else {
            kd[t][i] = reinterpret_cast<const uint32_t*>(row)[p * DT + i];
          }
        }
      }
      uint32_t ks[kKeys / 2], kb[kKeys / 2], vs[RG][kKeys / 2], vb[RG][kKeys / 2];
      scales_at(0, ks);
      scales_at(1, kb);
      f32x4 x[RG][2];
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const u32x4 f = codes.key(kd[t][i]);
#pragma unroll
          for (int g = 0; g < RG; ++g) x[g][t] = Half::mfma(f, q[g][i], i == 0 ? minus64[g] : x[g][t]);
        }
      float raw[RG][kKeys];
#pragma unroll
      for (int g = 0; g < RG; ++g) {
        scales_at(2, vs[g]);  // (of what the row attends)
        scales_at(3, vb[g]);
#pragma unroll
        for (int e = 0; e < kKeys; ++e) {
          float qc;
          if constexpr (FOLD == 1)
            qc = x[g][e >> 2][e & 3];
          else if constexpr (FOLD == 2)
            qc = c >= 8 ? x[g][1][e] : x[g][0][e];
          else
            qc = c >= 8 ? (c & 4 ? x[g][1][2 + e] : x[g][1][e]) : (c & 4 ? x[g][0][2 + e] : x[g][0][e]);
          raw[g][e] = fmaf(half_at(ks, e), qc, half_at(kb, e) * Q[g]);
        }
      }
      // Keys that are no context (drafted, or none at all), on no page, or before some row's
      // window: the wave masks.
      const int pos = index * 32;
      const uint32_t hole = holes >> 2 * slot & 3u;
      if (hole != 0 || pos + 32 > ctx || (a.window > 0 && pos < ctx + n_new - a.window)) {
        const int pos0 = pos + 8 * p;
        const uint32_t there = (hole >> (p >> 1)) & 1u ? 0u : low_bits(len - pos0);
#pragma unroll
        for (int g = 0; g < RG; ++g) {
          const uint32_t inside = a.window > 0 ? low_bits(a.sinks - pos0) | ~low_bits(since[g] - pos0) : ~0u;
          uint32_t seen;
          if (a.mask) {  // the context in the window, and the tree's bits
            seen = low_bits(ctx - pos0) & inside;
            const int j0 = pos0 - ctx;
            if (j0 > -8 && in[g]) {
              const int32_t* words = a.mask + ((int64_t)cu + tok[g]) * a.mask_words;
              const int w = j0 >> 5;
              const uint32_t w0 = w >= 0 && w < a.mask_words ? (uint32_t)words[w] : 0u;
              const uint32_t w1 = w + 1 < a.mask_words ? (uint32_t)words[w + 1] : 0u;
              seen |= (uint32_t)(((uint64_t)w1 << 32 | w0) >> (j0 & 31)) & 0xFFu;
            }
          } else {  // a chain: the tokens up to the row's own, in the window
            seen = low_bits(ctx + tok[g] + 1 - pos0) & inside;
          }
          seen = (seen & there) >> part;
#pragma unroll
          for (int e = 0; e < kKeys; ++e)
            if (!((seen >> e) & 1u)) raw[g][e] = -INFINITY;
#pragma unroll
          for (int i = 0; i < kKeys / 2; ++i) {  // (what masked places hold does not matter, NaN included)
            const uint32_t keep = (seen >> (2 * i) & 1u) * 0xFFFFu | (seen >> (2 * i + 1) & 1u) * 0xFFFF0000u;
            vs[g][i] &= keep;
            vb[g][i] &= keep;
          }
        }
      }

      // A row's reference m is a whole number that no exponent of p s exceeds by more than kLag.  The
      // probabilities are formed under the reference that the row has; where some p s passes 2^(kTop + kLag)
      // (rare after a request's first step) it goes up to the largest exponent of p s, each key's own,
      // the sums come down by a power of 2 and the probabilities are formed again.  A scale of 0
      // counts as 2^-60, which keeps the sums of p and p b in fp32's range.
      u32x4 hi[RG], lo[RG];
#pragma unroll
      for (int g = 0; g < RG; ++g) {
        float sum, offset;
        auto form = [&]() __attribute__((always_inline)) {
          // (over nothing every key's is infinite)
          const float ref = m[g] == -INFINITY ? 3e38f : kTop - m[g];
          sum = offset = 0.0f;
#pragma unroll
          for (int i = 0; i < kKeys / 2; ++i) {
            float prob[2], step[2];
            f16x2 h, rest;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              prob[j] = __builtin_amdgcn_exp2f(fmaf(raw[g][2 * i + j], by[g], ref));
              step[j] = half_at(vs[g], 2 * i + j);
              sum += prob[j];
              offset = fmaf(prob[j], half_at(vb[g], 2 * i + j), offset);
              h[j] = (_Float16)fmaf(prob[j], step[j], zero);
            }
            uint32_t bits = __builtin_bit_cast(uint32_t, h);
            asm("" : "+v"(bits));  // the very bits that the product takes are what is left out of the rest
            hi[g][i] = bits;
            h = pair_of(bits);
#pragma unroll
            for (int j = 0; j < 2; ++j) rest[j] = (_Float16)fmaf(prob[j], step[j], -(float)h[j]);
            lo[g][i] = __builtin_bit_cast(uint32_t, rest);
          }
        };
        form();
        // (p s are not negative: their bits are in their order)
        u16x2 most = {0, 0};
#pragma unroll
        for (int i = 0; i < kKeys / 2; ++i) {
          const uint32_t two = hi[g][i];
          most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, two));
        }
        if (__ballot((most[0] > most[1] ? most[0] : most[1]) > kMostBits || sum > 0x1p80f)) {
          float top = -INFINITY;
#pragma unroll
          for (int e = 0; e < kKeys; ++e) {
            const float s = half_at(vs[g], e);
            top = fmaxf(top, fmaf(raw[g][e], by[g], s > 0.0f ? __builtin_amdgcn_logf(s) : -60.0f));
          }
          top = fold_max<FOLD>(top);
          top = top > m[g] + kLag ? ceilf(top) : m[g];  // (a row's own keys alone raise it)
          const float down = m[g] - (top == -INFINITY ? 0.0f : top);
          m[g] = top;
          l[g] = scaled(l[g], down);
          B[g] = scaled(B[g], down);
#pragma unroll
          for (int i = 0; i < 4; ++i) W[g][i] = scaled(W[g][i], down);
#pragma unroll
          for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[g][t][i] = scaled(o[g][t][i], down);
          form();
        }
        l[g] += sum;
        B[g] += offset;
        if constexpr (FOLD > 1) gather<FOLD>(hi[g]);
        if constexpr (FOLD > 1) gather<FOLD>(lo[g]);
        W[g] = Half::mfma(ones, hi[g], W[g]);
        W[g] = Half::mfma(ones, lo[g], W[g]);
      }
      uint32_t vd[2 * DT];
#pragma unroll
      for (int u = 0; u < 2 * DT; ++u) {
        const int n = 2 * DT - u / 4 * 4 < 4 ? 2 : 4;
        vd[u] = reinterpret_cast<const uint32_t*>(from + value_at + u / 4 * 256)[n * c + (u & 3)];
      }
#pragma unroll
      for (int i = 0; i < DT; ++i) {
        const uint32_t w0 = vd[2 * i], w1 = vd[2 * i + 1], w0s = w0 >> 8, w1s = w1 >> 8;
        const u32x4 even = {codes.low(w0), codes.low(w0s), codes.low(w1), codes.low(w1s)};
        const u32x4 odd = {codes.high(w0), codes.high(w0s), codes.high(w1), codes.high(w1s)};
#pragma unroll
        for (int g = 0; g < RG; ++g) {
          o[g][2 * i] = Half::mfma(even, hi[g], o[g][2 * i]);
          o[g][2 * i + 1] = Half::mfma(odd, hi[g], o[g][2 * i + 1]);
          o[g][2 * i] = Half::mfma(even, lo[g], o[g][2 * i]);
          o[g][2 * i + 1] = Half::mfma(odd, lo[g], o[g][2 * i + 1]);
        }
      }
    };

    if (works) {
      int slot = 0;
      for (int v = first; v < end; v = next(v)) {
        const int free = slot == 0 ? S - 1 : slot - 1;  // (worked on the time before)
        if (ahead < end) {
          stage(free);
          wait_vm<(S - 1) * Staged::kLoads>();
        } else {
          wait_vm<0>();
        }
        asm volatile("" ::: "memory");
        work(slot, actual(v));
        slot = slot == S - 1 ? 0 : slot + 1;
      }
    }

    // quad j: four consecutive d (4 d4 ..), of tiles that hold them side by side
    f32x4 quad[RG][kTiles];
    float total[RG];
#pragma unroll
    for (int g = 0; g < RG; ++g) {
      total[g] = fold_sum<FOLD>(l[g]);
      const float offset = fmaf(W[g][0], 8.0f, fold_sum<FOLD>(B[g]));
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float x = fmaf(o[g][t][k], t & 1 ? 0.0625f : 1.0f, offset);
          const bool pair = 4 * (t / 4) + 4 > kTiles;  // two tiles left: two rows make a quad
          if (pair)
            quad[g][4 * (t / 4) + k / 2][2 * (k & 1) + (t & 1)] = x;
          else
            quad[g][4 * (t / 4) + k][t & 3] = x;
        }
    }
    auto d4_of = [&](int j) {
      return 4 * (j / 4) + 4 > kTiles ? 16 * (j / 4) + 2 * p + (j & 1) : 16 * (j / 4) + 4 * p + (j & 3);
    };
    auto put = [&](int g, int j, f32x4 v, float ref, float sum) {
      const int row = row0 + 16 * g + c;
      if (row >= rows || c >= kRows) return;
      const int d4 = d4_of(j);
      const float top = ref == -INFINITY ? ref : ref - kTop;
      if (!whole) {
        const int64_t place = 2 * (int64_t)share + (begins ? 1 : 0);
        const int64_t at = (place * a.Hkv + hk) * (a.max_new * group) + row;
        parts.out[at * (D / 4) + d4] = v;
        if (d4 == 0) parts.stat[at] = {top, sum};
      } else if (in[g]) {
        const int64_t t = (int64_t)cu + tok[g];
        const int h = hk * group + row - tok[g] * group;
        const float zero = top == -INFINITY ? 0.0f : top;
        write_row<E>(a, t, h, d4, v, zero, sum);
      }
    };
    if (key_waves == 1) {
#pragma unroll
      for (int g = 0; g < RG; ++g)
#pragma unroll
        for (int j = 0; j < kTiles; ++j) put(g, j, quad[g][j], m[g], total[g]);
      continue;
    }
    // the waves that shared the steps: each adds up some of the quads
    f32x4* sums = reinterpret_cast<f32x4*>(lds) + wave * (RG * kTiles * 64) + lane;
    float2* stats = reinterpret_cast<float2*>(lds + kWaves * RG * kTiles * 1024);
    lds_barrier();  // every wave's stages have been read
#pragma unroll
    for (int g = 0; g < RG; ++g) {
      if (p == 0) stats[(wave * RG + g) * 16 + c] = {m[g], total[g]};
#pragma unroll
      for (int j = 0; j < kTiles; ++j) sums[(g * kTiles + j) * 64] = quad[g][j];
    }
    lds_barrier();
    const int wave0 = wave - key_wave;
    const f32x4* all = reinterpret_cast<f32x4*>(lds) + wave0 * (RG * kTiles * 64) + lane;
#pragma unroll
    for (int g = 0; g < RG; ++g) {
      float top = -INFINITY, sum = 0.0f;
      for (int w = 0; w < key_waves; ++w) top = fmaxf(top, stats[((wave0 + w) * RG + g) * 16 + c].x);
      const float ref = top == -INFINITY ? 0.0f : top;
      for (int w = 0; w < key_waves; ++w) {
        const float2 s = stats[((wave0 + w) * RG + g) * 16 + c];
        sum += scaled(s.y, s.x - ref);
      }
      for (int j = key_wave; j < kTiles; j += key_waves) {
        f32x4 v = {};
        for (int w = 0; w < key_waves; ++w) {
          const float down = stats[((wave0 + w) * RG + g) * 16 + c].x - ref;
          const f32x4 x = all[(w * RG * kTiles + g * kTiles + j) * 64];
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] += scaled(x[k], down);
        }
        put(g, j, v, top, sum);
      }
    }
    lds_barrier();  // the sums have been read, and steps may be staged where they were
  }
}

namespace {

// How a call is laid out: groups of 16 rows a wave, times over that fewer rows fill one, waves along
// the keys, row blocks, shares
struct Layout {
  int groups, fold, key_waves, row_blocks, shares;
};

Layout layout_of(int64_t max_new, int64_t H, int64_t Hkv, int64_t D) {
  Layout p;
  const int64_t rows = max_new * (H / Hkv);
  // two groups of rows a wave share the conversion of the codes (256-wide heads have no registers for it)
  p.groups = rows <= 16 || D > 128 ? 1 : 2;
  p.fold = rows <= 4 ? 4 : rows <= 8 ? 2 : 1;
  const int64_t waves = (rows + 16 * p.groups - 1) / (16 * p.groups);  // that hold rows
  p.key_waves = waves == 1 ? 4 : waves == 2 ? 2 : 1;
  const int64_t block_rows = kWaves / p.key_waves * 16 * p.groups;
  p.row_blocks = (int)((rows + block_rows - 1) / block_rows);
  const int64_t target = units_per_cu(D, p.groups) * device_cu_count();
  p.shares = (int)std::max<int64_t>(1, target / (Hkv * p.row_blocks));
  return p;
}

template <class E, int DT>
hipError_t launch_rows(Kv4AttentionArgs a, hipStream_t stream) {
  Layout p = layout_of(a.max_new, a.H, a.Hkv, a.D);
  a.key_waves = (uint32_t)p.key_waves;
  // no more shares than the tables' room can fill (short contexts: one, and no join)
  int64_t room = (((int64_t)a.max_blocks << a.page_shift) + 31) / 32;
  if (a.window > 0)  // (rounded out to whole steps)
    room = std::min<int64_t>(room, ((int64_t)a.window + a.max_new + a.sinks) / 32 + 4);
  p.shares = (int)std::min<int64_t>(
      p.shares, std::max<int64_t>(1, a.B * (a.kHead + room) / a.least_share()));
  const int64_t units = (int64_t)p.shares * a.Hkv;
  const dim3 grid = p.row_blocks == 1 ? dim3((unsigned)a.Hkv, (unsigned)p.shares)
                                      : dim3((unsigned)((units + 7) / 8 * 8 * p.row_blocks));
  // stages: what a workgroup's share of a compute unit's LDS holds
  constexpr int S = DT <= 4 ? 3 : 2, S2 = 4;
  auto* kernel = p.fold == 4   ? kv4_attention_kernel<E, DT, 1, 4, S>
                 : p.fold == 2 ? kv4_attention_kernel<E, DT, 1, 2, S>
                               : kv4_attention_kernel<E, DT, 1, 1, S>;
  if constexpr (DT <= 4) {
    if (p.groups == 2) kernel = kv4_attention_kernel<E, DT, 2, 1, S2>;
  }
  const size_t sums =
      p.key_waves == 1 ? 0 : (size_t)kWaves * p.groups * (2 * DT * 1024 + 16 * sizeof(float2));
  const size_t lds =
      std::max(sums, (size_t)kWaves * (p.groups == 2 ? S2 : S) * Stage<DT>::kBytes);
  const hipError_t e = launch_kernel_lds(kernel, grid, dim3(64 * kWaves), lds, stream, a, p.shares,
                                         p.row_blocks, p.key_waves);
  if (e != hipSuccess || p.shares == 1) return e;
  return launch_join<Kv4AttentionArgs, E, DT>(a, p.shares, stream);
}

template <class E>
hipError_t launch_width(const Kv4AttentionArgs& a, hipStream_t stream) {
  switch (a.D) {
    case 64: return launch_rows<E, 2>(a, stream);
    case 96: return launch_rows<E, 3>(a, stream);
    case 128: return launch_rows<E, 4>(a, stream);
    default: return launch_rows<E, 8>(a, stream);
  }
}

}  // namespace

size_t kv4_attention_workspace_bytes(int64_t B, int64_t max_new, int64_t H, int64_t Hkv,
                                     int64_t D) {
  return parts_bytes(B, max_new, H, D, layout_of(max_new, H, Hkv, D).shares);
}

hipError_t launch_kv4_attention(const Kv4AttentionArgs& a, bool bf16, hipStream_t stream) {
  return bf16 ? launch_width<Bfloat>(a, stream) : launch_width<Half>(a, stream);
}

}  // namespace flexq
