// serve_kv4_attention.hip -- attention of drafted tokens over a paged cache of 4-bit codes, with
// an optional sliding window whose first tokens stay visible.
//
// A key is k = b + s c with codes c = 0 .. 15 and a scale and an offset for its token and head, a
// value likewise.  For a row with queries q, Q = sum q:
//   q.k = s (q.(c - 8) + 8 Q) + b Q
//   sum_j p_j v_j = sum_j (p_j s_j) (c_j - 8) + sum_j p_j (b_j + 8 s_j)
// so both products are MFMAs on c - 8, which fp16 holds exactly, whatever the tensors' type, and the
// scales meet scores and probabilities.  (c - 8 rather than c: sums of codes of one sign would
// err with their size, not their result's.)  The queries enter as fp16 after a row's power of
// two, whole down to 2^-24 of the row's largest and below within 2^-34 of it.
// w_j = p_j s_j enters as the sum of two fp16 parts, within 2^-22 of itself or 2^-35 of the row's
// largest, whichever is more.
//
// Codes to fp16, nine instructions for eight: an and-or puts the code's bits below an exponent
// (1024 + c, or 1024 + 16 c of the next four bits), and one addition of a pair takes the rest
// off, leaving c - 8 or 16 (c - 8).  The factor 16 goes into the queries or out of the sums.
//
// A wave stages its own 32-key steps in LDS straight from memory, S - 1 of them on their way while one
// is worked on, and needs no barrier until a request's end.  Rows are
// columns of the MFMAs (16 a group), so a lane owns one row's statistics, and the keys are
// dealt to the score tiles' rows so that a lane's scores are those that its fragment of P takes:
// row r of score tile t holds key 8 (r / 4) + 4 t + r % 4, lane l keys 8 (l / 16) .. + 7.  Waves
// that the rows leave over take the steps in turn and add up in LDS.
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

// Workgroups a compute unit holds.
constexpr int units_per_cu(int64_t D, int groups) { return groups == 1 && D <= 128 ? 3 : 2; }

// (by value: a bit cast of a vector's element takes the whole vector's first bits)
__device__ __forceinline__ f16x2 pair_of(uint32_t v) { return __builtin_bit_cast(f16x2, v); }

// Eight codes of a dword, four pairs: c - 8 from the low four bits of its bytes, 16 (c - 8) from the
// high ones.  The constants sit in registers: as literals they would take an and and an or.
struct Codes {
  uint32_t base = 0x64006400u, low_bits = 0x000F000Fu, high_bits = 0x00F000F0u;
  __device__ __forceinline__ Codes() {
    asm("" : "+v"(base));
    asm("" : "+s"(low_bits));
    asm("" : "+s"(high_bits));
  }
  __device__ __forceinline__ uint32_t low(uint32_t w) const {
    return __builtin_bit_cast(uint32_t, pair_of((w & low_bits) | base) - f16x2{1032.0f16, 1032.0f16});
  }
  __device__ __forceinline__ uint32_t high(uint32_t w) const {
    return __builtin_bit_cast(uint32_t, pair_of((w & high_bits) | base) - f16x2{1152.0f16, 1152.0f16});
  }
};

__device__ __forceinline__ float half_at(const u32x4& v, int e) {
  return half_bits_to_float((uint16_t)(e & 1 ? v[e >> 1] >> 16 : v[e >> 1] & 0xFFFFu));
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
template <int DT, int RG, int S>
__global__ __launch_bounds__(64 * kWaves, units_per_cu(32 * DT, RG)) void kv4_attention_kernel(const Kv4AttentionArgs a,
                                                                      int shares, int row_blocks,
                                                                      int key_waves) {
  constexpr int D = 32 * DT;
  constexpr int kTiles = 2 * DT;  // of O, and quads of consecutive d that a lane ends up with
  extern __shared__ __attribute__((aligned(1024))) char lds[];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, p = lane >> 4;
  const int key_wave = wave & (key_waves - 1), row_wave = wave / key_waves;
  const int block_rows = kWaves / key_waves * (16 * RG);
  // Workgroups 8 apart share an XCD: the row blocks that read the same keys do.
  const int id = blockIdx.x;
  const int unit = id / (8 * row_blocks) * 8 + id % 8;
  const int hk = unit % a.Hkv;
  const uint32_t share = unit / a.Hkv;
  const int block_row0 = id / 8 % row_blocks * block_rows;
  int b;
  uint32_t before;
  Window window;
  const Plan plan = make_plan(a, shares, share, b, before, window);
  if (b >= a.B) return;
  const uint32_t share_begin = plan.start(share), share_end = plan.start(share + 1);
  const int group = a.H / a.Hkv;
  const Parts parts = parts_of(a, shares, a.max_new * group);
  const int per_page = 1 << (a.page_shift - 4);  // 16-token blocks of a page

  // This wave's stages, and the lane's places in one: its first key's quarter row (the other
  // key's is four rows on), its eight keys' value pairs, their scales.
  using Staged = Stage<DT>;
  char* const ring = lds + wave * (S * Staged::kBytes);
  const int key_row = 8 * (c >> 2 & 1) + (c & 3);
  const int key_at = (c >> 3) * 8 * D + key_row * (D / 2);
  const int value_at = 16 * D + (p >> 1) * 8 * D + (p & 1) * 4 * D;
  const int scale_at = 32 * D + (p >> 1) * 128 + (p & 1) * 16;
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
    const uint32_t s0 = plan.share_of(first_step), s1 = plan.share_of(first_step + steps - 1);
    if (threadIdx.x == 0 && hk == 0 && block_row0 == 0 && share == s0)
      parts.plan[b] = {(int)s0, (int)s1};
    const int rows = n_new * group;
    if (block_row0 >= rows) continue;
    // Steps count without the gap: step v is the request's step v, or v + gap behind the sinks.
    const int sink_steps = r.gap > 0 ? (a.sinks + 31) >> 5 : 0;
    int gap = r.gap, skip = 0;  // of this row block: what its own window passes over besides
    if (!a.mask) {  // a chain: nothing past the last row's token, or before the first's window
      const int last = min(block_row0 + block_rows, rows) - 1;
      const int to = (ctx + last / group + 32) >> 5;
      end = min(end, to <= sink_steps ? to : max(sink_steps, to - gap));
      if (gap > 0) skip = max(0, ((ctx + block_row0 / group + 1 - a.window) >> 5) - gap - sink_steps);
    }
    auto actual = [&](int v) { return v < sink_steps ? v : v + gap; };
    auto following = [&](int v) { return v >= sink_steps && v < sink_steps + skip ? sink_steps + skip : v; };

    const int row0 = block_row0 + row_wave * (16 * RG);
    // the lane's rows, their tokens in the request, and those tokens' places in q
    int tok[RG];
    bool in[RG];
    float Q[RG], by[RG];       // sum of the fp16 queries; from raw scores to exponents of 2
    u32x4 loaded[RG][DT];
    uint32_t q[RG][DT][4];
    int since[RG];             // first key of the row's window
#pragma unroll
    for (int g = 0; g < RG; ++g) {
      const int row = row0 + 16 * g + c;
      tok[g] = row / group;
      const int64_t at = (int64_t)cu + tok[g];
      in[g] = row < rows && at >= 0 && at < a.T;
      const uint16_t* from = a.q + at * a.q_st + (int64_t)(hk * group + row % group) * a.q_sh + p * 8 * DT;
#pragma unroll
      for (int i = 0; i < DT; ++i)
        loaded[g][i] = in[g] ? *reinterpret_cast<const u32x4*>(from + 8 * i) : u32x4{};
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
          const int part = u % kEach, i = 64 * part + lane;
          const int row = i / (DT / 4 * 4), piece = i % (DT / 4 * 4) ^ Staged::swizzle(row);
          from = u < DT / 2 ? keys + (u / kEach ? at1 : at0) + (row * (DT / 4 * 4) + piece) * 16
                            : values + (u / kEach % 2 ? at1 : at0) + i * 16;
        } else {
          const int i = 64 * u + lane, j = i % D;
          from = (i < D ? keys : values) + (j < D / 2 ? at0 : at1) + j % (D / 2) * 16;
        }
        __builtin_amdgcn_global_load_lds((global_ptr_t)from, (lds_ptr_t)(to + u * 1024), 16, 0,
                                         kNonTemporal);
      }
      const char* from = reinterpret_cast<const char*>(a.scales) +
                         (int64_t)max(lane < 32 ? b0 : b1, 0) * 128 + (lane & 31) * 4;
      __builtin_amdgcn_global_load_lds((global_ptr_t)from, (lds_ptr_t)(to + 32 * D), 4, 0,
                                       kNonTemporal);
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
      float x[DT][8];
      float most = 0.0f;
#pragma unroll
      for (int i = 0; i < DT; ++i) {
        asm volatile("" : "+v"(loaded[g][i]));  // (not before the first steps are on their way)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t two = loaded[g][i][e >> 1];
          const uint16_t bits = (uint16_t)(e & 1 ? two >> 16 : two & 0xFFFFu);
          x[i][e] = a.bf16 ? Bfloat::value(bits) : Half::value(bits);
          most = fmaxf(most, fabsf(x[i][e]));
        }
      }
      // A row's largest query becomes 2^14 to 2^15; a negative scale goes into the sign, a zero
      // one into the queries.
      most = row_max<16>(most);
      const int up = 15 - __builtin_amdgcn_frexp_expf(most);
      Q[g] = 0.0f;
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          float y[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            y[j] = __builtin_amdgcn_ldexpf(x[i][e + j], up);
            y[j] = a.scale == 0.0f ? 0.0f : a.scale < 0.0f ? -y[j] : y[j];
            const float h = (float)(_Float16)y[j];
            Q[g] += h;
            y[j] = e & 2 ? h * 0.0625f : h;  // (codes there come as 16 (c - 8))
          }
          q[g][i][e >> 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(y[0], y[1]));
        }
      Q[g] = row_sum<16>(Q[g]);
      by[g] = __builtin_amdgcn_ldexpf(a.scale != 0.0f ? fabsf(a.scale) * kLog2e : 1.0f, -up);
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
    float m[RG], l[RG], B[RG];  // reference, sum of p, sum of p (b + 8 s)
#pragma unroll
    for (int g = 0; g < RG; ++g) m[g] = -INFINITY, l[g] = B[g] = 0.0f;

    auto work = [&](int slot, int index) __attribute__((always_inline)) {
      const char* const from = ring + slot * Staged::kBytes;
      auto scales_at = [&](int which) {
        return *reinterpret_cast<const u32x4*>(from + scale_at + 32 * which);
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
      const u32x4 ks = scales_at(0), kb = scales_at(1);
      f32x4 x[RG][2];
#pragma unroll
      for (int g = 0; g < RG; ++g)
#pragma unroll
        for (int t = 0; t < 2; ++t) x[g][t] = f32x4{8 * Q[g], 8 * Q[g], 8 * Q[g], 8 * Q[g]};
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint32_t w = kd[t][i], w8 = w >> 8;
          const u32x4 f = {codes.low(w), codes.high(w), codes.low(w8), codes.high(w8)};
#pragma unroll
          for (int g = 0; g < RG; ++g)
            x[g][t] = Half::mfma(f, u32x4{q[g][i][0], q[g][i][1], q[g][i][2], q[g][i][3]}, x[g][t]);
        }
      u32x4 vs[RG], vb[RG];  // of what the row attends
      float raw[RG][8];
#pragma unroll
      for (int g = 0; g < RG; ++g) {
        vs[g] = scales_at(2);
        vb[g] = scales_at(3);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          raw[g][e] = fmaf(half_at(ks, e), x[g][e >> 2][e & 3], half_at(kb, e) * Q[g]);
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
          seen &= there;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (!((seen >> e) & 1u)) raw[g][e] = -INFINITY;
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // (what masked places hold does not matter, NaN included)
            const uint32_t keep = (seen >> (2 * i) & 1u) * 0xFFFFu | (seen >> (2 * i + 1) & 1u) * 0xFFFF0000u;
            vs[g][i] &= keep;
            vb[g][i] &= keep;
          }
        }
      }

      // A row's reference m is a whole number that its exponents with the values' scales
      // exceed by kLag at most; raised where they would, it takes the sums down by a power of 2.
      u32x4 hi[RG], lo[RG];
#pragma unroll
      for (int g = 0; g < RG; ++g) {
        float top = raw[g][0];
#pragma unroll
        for (int e = 1; e < 8; ++e) top = fmaxf(top, raw[g][e]);
        // (scales are not negative: their bits are in their order)
        u16x2 most = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t two = vs[g][i];
          most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, two));
        }
        const float scale = half_bits_to_float(most[0] > most[1] ? most[0] : most[1]);
        top = fmaf(top, by[g], (float)__builtin_amdgcn_frexp_expf(scale));
        if (__ballot(top > m[g] + kLag)) {  // rare after a request's first step
          top = row_max<16>(top);
          top = fmaxf(m[g], ceilf(top));
          const float down = m[g] - (top == -INFINITY ? 0.0f : top);
          m[g] = top;
          l[g] = scaled(l[g], down);
          B[g] = scaled(B[g], down);
#pragma unroll
          for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[g][t][i] = scaled(o[g][t][i], down);
        }
        const float ref = m[g] == -INFINITY ? 0.0f : kTop - m[g];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float prob[2], step[2];
          f16x2 h, rest;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            prob[j] = __builtin_amdgcn_exp2f(fmaf(raw[g][2 * i + j], by[g], ref));
            step[j] = half_at(vs[g], 2 * i + j);
            l[g] += prob[j];
            B[g] = fmaf(prob[j], fmaf(step[j], 8.0f, half_at(vb[g], 2 * i + j)), B[g]);
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
      }
      // tile 4 u + j of O (2 u + j of the last two where D = 96) is d = 64 u + 4 row + j
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
      total[g] = row_sum<16>(l[g]);
      const float offset = row_sum<16>(B[g]);
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
      if (row >= rows) return;
      const int d4 = d4_of(j);
      const float top = ref == -INFINITY ? ref : ref - kTop;
      if (s0 != s1) {
        const int64_t place = 2 * (int64_t)share + (share == s0 ? 1 : 0);
        const int64_t at = (place * a.Hkv + hk) * (a.max_new * group) + row;
        parts.out[at * (D / 4) + d4] = v;
        if (d4 == 0) parts.stat[at] = {top, sum};
      } else if (in[g]) {
        const int64_t t = (int64_t)cu + tok[g];
        const int h = hk * group + row % group;
        const float zero = top == -INFINITY ? 0.0f : top;
        if (a.bf16)
          write_row<Bfloat>(a, t, h, d4, v, zero, sum);
        else
          write_row<Half>(a, t, h, d4, v, zero, sum);
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

// How a call is laid out: groups of 16 rows a wave, waves along the keys, row blocks, shares
struct Layout {
  int groups, key_waves, row_blocks, shares;
};

Layout layout_of(int64_t max_new, int64_t H, int64_t Hkv, int64_t D) {
  Layout p;
  const int64_t rows = max_new * (H / Hkv);
  p.groups = rows <= 16 || D > 128 ? 1 : 2;
  const int64_t waves = (rows + 16 * p.groups - 1) / (16 * p.groups);  // that hold rows
  p.key_waves = waves == 1 ? 4 : waves == 2 ? 2 : 1;
  const int64_t block_rows = kWaves / p.key_waves * 16 * p.groups;
  p.row_blocks = (int)((rows + block_rows - 1) / block_rows);
  const int64_t target = units_per_cu(D, p.groups) * device_cu_count();
  p.shares = (int)std::max<int64_t>(1, target / (Hkv * p.row_blocks));
  return p;
}

template <int DT>
hipError_t launch_rows(const Kv4AttentionArgs& a, hipStream_t stream) {
  Layout p = layout_of(a.max_new, a.H, a.Hkv, a.D);
  // no more shares than the tables' room can fill (short contexts: one, and no join)
  int64_t room = (((int64_t)a.max_blocks << a.page_shift) + 31) / 32;
  if (a.window > 0)  // (rounded out to whole steps)
    room = std::min<int64_t>(room, ((int64_t)a.window + a.max_new + a.sinks) / 32 + 4);
  p.shares = (int)std::min<int64_t>(
      p.shares, std::max<int64_t>(1, a.B * (a.kHead + room) / a.kMinShare));
  const int64_t units = (int64_t)p.shares * a.Hkv;
  const dim3 grid((unsigned)((units + 7) / 8 * 8 * p.row_blocks));
  constexpr int S1 = DT <= 4 ? 3 : 2;
  int S = S1;
  auto* kernel = kv4_attention_kernel<DT, 1, S1>;
  if constexpr (DT <= 4) {
    if (p.groups == 2) kernel = kv4_attention_kernel<DT, 2, 4>, S = 4;
  }
  const size_t sums =
      p.key_waves == 1 ? 0 : (size_t)kWaves * p.groups * (2 * DT * 1024 + 16 * sizeof(float2));
  const size_t lds = std::max(sums, (size_t)kWaves * S * Stage<DT>::kBytes);
  const hipError_t e = launch_kernel_lds(kernel, grid, dim3(64 * kWaves), lds, stream, a, p.shares,
                                         p.row_blocks, p.key_waves);
  if (e != hipSuccess || p.shares == 1) return e;
  return a.bf16 ? launch_join<Kv4AttentionArgs, Bfloat, DT>(a, p.shares, stream)
                : launch_join<Kv4AttentionArgs, Half, DT>(a, p.shares, stream);
}

}  // namespace

size_t kv4_attention_workspace_bytes(int64_t B, int64_t max_new, int64_t H, int64_t Hkv,
                                     int64_t D) {
  return parts_bytes(B, max_new, H, D, layout_of(max_new, H, Hkv, D).shares);
}

hipError_t launch_kv4_attention(const Kv4AttentionArgs& a, hipStream_t stream) {
  switch (a.D) {
    case 64: return launch_rows<2>(a, stream);
    case 96: return launch_rows<3>(a, stream);
    case 128: return launch_rows<4>(a, stream);
    default: return launch_rows<8>(a, stream);
  }
}

}  // namespace flexq
