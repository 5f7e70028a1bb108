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
// A wave takes 32-key steps straight from memory into registers, the next step's loads on
// their way while one is worked on, and needs no barrier until a request's end.  Rows are
// columns of the MFMAs (16 a group), so a lane owns one row's statistics, and the keys are
// dealt to the score tiles' rows so that a lane's scores are those that its fragment of P takes:
// row r of score tile t holds key 8 (r / 4) + 4 t + r % 4, lane l keys 8 (l / 16) .. + 7.  Waves
// that the rows leave over take the steps in turn and add up in LDS.
#include "serve_plan.h"

namespace flexq {

namespace {

constexpr int kWaves = 4;
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// A row's largest w is held as 2^(kTop - 1) to 2^(kTop + kLag): fp16 reaches no further up, and
// down to 2^-24, so that small ones keep their bits.
constexpr float kTop = 11.0f, kLag = 4.0f;

// Eight codes of a dword, four instructions and a shift each for c - 8 (even pairs: low four
// bits of the bytes) and 16 (c - 8).
struct Codes {
  uint32_t base = 0x64006400u;
  __device__ __forceinline__ uint32_t low(uint32_t w) const {
    const f16x2 v = __builtin_bit_cast(f16x2, (w & 0x000F000Fu) | base);
    return __builtin_bit_cast(uint32_t, v - f16x2{1032.0f16, 1032.0f16});
  }
  __device__ __forceinline__ uint32_t high(uint32_t w) const {
    const f16x2 v = __builtin_bit_cast(f16x2, (w & 0x00F000F0u) | base);
    return __builtin_bit_cast(uint32_t, v - f16x2{1152.0f16, 1152.0f16});
  }
};

// (by value: a bit cast of a vector's element takes the whole vector's first bits)
__device__ __forceinline__ f16x2 pair_of(uint32_t v) { return __builtin_bit_cast(f16x2, v); }

__device__ __forceinline__ float half_at(const u32x4& v, int e) {
  return half_bits_to_float((uint16_t)(e & 1 ? v[e >> 1] >> 16 : v[e >> 1] & 0xFFFFu));
}

// What a lane holds of a 32-key step: key dwords of tile t (consecutive eights of its quarter of D),
// value dwords (pairs of d, four keys each), scales and offsets of its eight keys.
template <int DT>
struct Step {
  uint32_t k[2][DT];
  uint32_t v[2 * DT];
  u32x4 ks, kb, vs, vb;
  int index;      // of the step in the request
  uint32_t hole;  // bit h: no page behind keys 16 h ..
};

template <int N>
__device__ __forceinline__ void load_dwords(uint32_t (&to)[N], int at, const uint32_t* from, int n) {
  if (n == 4) {
    const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(from));
#pragma unroll
    for (int i = 0; i < 4; ++i) to[at + i] = v[i];
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i) to[at + i] = from[i];
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
template <int DT, int RG>
__global__ __launch_bounds__(64 * kWaves, 2) void kv4_attention_kernel(const Kv4AttentionArgs a,
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

  // a lane's places in a block of 2 D dwords of codes and 64 scales
  const uint32_t* kc = reinterpret_cast<const uint32_t*>(a.kc) +
                       (8 * (c >> 2 & 1) + (c & 3)) * (D / 8) + p * DT;
  const uint32_t* vc = reinterpret_cast<const uint32_t*>(a.vc) + (p & 1) * D;
  const uint16_t* sc = a.scales + (p & 1) * 8;
  const int key_half = c >> 3, value_half = p >> 1;
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
    uint32_t q[RG][DT][4];
    int since[RG];             // first key of the row's window
#pragma unroll
    for (int g = 0; g < RG; ++g) {
      const int row = row0 + 16 * g + c;
      tok[g] = row / group;
      const int64_t at = (int64_t)cu + tok[g];
      in[g] = row < rows && at >= 0 && at < a.T;
      const uint16_t* from = a.q + at * a.q_st + (int64_t)(hk * group + row % group) * a.q_sh + p * 8 * DT;
      float x[DT][8];
      float most = 0.0f;
#pragma unroll
      for (int i = 0; i < DT; ++i) {
        const u32x4 v = in[g] ? *reinterpret_cast<const u32x4*>(from + 8 * i) : u32x4{};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint16_t bits = (uint16_t)(e & 1 ? v[e >> 1] >> 16 : v[e >> 1] & 0xFFFFu);
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
            const int32_t* words = a.mask + at * a.mask_words;
            for (int w = 0; w < a.mask_words && 32 * w < n_new; ++w) {
              const int bits = n_new - 32 * w;
              drafted += __builtin_popcount((uint32_t)words[w] & (bits >= 32 ? ~0u : (1u << bits) - 1u));
            }
          }
        }
        since[g] = ctx + drafted - a.window;
      }
    }
    const bool idle = row0 >= rows;

    const scalar_ptr_t table = (scalar_ptr_t)(a.table + (int64_t)b * a.max_blocks);
    auto page_of = [&](int step, int half) {
      const int pos = step * 32 + half * 16;
      return pos < len ? table[pos >> a.page_shift] : -1;
    };
    auto block_of = [&](int page, int step, int half) {
      if ((unsigned)page >= (unsigned)a.num_pages) return -1;
      return (page * a.Hkv + hk) * per_page + ((step * 2 + half) & (per_page - 1));
    };
    const int first = following(begin + key_wave);
    auto next = [&](int v) { return following(v + key_waves); };
    int page0 = page_of(actual(min(first, end - 1)), 0), page1 = page_of(actual(min(first, end - 1)), 1);
    // Loads step v, whose pages are known, and fetches the pages of the one after it.
    auto load = [&](Step<DT>& s, int v) {
      s.index = actual(v);
      const int b0 = block_of(page0, s.index, 0), b1 = block_of(page1, s.index, 1);
      s.hole = (b0 < 0 ? 1u : 0u) | (b1 < 0 ? 2u : 0u);
      const int64_t kb = max(key_half ? b1 : b0, 0), vb = max(value_half ? b1 : b0, 0);
      const uint32_t* k = kc + kb * (2 * D);
      const uint32_t* vv = vc + vb * (2 * D);
      const uint16_t* sv = sc + vb * 64;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < DT; i += 4)
          load_dwords(s.k[t], i, k + 4 * t * (D / 8) + i, DT - i < 4 ? DT - i : 4);
#pragma unroll
      for (int u = 0; u < 2 * DT; u += 4) {
        const int n = 2 * DT - u < 4 ? 2 * DT - u : 4;
        load_dwords(s.v, u, vv + 16 * u + n * c, n);
      }
      s.ks = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(sv));
      s.kb = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(sv + 16));
      s.vs = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(sv + 32));
      s.vb = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(sv + 48));
      const int after = actual(min(next(v), end - 1));
      page0 = page_of(after, 0);
      page1 = page_of(after, 1);
    };

    f32x4 o[RG][kTiles] = {};
    float m[RG], l[RG], B[RG];  // reference, sum of p, sum of p (b + 8 s)
#pragma unroll
    for (int g = 0; g < RG; ++g) m[g] = -INFINITY, l[g] = B[g] = 0.0f;

    auto work = [&](Step<DT>& s) __attribute__((always_inline)) {
      const Codes codes;
      f32x4 x[RG][2];
#pragma unroll
      for (int g = 0; g < RG; ++g)
#pragma unroll
        for (int t = 0; t < 2; ++t) x[g][t] = f32x4{8 * Q[g], 8 * Q[g], 8 * Q[g], 8 * Q[g]};
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint32_t w = s.k[t][i], w8 = w >> 8;
          const u32x4 f = {codes.low(w), codes.high(w), codes.low(w8), codes.high(w8)};
#pragma unroll
          for (int g = 0; g < RG; ++g)
            x[g][t] = Half::mfma(f, u32x4{q[g][i][0], q[g][i][1], q[g][i][2], q[g][i][3]}, x[g][t]);
        }
      u32x4 vs[RG], vb[RG];  // of what the row attends
      float raw[RG][8];
#pragma unroll
      for (int g = 0; g < RG; ++g) {
        vs[g] = s.vs;
        vb[g] = s.vb;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          raw[g][e] = fmaf(half_at(s.ks, e), x[g][e >> 2][e & 3], half_at(s.kb, e) * Q[g]);
      }
      // Keys that are no context (drafted, or none at all), on no page, or before some row's
      // window: the wave masks.
      const int pos = s.index * 32;
      if (s.hole != 0 || pos + 32 > ctx || (a.window > 0 && pos < ctx + n_new - a.window)) {
        const int pos0 = pos + 8 * p;
        const uint32_t there = (s.hole >> value_half) & 1u ? 0u : low_bits(len - pos0);
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
#pragma unroll
      for (int i = 0; i < DT; ++i) {
        const uint32_t w0 = s.v[2 * i], w1 = s.v[2 * i + 1], w0s = w0 >> 8, w1s = w1 >> 8;
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

    if (!idle && first < end) {
      Step<DT> one, two;
      int v = first;
      load(one, v);
      for (;;) {
        v = next(v);
        load(two, min(v, end - 1));
        work(one);
        if (v >= end) break;
        v = next(v);
        load(one, min(v, end - 1));
        work(two);
        if (v >= end) break;
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
    lds_barrier();  // those of the request before have been read
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
  const int64_t target = 2 * device_cu_count();
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
  auto* kernel = kv4_attention_kernel<DT, 1>;
  if constexpr (DT <= 4) {
    if (p.groups == 2) kernel = kv4_attention_kernel<DT, 2>;
  }
  const size_t lds =
      p.key_waves == 1 ? 0 : (size_t)kWaves * p.groups * (2 * DT * 1024 + 16 * sizeof(float2));
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
