// serve_attention.hip -- attention of drafted tokens over the paged cache.
//
// For the rows of one request and key head (new tokens x query heads of the group), with
// K and V of up to ctx + new tokens: S = scale K Q^T, P = 2^(S log2 e - m) with a running
// maximum m per row, O = V^T P, l = sum P; out = O / l.  One pass over the cache.
//
// Both products are 16x16x32 MFMAs with the rows as columns, so a lane owns one row's
// statistics: D of K Q^T gives lane l the scores of row l % 16 at four keys, and the
// fragment of P that V^T P takes wants eight consecutive keys of that row.  The keys of
// a 32-key step are dealt to the two score tiles so that they are the same eight: row r
// of score tile t holds key 8 (r / 4) + 4 t + r % 4, so lane l ends up with keys
// 8 (l / 16) .. + 7 and no exchange between lanes is needed.  K and V fragments come
// straight from memory, 16 bytes a lane, in the cache's own order.
#include <algorithm>

#include "kernels.h"
#include "serve_device.h"
#include "serve_kernels.h"

namespace flexq {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWaves = 4;

// Workgroups the plan aims at per compute unit.
constexpr int kUnitsPerCu = 4;
// Least 32-key steps of a piece of a request: one a wave.
constexpr int kMinSteps = kWaves;

// (max, sum) over the four lanes that hold one row (l, l ^ 16, l ^ 32, l ^ 48)
__device__ __forceinline__ float row_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float row_sum(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

// the low n bits, n clamped to 0 .. 8
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : (n >= 8 ? 0xFFu : (1u << n) - 1u);
}

}  // namespace

// The plan.  A request of ctx + new tokens has steps = ceil((ctx + new) / 32) 32-key steps and
// is cut into pieces of at most C of them, C = max(kMinSteps, ceil(sum of steps /
// extra)), so that there are at most B + extra pieces and at most 2 extra of requests cut at
// all.  Every workgroup forms it from the lengths (they live on the GPU) and looks up
// its piece; the statistics and sums of cut requests go to the workspace and a second
// kernel joins them in order.  extra = 0: no request is cut.
struct Piece {
  int b;             // request, -1: no such piece
  int index, count;  // piece `index` of the request's `count`
  int part;          // the request's first place in the workspace
};

struct PlanShared {
  uint32_t sum[kWaves];
  int2 scan[kWaves];
  Piece piece;
};

__device__ __forceinline__ int request_rows_tokens(const AttentionArgs& a, int b) {
  return min(max(0, a.cu[b + 1] - a.cu[b]), a.max_new);
}

__device__ __forceinline__ int request_ctx(const AttentionArgs& a, int b) {
  return min(max(0, a.ctx[b]), a.max_blocks << a.page_shift);
}

__device__ __forceinline__ uint32_t request_steps(const AttentionArgs& a, int b) {
  const int n = request_rows_tokens(a, b);
  if (n == 0) return 0;
  const int len = min(request_ctx(a, b) + n, a.max_blocks << a.page_shift);
  return max(1u, (uint32_t)(len + 31) >> 5);  // a request without a key still has rows
}

__device__ Piece find_piece(const AttentionArgs& a, int slot, int extra, PlanShared& sh) {
  constexpr int kThreads = 64 * kWaves;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  uint32_t sum = 0;
  for (int b = b0; b < b1; ++b) sum += request_steps(a, b);
  uint32_t total = sum;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) total += __shfl_xor(total, o);
  if (lane == 0) sh.sum[wave] = total;
  if (tid == 0) sh.piece.b = -1;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) total += sh.sum[w];
  const uint32_t most =
      extra > 0 ? max((uint32_t)kMinSteps, (total + extra - 1) / (uint32_t)extra) : 0xFFFFFFFFu;
  // pieces, and pieces of cut requests, before this thread's requests
  int2 mine = {0, 0};
  for (int b = b0; b < b1; ++b) {
    const uint32_t steps = per == 1 ? sum : request_steps(a, b);
    const int n = steps == 0 ? 0 : (int)((steps - 1) / most) + 1;
    mine.x += n;
    mine.y += n > 1 ? n : 0;
  }
  int2 inc = mine;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const int x = __shfl_up(inc.x, o), y = __shfl_up(inc.y, o);
    if (lane >= o) {
      inc.x += x;
      inc.y += y;
    }
  }
  if (lane == 63) sh.scan[wave] = inc;
  __syncthreads();
  int2 before = {inc.x - mine.x, inc.y - mine.y};
#pragma unroll
  for (int w = 0; w < kWaves; ++w)
    if (w < wave) {
      before.x += sh.scan[w].x;
      before.y += sh.scan[w].y;
    }
  if (slot >= before.x && slot < before.x + mine.x) {
    for (int b = b0; b < b1; ++b) {
      const uint32_t steps = per == 1 ? sum : request_steps(a, b);
      const int n = steps == 0 ? 0 : (int)((steps - 1) / most) + 1;
      if (slot < before.x + n) {
        sh.piece = {b, slot - before.x, n, before.y};
        break;
      }
      before.x += n;
      before.y += n > 1 ? n : 0;
    }
  }
  __syncthreads();
  return sh.piece;
}

// Where the workspace keeps what: (first place, pieces) of every cut request, then for
// every place, key head and row the maximum and sum, then the unnormalized output.
struct Parts {
  int2* plan;
  float2* stat;
  f32x4* out;
};

__host__ __device__ __forceinline__ size_t round16(size_t n) { return (n + 15) / 16 * 16; }

__device__ __forceinline__ Parts parts_of(const AttentionArgs& a, int extra, int rows) {
  char* p = static_cast<char*>(a.workspace);
  Parts w;
  w.plan = reinterpret_cast<int2*>(p);
  p += round16(sizeof(int2) * a.B);
  w.stat = reinterpret_cast<float2*>(p);
  p += round16(sizeof(float2) * 2 * extra * a.Hkv * rows);
  w.out = reinterpret_cast<f32x4*>(p);
  return w;
}

// 0xFFFF in each 16-bit half of v that is infinite or NaN.
template <class E>
__device__ __forceinline__ uint32_t not_finite(uint32_t v) {
  return ((v & E::kExponent) == E::kExponent ? 0xFFFFu : 0u) |
         (((v >> 16) & E::kExponent) == E::kExponent ? 0xFFFF0000u : 0u);
}

// Four elements of a row of out, and its lse.
template <class E>
__device__ __forceinline__ void write_row(const AttentionArgs& a, int64_t t, int h, int d4,
                                          f32x4 acc, float ref, float total) {
  const float by = total != 0.0f ? 1.0f / total : 0.0f;
  u32x2 v;
#pragma unroll
  for (int k = 0; k < 2; ++k)
    v[k] = E::bits(acc[2 * k] * by) | (uint32_t)E::bits(acc[2 * k + 1] * by) << 16;
  *reinterpret_cast<u32x2*>(a.out + (t * a.H + h) * a.D + 4 * d4) = v;
  if (a.lse && d4 == 0)
    a.lse[t * a.H + h] = total != 0.0f ? (ref + log2f(total)) * kLn2 : -INFINITY;
}

// One workgroup = one piece of a request, key head and block of 16 NT rows; its four waves
// take the 32-key steps in turn and join their (m, l, O) through LDS at the end.
//
// The keys' and values' fragments of a wave's next step are on their way while it works
// on the present one: the keys' registers are free after the scores, the values' after
// the second product.
template <class E, int DT, int NT>
__global__ __launch_bounds__(64 * kWaves) void tree_attention_kernel(const AttentionArgs a,
                                                                     int extra, int row_blocks) {
  constexpr int D = 32 * DT;
  constexpr int OT = 2 * DT;  // 16-wide slices of D
  __shared__ PlanShared plan;
  __shared__ f32x4 part[kWaves][16][D / 4 + 1];  // [wave][row][d / 4], padded rows
  __shared__ float stat[2][kWaves][16];

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 15, p = lane >> 4;
  // Workgroups 8 apart share an XCD: the row blocks that read the same keys do.
  const int id = blockIdx.x;
  const int unit = id / (8 * row_blocks) * 8 + id % 8;
  const int hk = unit % a.Hkv;
  const Piece piece = find_piece(a, unit / a.Hkv, extra, plan);
  if (piece.b < 0) return;
  const int b = piece.b;
  const int group = a.H / a.Hkv;
  const int cu = a.cu[b];
  const int n_new = request_rows_tokens(a, b);
  const int ctx = request_ctx(a, b);
  const int rows = n_new * group;
  const int row0 = id / 8 % row_blocks * (16 * NT);
  const Parts parts = parts_of(a, extra, a.max_new * group);
  if (threadIdx.x == 0 && hk == 0 && row0 == 0 && piece.index == 0)
    parts.plan[b] = {piece.part, piece.count};
  if (row0 >= rows) return;
  const int len = min(ctx + n_new, a.max_blocks << a.page_shift);
  const int steps = (int)request_steps(a, b);
  const int begin = (int)((int64_t)steps * piece.index / piece.count);
  int end = (int)((int64_t)steps * (piece.index + 1) / piece.count);
  if (!a.mask) {  // a chain: nothing past the last row's token
    const int last = min(row0 + 16 * NT, rows) - 1;
    end = min(end, (ctx + last / group + 32) >> 5);
  }

  u32x4 qf[NT][DT];
  int tok[NT];  // the row's token in its request
#pragma unroll
  for (int rt = 0; rt < NT; ++rt) {
    const int r = row0 + rt * 16 + c;
    tok[rt] = r / group;
    const int64_t t = (int64_t)cu + tok[rt];
    const bool in = r < rows && t >= 0 && t < a.T;
    const uint16_t* src = a.q + t * a.q_st + (int64_t)(hk * group + r % group) * a.q_sh + 8 * p;
#pragma unroll
    for (int ks = 0; ks < DT; ++ks)
      qf[rt][ks] = in ? *reinterpret_cast<const u32x4*>(src + 32 * ks) : u32x4{};
  }

  const int per_page = 1 << (a.page_shift - 4);  // 16-token blocks of a page
  const int32_t* table = a.table + (int64_t)b * a.max_blocks;
  // Table entry of the 16 tokens at 32 step + 16 half (-1 past the request's tokens), and
  // the 16-token block of the cache it stands for (-1 where there is none).
  auto page_of = [&](int step, int half) {
    const int pos = step * 32 + half * 16;
    return pos < len ? table[pos >> a.page_shift] : -1;
  };
  auto block_of = [&](int id, int step, int half) {
    if ((unsigned)id >= (unsigned)a.num_pages) return -1;
    return (id * a.Hkv + hk) * per_page + ((step * 2 + half) & (per_page - 1));
  };

  f32x4 o[NT][OT] = {};
  float m[NT], l[NT];
#pragma unroll
  for (int rt = 0; rt < NT; ++rt) {
    m[rt] = -INFINITY;
    l[rt] = 0.0f;
  }
  const float scale = a.scale * kLog2e;

  u32x4 kf[2][DT], vf[OT];
  const int koff = (8 * ((c >> 2) & 1) + (c & 3)) * 32 + 8 * p;
  const int voff = c * 16 + 8 * (p & 1);
  auto load_keys = [&](int block) {
    const uint16_t* src = a.kc + (int64_t)max(block, 0) * (16 * D) + koff;
#pragma unroll
    for (int ks = 0; ks < DT; ++ks)
#pragma unroll
      for (int t = 0; t < 2; ++t)
        kf[t][ks] = *reinterpret_cast<const u32x4*>(src + ks * 512 + t * 128);
  };
  auto load_values = [&](int block) {
    const uint16_t* src = a.vc + (int64_t)max(block, 0) * (16 * D) + voff;
#pragma unroll
    for (int dt = 0; dt < OT; ++dt) vf[dt] = *reinterpret_cast<const u32x4*>(src + dt * 256);
  };

  int step = begin + wave;
  int vblk = -1, kid = -1, vid = -1;
  if (step < end) {
    load_keys(block_of(page_of(step, c >> 3), step, c >> 3));
    vblk = block_of(page_of(step, p >> 1), step, p >> 1);
    load_values(vblk);
    kid = page_of(step + kWaves, c >> 3);
    vid = page_of(step + kWaves, p >> 1);
  }
  for (; step < end; step += kWaves) {
    const int next = step + kWaves;
    const bool more = next < end;
    f32x4 s[NT][2] = {};
#pragma unroll
    for (int ks = 0; ks < DT; ++ks)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int rt = 0; rt < NT; ++rt) s[rt][t] = E::mfma(kf[t][ks], qf[rt][ks], s[rt][t]);
    __builtin_amdgcn_sched_barrier(0);
    const int vnext = block_of(vid, next, p >> 1);
    if (more) load_keys(block_of(kid, next, c >> 3));
    kid = page_of(next + kWaves, c >> 3);
    vid = page_of(next + kWaves, p >> 1);
    __builtin_amdgcn_sched_barrier(0);

    // Keys that are no context (drafted, or none at all) or on no page: the wave masks.
    const int key0 = step * 32 + 8 * p;  // this lane's first key
    const bool masked = __ballot(vblk < 0 || key0 + 8 > ctx) != 0;
    const uint32_t there = vblk < 0 ? 0u : low_bits(len - key0);  // keys that exist
    bool poison = false;  // a value in this step is infinite or NaN
    uint32_t seen[NT];
    u32x4 hi[NT], lo[NT];
#pragma unroll
    for (int rt = 0; rt < NT; ++rt) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = s[rt][e >> 2][e & 3] * scale;
      seen[rt] = 0xFFu;
      if (masked) {
        // attended keys among this lane's eight: the context, then the tree's bits (or,
        // for a chain, the tokens up to the row's own)
        const int j0 = key0 - ctx;  // drafted index of the first key (may be negative)
        if (a.mask) {
          seen[rt] = low_bits(-j0);
          const int64_t t = (int64_t)cu + tok[rt];
          if (j0 > -8 && tok[rt] < n_new && t >= 0 && t < a.T) {
            const int32_t* words = a.mask + t * a.mask_words;
            const int w = j0 >> 5;
            const uint32_t w0 = w >= 0 && w < a.mask_words ? (uint32_t)words[w] : 0u;
            const uint32_t w1 = w + 1 < a.mask_words ? (uint32_t)words[w + 1] : 0u;
            seen[rt] |= (uint32_t)(((uint64_t)w1 << 32 | w0) >> (j0 & 31)) & 0xFFu;
          }
        } else {
          seen[rt] = low_bits(tok[rt] + 1 - j0);
        }
        seen[rt] &= there;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (!((seen[rt] >> e) & 1u)) x[e] = -INFINITY;
      }
      float top = x[0];
#pragma unroll
      for (int e = 1; e < 8; ++e) top = fmaxf(top, x[e]);
      top = row_max(top);
      if (__ballot(top > m[rt])) {  // most steps raise no row's maximum
        top = fmaxf(m[rt], top);
        const float by = __builtin_amdgcn_exp2f(m[rt] - (top == -INFINITY ? 0.0f : top));
        m[rt] = top;
        l[rt] *= by;
#pragma unroll
        for (int dt = 0; dt < OT; ++dt)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[rt][dt][i] *= by;
      }
      const float ref = m[rt] == -INFINITY ? 0.0f : m[rt];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v0 = __builtin_amdgcn_exp2f(x[2 * i] - ref);
        const float v1 = __builtin_amdgcn_exp2f(x[2 * i + 1] - ref);
        l[rt] += v0 + v1;
        const u32x2 parts2 = E::split(v0, v1);
        hi[rt][i] = parts2[0];
        lo[rt][i] = parts2[1];
      }
    }

    if (masked) {
      // values of keys that do not exist are zeroed, and infinite and NaN ones for now
      uint32_t keep[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        keep[i] = ((there >> (2 * i)) & 1u) * 0xFFFFu | ((there >> (2 * i + 1)) & 1u) * 0xFFFF0000u;
      bool bad = false;
#pragma unroll
      for (int dt = 0; dt < OT; ++dt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t v = vf[dt][i] & keep[i], ex = not_finite<E>(v);
          bad |= ex != 0;
          vf[dt][i] = v & ~ex;
        }
      poison = __ballot(bad) != 0;
    }
#pragma unroll
    for (int dt = 0; dt < OT; ++dt)
#pragma unroll
      for (int rt = 0; rt < NT; ++rt) {
        o[rt][dt] = E::mfma(vf[dt], hi[rt], o[rt][dt]);
        o[rt][dt] = E::mfma(vf[dt], lo[rt], o[rt][dt]);
      }
    if (poison) {
      // Infinite and NaN values reach only the rows that attend their keys: one key at a
      // time, and a row that does not attend it keeps its sum.
      const uint16_t* src = a.vc + (int64_t)max(vblk, 0) * (16 * D) + voff;
      for (int k = 0; k < 32; ++k) {
        const int e = k & 7;
        const bool mine = p == (k >> 3) && ((there >> e) & 1u);
#pragma unroll
        for (int dt = 0; dt < OT; ++dt) {
          const uint32_t v = mine ? src[dt * 256 + e] : 0u;
          const u32x4 one_v = {v & not_finite<E>(v), 0u, 0u, 0u};
#pragma unroll
          for (int rt = 0; rt < NT; ++rt) {
            const uint32_t pair = e < 4 ? (e < 2 ? hi[rt][0] : hi[rt][1])
                                        : (e < 6 ? hi[rt][2] : hi[rt][3]);
            const u32x4 one_p = {mine ? (pair >> (16 * (e & 1))) & 0xFFFFu : 0u, 0u, 0u, 0u};
            const bool attends = (__shfl((int)seen[rt], (k >> 3) * 16 + c) >> e) & 1;
            const f32x4 with = E::mfma(one_v, one_p, o[rt][dt]);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[rt][dt][i] = attends ? with[i] : o[rt][dt][i];
          }
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    vblk = vnext;
    if (more) load_values(vblk);
    __builtin_amdgcn_sched_barrier(0);
  }

  // Join the four waves, one 16-row tile at a time.
#pragma unroll
  for (int rt = 0; rt < NT; ++rt) {
    const float sum = row_sum(l[rt]);
#pragma unroll
    for (int dt = 0; dt < OT; ++dt) part[wave][c][4 * dt + p] = o[rt][dt];
    if (p == 0) {
      stat[0][wave][c] = m[rt];
      stat[1][wave][c] = sum;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * (D / 4); i += 64 * kWaves) {
      const int r = i / (D / 4), d4 = i % (D / 4);
      const int row = row0 + rt * 16 + r;
      const int64_t t = (int64_t)cu + row / group;
      float top = -INFINITY, total = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top = fmaxf(top, stat[0][w][r]);
      const float ref = top == -INFINITY ? 0.0f : top;
      f32x4 acc = {};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float by = __builtin_amdgcn_exp2f(stat[0][w][r] - ref);
        total = fmaf(stat[1][w][r], by, total);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] = fmaf(part[w][r][d4][k], by, acc[k]);
      }
      if (row < rows) {
        if (piece.count > 1) {
          const int64_t at =
              ((int64_t)(piece.part + piece.index) * a.Hkv + hk) * (a.max_new * group) + row;
          parts.out[at * (D / 4) + d4] = acc;
          if (d4 == 0) parts.stat[at] = {top, total};
        } else if (t >= 0 && t < a.T) {
          write_row<E>(a, t, hk * group + row % group, d4, acc, ref, total);
        }
      }
    }
    __syncthreads();
  }
}

// Joins the pieces of cut requests in order: thread = four elements of one row.
template <class E, int DT>
__global__ __launch_bounds__(256) void join_pieces_kernel(const AttentionArgs a, int extra) {
  constexpr int D = 32 * DT;
  constexpr int kRows = 256 / (D / 4);
  const int b = blockIdx.z, hk = blockIdx.y;
  const int group = a.H / a.Hkv;
  const int row = blockIdx.x * kRows + threadIdx.x / (D / 4), d4 = threadIdx.x % (D / 4);
  if (threadIdx.x >= kRows * (D / 4) || row >= request_rows_tokens(a, b) * group) return;
  const Parts parts = parts_of(a, extra, a.max_new * group);
  const int2 plan = parts.plan[b];
  if (plan.y <= 1) return;
  const int64_t stride = (int64_t)a.Hkv * (a.max_new * group);
  const int64_t at = ((int64_t)plan.x * a.Hkv + hk) * (a.max_new * group) + row;
  float top = -INFINITY, total = 0.0f;
  f32x4 acc = {};
  for (int i = 0; i < plan.y; ++i) top = fmaxf(top, parts.stat[at + i * stride].x);
  const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll 4
  for (int i = 0; i < plan.y; ++i) {
    const float2 s = parts.stat[at + i * stride];
    const f32x4 o = parts.out[(at + i * stride) * (D / 4) + d4];
    const float by = __builtin_amdgcn_exp2f(s.x - ref);
    total = fmaf(s.y, by, total);
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = fmaf(o[k], by, acc[k]);
  }
  const int64_t t = (int64_t)a.cu[b] + row / group;
  if (t >= 0 && t < a.T) write_row<E>(a, t, hk * group + row % group, d4, acc, ref, total);
}

namespace {

// How a call is laid out: 16-row tiles a wave holds, row blocks, pieces to cut into
struct Layout {
  int nt, row_blocks, extra;
};

Layout layout_of(int64_t max_new, int64_t H, int64_t Hkv, int64_t D) {
  Layout p;
  const int64_t rows = max_new * (H / Hkv);
  p.nt = rows <= 16 || D > 128 ? 1 : 2;
  p.row_blocks = (int)((rows + 16 * p.nt - 1) / (16 * p.nt));
  const int64_t target = kUnitsPerCu * device_cu_count();
  const int64_t units = Hkv * p.row_blocks;
  p.extra = units >= target ? 0 : (int)((target + units - 1) / units);
  return p;
}

template <class E, int DT>
hipError_t launch_rows(const AttentionArgs& a, hipStream_t stream) {
  const Layout p = layout_of(a.max_new, a.H, a.Hkv, a.D);
  const int64_t units = (int64_t)(a.B + p.extra) * a.Hkv;
  const dim3 grid((unsigned)((units + 7) / 8 * 8 * p.row_blocks));
  auto* kernel = tree_attention_kernel<E, DT, 1>;
  if constexpr (DT <= 4)
    if (p.nt == 2) kernel = tree_attention_kernel<E, DT, 2>;
  const hipError_t e =
      launch_kernel(kernel, grid, dim3(64 * kWaves), stream, a, p.extra, p.row_blocks);
  if (e != hipSuccess || p.extra == 0) return e;
  const int rows = a.max_new * (a.H / a.Hkv), per = 256 / (8 * DT);
  return launch_kernel(join_pieces_kernel<E, DT>,
                       dim3((unsigned)((rows + per - 1) / per), (unsigned)a.Hkv, (unsigned)a.B),
                       dim3(256), stream, a, p.extra);
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
  const Layout p = layout_of(max_new, H, Hkv, D);
  const size_t places = (size_t)2 * p.extra * H * max_new;  // key head x row
  return round16(sizeof(int2) * B) + round16(sizeof(float2) * places) + sizeof(float) * places * D;
}

hipError_t launch_tree_attention(const AttentionArgs& a, bool bf16, hipStream_t stream) {
  return bf16 ? launch_width<Bfloat>(a, stream) : launch_width<Half>(a, stream);
}

}  // namespace flexq
