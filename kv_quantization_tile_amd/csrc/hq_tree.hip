// hq_tree.hip -- attention of a tree of drafted tokens over the paged SRFT cache (the mathematics and the operands'
// layout: hq_attend.hip).
//
// The drafts are a sequence's last cached tokens.  Draft i sees the held tokens before them and, of the drafts, its path from
// the root: a bit each, found by walking up from the draft in LDS.  Held tokens need no bits, so only the steps that reach the
// drafts look at them.
//
// Rows are queries x heads of the group, of a sequence and a KV head; a workgroup takes a tile of them and one split of the
// tokens.  Up to 32 rows, or little work: its four wavefronts take 32 tokens in turn, every wavefront with all the rows, so that codes become
// operands in registers and nothing is shared but the join at the end.  Otherwise operands are made once, 16 tokens by each
// wavefront, and shared through LDS, and each wavefront owns 16 or 32 rows.  (32 rows a workgroup for 64 and 256 of them makes
// the operands two and eight times: 92 us against 71 for 16 drafts on 16 x 8192 tokens, 95 against 75 for 64 on 32768;
// 64 rows in one wavefront's registers, one wavefront a SIMD, 142 and 136.)
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/hq.h"
#include "hq_attend_device.h"

namespace hq_kv {

constexpr int kMaxTree = 256;  // drafts of a sequence

struct TreeArgs {
  const int32_t* parents;
  uint32_t tiles, splits, chunk;  // of a sequence, at most; of a tile, and their tokens
  float *po, *pml;                // [seqs][tiles][heads][splits][16 R], 128 and 2 values
};

// Tokens that some row of [r0, r0 + count) sees, as one range: draft i sees drafts up to itself, and no fewer held tokens
// than a root.
__device__ __forceinline__ void tree_range(const AttendArgs& a, const Seq& s, uint32_t r0, uint32_t count, int32_t* lo, int32_t* hi) {
  const uint32_t rows = (uint32_t)s.m * a.group;
  if (r0 >= rows) {
    *lo = *hi = 0;
    return;
  }
  int32_t x;
  visible(a, s, 0, lo, &x);
  visible(a, s, (int32_t)query_of(a, (r0 + count < rows ? r0 + count : rows) - 1u), &x, hi);
  if (*lo > *hi) *lo = *hi;
}
// Held tokens that every row up to query `last` sees: those that a draft as deep as its index sees.
__device__ __forceinline__ void tree_common(const AttendArgs& a, const Seq& s, uint32_t last, int32_t* lo, int32_t* hi) {
  int32_t x;
  visible(a, s, (int32_t)last, lo, &x);
  *hi = s.back > 0 ? s.back : 0;
}

template <int QUERIES>
struct Tree {
  int32_t parent[kMaxTree];
  uint32_t seen[QUERIES][kMaxTree / 32];
  uint32_t depth[QUERIES];
};
// Walks up from queries [i0, i0 + count) with the workgroup's threads.  With a window, of a query's path the last `window`.  A
// parent that is not before its draft counts as none.
template <int QUERIES>
__device__ __forceinline__ void climb(const AttendArgs& a, const int32_t* parents, const Seq& s, uint32_t i0, uint32_t count, Tree<QUERIES>& t) {
  for (uint32_t i = threadIdx.x; i < i0 + count; i += kAttBlock) {
    const int32_t p = parents[(uint64_t)s.q0 + i];
    t.parent[i] = p >= 0 && p < (int32_t)i ? p : -1;
  }
  __syncthreads();
  for (uint32_t q = threadIdx.x; q < count; q += kAttBlock) {
#pragma unroll
    for (int w = 0; w < kMaxTree / 32; ++w) t.seen[q][w] = 0;
    uint32_t depth = 0;
    for (int32_t i = (int32_t)(i0 + q); i >= 0; i = t.parent[i], ++depth)
      if (a.window == 0 || depth < a.window) t.seen[q][i >> 5] |= 1u << (i & 31);
    t.depth[q] = depth - 1u;
  }
  __syncthreads();
}
// The first held token that a query of this depth sees.
__device__ __forceinline__ int32_t tree_lo(const AttendArgs& a, const Seq& s, uint32_t depth) {
  const int64_t l = a.window ? (int64_t)s.back + depth + 1 - (int64_t)a.window : 0;
  return l < 0 ? 0 : l > 0x7FFFFFFF ? 0x7FFFFFFF : (int32_t)l;
}

// Whether a query sees token `tok`, which its tile sees; `lo` is the first held token it sees.  Without branches, here and where a score
// is hidden by it: with short-circuit conditions around stores to single scores, scores were seen to stay unmasked in this compiler's
// output (ROCm 7.2.0's clang at -O3; the same source masked them with a printf beside it).
template <int QUERIES>
__device__ __forceinline__ bool tree_sees(const Tree<QUERIES>& t, int32_t back, uint32_t query, int32_t lo, int32_t tok) {
  const uint32_t j = (uint32_t)(tok - back) & (kMaxTree - 1);
  const bool draft = (t.seen[query][j >> 5] >> (j & 31u)) & 1u;
  return bool(((tok < back) & (tok >= lo)) | ((tok >= back) & draft));
}

// What a workgroup takes.  Consecutive workgroups go to the 8 XCDs in turn: the tiles of one (sequence, head, split), which
// read the same codes, meet in one XCD's L2.
struct TreeItem {
  uint32_t b, h, split, tile;
};
__device__ __forceinline__ TreeItem tree_item(const AttendArgs& a, const TreeArgs& g) {
  const uint32_t item = blockIdx.x / (8u * g.tiles) * 8u + blockIdx.x % 8u;
  return {item / g.splits / a.heads, item / g.splits % a.heads, item % g.splits, blockIdx.x / 8u % g.tiles};
}

// 32 rows on 32 x 4096 tokens: 58 us with the join, 201 MB at 3.5 TB/s; 26 rows on 64 ragged sequences of up to 2001 at 8 bits
// 46 us.  A step of 32 tokens and 32 rows is about 560 vector instructions, 380 of them for the operands, which bound it where
// memory does not.  One sequence of 301 tokens takes 15 us: 2 until its codes are asked for, 3 for its rows, 1 for the
// tree, 4 for three steps, 3 for the join and the way back.
template <int BITS, int R>
__global__ __launch_bounds__(kAttBlock, R == 2 || BITS == 8 ? 2 : 3) void attend_tree_kernel(AttendArgs a, TreeArgs g, Tables K) {
  constexpr uint32_t kRows = 16u * R;
  __shared__ __align__(16) float s_o[kAttWaves][16][kPad];
  __shared__ __align__(16) _Float16 s_q[kRows][kD + 8];
  __shared__ float s_f[kRows], s_m[kAttWaves][kRows], s_l[kAttWaves][kRows], s_lam[2][kD];
  __shared__ Tree<(int)kRows> s_tree;
  const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 15u, b4 = lane >> 4;
  const TreeItem at = tree_item(a, g);
  const uint32_t b = at.b, h = at.h, split = at.split, tile = at.tile;
  if (b >= a.seqs) return;
  const Seq s = seq_of(a, b);
  const uint32_t r0 = tile * kRows, all = (uint32_t)s.m * a.group;
  if (r0 >= all) return;
  const uint32_t rows = all - r0 < kRows ? all - r0 : kRows, i0 = query_of(a, r0), last = query_of(a, r0 + rows - 1u);
  int32_t lo, hi;
  tree_range(a, s, r0, kRows, &lo, &hi);
  int32_t t0 = (lo & ~15) + (int32_t)(split * g.chunk), t1 = t0 + (int32_t)g.chunk;
  t1 = t1 < hi ? t1 : hi;
  if (a.pages == 0) t1 = t0;
  if (t0 >= t1 && g.splits > 1) return;  // the same for the whole workgroup
  const uint32_t P = 1u << a.page_log2;
  const uint64_t page_size = (uint64_t)P * Page<BITS>::kToken;

  Share<BITS> cur[2], nxt[2];
  auto load = [&](int32_t t, int32_t page, Share<BITS>& sh) __attribute__((always_inline)) {
    // an absent page's place is taken by page 0, masked below
    const uint8_t* p = a.cache + ((uint64_t)(page < 0 ? 0 : page) * a.heads + h) * page_size;
    load_keys<BITS>(p, P, (uint32_t)t & (P - 1u), lane, sh);
    load_values<BITS>(p, P, (uint32_t)t & (P - 1u), lane, sh);
  };
  constexpr int32_t kStep = 32 * kAttWaves;
  int32_t t = t0 + 32 * (int32_t)wave;
  int32_t pg0 = page_of(a, b, t, t1), pg1 = page_of(a, b, t + 16, t1);
  if (t < t1) {
    load(t, pg0, cur[0]);
    load(t + 16, pg1, cur[1]);
  }
  int32_t en0 = entry_of(a, b, t + kStep, t1), en1 = entry_of(a, b, t + kStep + 16, t1);

  stage_tables(K, s_lam);
  {  // the rows: 16 at a time, four to a wavefront, 16 lanes each
    const LaneForward forward = lane_forward(K, n);
#pragma unroll 1
    for (uint32_t r = threadIdx.x >> 4; r < kRows; r += 16u) {
      float f = 1.0f;
      if ((r & ~3u) < rows) f = rotate_row<BITS>(a, K, s_lam[0], h, (uint32_t)s.q0 * a.group + r0 + r, r < rows, n, forward, s_q[r], nullptr);
      else *reinterpret_cast<f16x8*>(&s_q[r][8 * n]) = (f16x8)(_Float16)0.0f;
      if (n == 0) s_f[r] = f;
    }
  }
  // splits of held tokens alone need no tree, unless a window ends among them
  const bool climbs = a.window || t1 > s.back;
  if (climbs) climb(a, g.parents, s, i0, last - i0 + 1u, s_tree);
  else __syncthreads();

  const bool cap = a.cap_in > 0.0f;
  f16x8 q[R][4];
  float qf[R], eff[R], m[R], poison[R];
  uint32_t query[R];
  int32_t row_lo[R];
  f32x4 o[R][8], ones[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int j = 0; j < 4; ++j) q[r][j] = *reinterpret_cast<const f16x8*>(&s_q[16 * r + n][8 * (4 * b4 + j)]);
    qf[r] = s_f[16 * r + n];
    eff[r] = cap ? 1.0f : qf[r];  // scores are eff sc: the product with qf waits for the exponent's fma
    m[r] = kLowest;
    poison[r] = 0.0f;
    query[r] = 16u * r + n < rows ? query_of(a, r0 + 16u * r + n) - i0 : 0u;
    row_lo[r] = climbs ? tree_lo(a, s, s_tree.depth[query[r]]) : 0;
    ones[r] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 8; ++i) o[r][i] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  }
  // the tokens every row sees need no mask (rows past the last are products with zero)
  int32_t all_lo, all_hi;
  tree_common(a, s, last, &all_lo, &all_hi);
  for (; t < t1; t += kStep) {
    const bool there[2] = {pg0 >= 0, pg1 >= 0};
    pg0 = page_in(a, en0);
    pg1 = page_in(a, en1);
    en0 = entry_of(a, b, t + 2 * kStep, t1);
    en1 = entry_of(a, b, t + 2 * kStep + 16, t1);
    if (t + kStep < t1) {
      load(t + kStep, pg0, nxt[0]);
      load(t + kStep + 16, pg1, nxt[1]);
    }
    uint32_t large = 0, gone = 0;  // bit u: shrunk keys, bit 2 + u: shrunk values; tokens that take no part
    f32x4 sc[R][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (__builtin_amdgcn_ballot_w64(odd_scales<BITS>(most(cur[u].ks[0], cur[u].ks[1])))) {
        const int32_t tok = t + 16 * u + (int32_t)n;
        if (!there[u] || tok < lo || tok >= t1) cur[u].ks[0] = cur[u].ks[1] = 0u;  // a token that no row sees may hold anything
        gone |= gone_keys(cur[u].ks) << (16 * u);
        if (shrink<BITS>(cur[u].ks)) large |= 1u << u;
      }
      f16x8 kh[4], kl[4];
      key_operands<BITS, false>(cur[u], kh, kl);
#pragma unroll
      for (int r = 0; r < R; ++r) sc[r][u] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < R; ++r) sc[r][u] = mfma(kh[j], q[r][j], sc[r][u]);
    }
    if (large & 3u) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int u = 0; u < 2; ++u) sc[r][u] *= (large >> u) & 1u ? kShrunk : 1.0f;
    }
    if (cap) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 8; ++i) sc[r][i >> 2][i & 3] = a.cap_out * tanh32(sc[r][i >> 2][i & 3] * qf[r] * a.cap_in);
    }
    // Value vectors with NaN scales make the rows that see them NaN and no other (0 NaN in the product would reach every row):
    // their scales count as 0, and the rows are poisoned.
    uint32_t bad[2] = {0u, 0u};
    const bool odd = __builtin_amdgcn_ballot_w64(odd_scales<BITS>(__builtin_elementwise_max(most(cur[0].vs[0], cur[0].vs[1]), most(cur[1].vs[0], cur[1].vs[1])))) != 0u;
    if (odd) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t drop = bad[u] = bad_scales(cur[u].vs);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int32_t tok = t + 16 * u + 4 * (int32_t)b4 + i;
          if (!there[u] || tok < lo || tok >= t1) drop |= 1u << i;  // as with the keys
        }
        // the 16 lanes of a token hold one group each: a vector with one NaN scale is NaN as a whole, and poisons by each of them
        drop_scales(cur[u].vs, drop);
        if (shrink<BITS>(cur[u].vs)) large |= 4u << u;
      }
    }
    if (gone || !(there[0] && there[1] && t >= all_lo && t + 32 <= all_hi && t + 32 <= t1)) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int32_t tok = t + 16 * (i >> 2) + 4 * (int32_t)b4 + (i & 3);
          const bool hidden = (gone >> (4u * b4) >> (16 * (i >> 2) + (i & 3))) & 1u;
          const bool shown = !hidden & there[i >> 2] & (tok < t1) & tree_sees(s_tree, s.back, query[r], row_lo[r], tok);
          sc[r][i >> 2][i & 3] = shown ? sc[r][i >> 2][i & 3] : -__builtin_inff();
        }
    }
    if (odd) {
      // which of 16 tokens have a NaN scale in some lane
      uint32_t word[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        word[u] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t votes = __builtin_amdgcn_ballot_w64((bad[u] >> i) & 1u);
#pragma unroll
          for (int k = 0; k < 4; ++k) word[u] |= (votes >> (16 * k)) & 0xFFFFu ? 1u << (4 * k + i) : 0u;
        }
        drop_scales(cur[u].vs, (word[u] >> (4 * b4)) & 15u);
      }
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if ((word[i >> 2] >> (4 * b4 + (i & 3))) & 1u && sc[r][i >> 2][i & 3] != -__builtin_inff()) poison[r] = __builtin_nanf("");
    }
    float top[R];
    bool rise = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      top[r] = sc[r][0][0];
#pragma unroll
      for (int i = 1; i < 8; ++i) top[r] = fmaxf(top[r], sc[r][i >> 2][i & 3]);
      top[r] *= eff[r];
      rise |= top[r] > m[r] + kSlack;
    }
    // with shrunk values, P goes up to 2^15 against the maximum itself
    if (large >= 4u || __builtin_amdgcn_ballot_w64(rise)) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float mn = fmaxf(m[r], blocks_max(top[r])), f = __builtin_amdgcn_exp2f(m[r] - mn);
        m[r] = mn;
        ones[r] *= f;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[r][i] *= f;
      }
    }
    f16x8 p[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float base = kPScaleLog2 - m[r];
      U32x4 x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[r][i >> 1][2 * (i & 1)], eff[r], base));
        const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[r][i >> 1][2 * (i & 1) + 1], eff[r], base));
        x.v[i] = u2((f16x2){(_Float16)p0, (_Float16)p1});
      }
      p[r] = frag(x);
      // the sum of the rounded P, the one the output is weighted with, is one more product
      ones[r] = mfma((f16x8)(_Float16)1.0f, p[r], ones[r]);
      if (large >= 4u) {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[r][i] *= (large >> (2 + (i >> 2))) & 1u ? (_Float16)kShrunk : (_Float16)1.0f;
      }
    }
    uint32_t v0[8][2], v1[8][2];
    value_operands<BITS>(cur[0], v0);
    value_operands<BITS>(cur[1], v1);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const U32x4 v = {{v0[i][0], v0[i][1], v1[i][0], v1[i][1]}};
#pragma unroll
      for (int r = 0; r < R; ++r) o[r][i] = mfma(frag(v), p[r], o[r][i]);
    }
    cur[0] = nxt[0];
    cur[1] = nxt[1];
  }

  // the wavefronts' parts, joined in order, 16 rows at a time
#pragma unroll
  for (int r = 0; r < R; ++r) {
    poison[r] = blocks_sum(poison[r]);
    if (b4 == 0) {
      s_m[wave][16 * r + n] = m[r];
      s_l[wave][16 * r + n] = ones[r][0];
    }
  }
  __syncthreads();
  const uint32_t row = threadIdx.x >> 4;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (16u * r >= rows) break;  // the same for the whole workgroup
    float mm = s_m[0][16 * r + n];
#pragma unroll
    for (int w = 1; w < kAttWaves; ++w) mm = fmaxf(mm, s_m[w][16 * r + n]);
    const float f = __builtin_amdgcn_exp2f(m[r] - mm);
    if (r) __syncthreads();
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int i = 0; i < 8; i += 4)
        *reinterpret_cast<f32x4*>(&s_o[wave][n][8 * (4 * b4 + c) + i]) =
            (f32x4){o[r][i][c] * f + poison[r], o[r][i + 1][c] * f + poison[r], o[r][i + 2][c] * f + poison[r], o[r][i + 3][c] * f + poison[r]};
    __syncthreads();
    const uint32_t x = 16u * r + row;
    if ((x & ~3u) >= rows) continue;
    float total = 0.0f, mr = s_m[0][x], y[8];
#pragma unroll
    for (int w = 1; w < kAttWaves; ++w) mr = fmaxf(mr, s_m[w][x]);
#pragma unroll
    for (int w = 0; w < kAttWaves; ++w) total += s_l[w][x] * __builtin_amdgcn_exp2f(s_m[w][x] - mr);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = s_o[0][row][8 * n + i];
#pragma unroll
    for (int w = 1; w < kAttWaves; ++w)
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] += s_o[w][row][8 * n + i];
    if (g.splits == 1) {
      store_row<BITS>(a, K, s_lam[1], s, h, r0 + x, n, lane_inverse(K, n), y, total);
      continue;
    }
    const uint64_t p = ((((uint64_t)b * g.tiles + tile) * a.heads + h) * g.splits + split) * kRows + x;
    *reinterpret_cast<f32x4*>(g.po + p * kD + 8 * n) = (f32x4){y[0], y[1], y[2], y[3]};
    *reinterpret_cast<f32x4*>(g.po + p * kD + 8 * n + 4) = (f32x4){y[4], y[5], y[6], y[7]};
    if (n == 0) *reinterpret_cast<f32x2*>(g.pml + p * 2) = (f32x2){mr, total};
  }
}

// More rows: the queries' rows transformed once, to the workspace, 16 a workgroup.
template <int BITS>
__global__ __launch_bounds__(kAttBlock) void rotate_tree_kernel(AttendArgs a, Tables K) {
  __shared__ __align__(16) _Float16 s_q[16][kD + 8];
  __shared__ float s_lam[2][kD];
  stage_tables(K, s_lam);
  const uint32_t l = threadIdx.x & 15u, k = threadIdx.x >> 4, per = (a.rows + 15u) / 16u, h = blockIdx.x / per, row = blockIdx.x % per * 16u + k;
  const float f = rotate_row<BITS>(a, K, s_lam[0], h, row, row < a.rows, l, lane_forward(K, l), s_q[k], nullptr);
  // a row is written and read by the same wavefront
  wave_sync();
  if (row >= a.rows) return;
  const uint64_t at = (uint64_t)h * a.rows + row;
  if (l == 0) a.qf[at] = f;
  *reinterpret_cast<f16x8*>(a.qhi + at * kD + 8 * l) = *reinterpret_cast<const f16x8*>(&s_q[k][8 * l]);
}

struct TreeStage {
  f16x8 k[kAttWaves][4][64];      // [16 tokens][step][lane]
  f16x8 v[kAttWaves / 2][8][64];  // [32 tokens][coordinate][lane]
};

// 64 drafts (256 rows) on 32768 tokens: 66 us, 520 TFLOP/s; 16 (64 rows) on 16 ragged sequences of up to 8192: 59 us, 385 TFLOP/s.
// Matrix instructions take a fifth of the cycles and vector instructions a third: a turn of 64 tokens is a chain of loads,
// operands, a barrier and products, which two to four workgroups a CU overlap in part, and starts and ends are 28 % of the launch.
// R = 1 (up to 64 rows): one stage, four workgroups a CU.  R = 2: two stages, so that a turn has one barrier, and two workgroups.
template <int R>
constexpr size_t tree_lds() { return R == 1 ? sizeof(float) * kAttWaves * 16 * kPad : 2 * sizeof(TreeStage); }

template <int BITS, int R>
__global__ __launch_bounds__(kAttBlock, R == 1 ? 4 : 2) void attend_tree_many_kernel(AttendArgs a, TreeArgs g, Tables K) {
  constexpr int32_t kTok = 16 * kAttWaves;
  constexpr uint32_t kRows = 16u * R * kAttWaves;
  extern __shared__ __align__(16) uint8_t raw[];
  TreeStage* st = reinterpret_cast<TreeStage*>(raw);
  float(*s_o)[16][kPad] = reinterpret_cast<float(*)[16][kPad]>(raw);  // [wavefront], after the last product
  // bits 0..15: tokens with NaN value scales, 16..31: tokens that take no part; bits 0 and 1: shrunk keys, values
  __shared__ uint2 s_flags[2][kAttWaves];
  __shared__ Tree<(int)kRows> s_tree;
  const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 15u, b4 = lane >> 4;
  const TreeItem at = tree_item(a, g);
  if (at.b >= a.seqs) return;
  const uint32_t h = at.h;
  const Seq s = seq_of(a, at.b);
  const uint32_t rows = (uint32_t)s.m * a.group, r0 = at.tile * kRows, w0 = r0 + wave * 16u * R;
  if (r0 >= rows) return;
  const uint32_t i0 = query_of(a, r0), last = query_of(a, (r0 + kRows < rows ? r0 + kRows : rows) - 1u);
  int32_t lo, hi, wlo, whi, all_lo, all_hi;
  tree_range(a, s, r0, kRows, &lo, &hi);
  tree_range(a, s, w0, 16u * R, &wlo, &whi);
  tree_common(a, s, last, &all_lo, &all_hi);
  // Rows that are not there see nothing.  Such a wavefront takes the masked loop for every token, and the others wait for it: 60 drafts
  // x 4 heads on 32768 tokens 107 us, 64 x 4 78; 15 x 4 on 16 x 8192 123, 16 x 4 86.
  if (w0 + 16u * R > rows) all_lo = all_hi = 0;
  int32_t t0 = (lo & ~15) + (int32_t)(at.split * g.chunk), t1 = t0 + (int32_t)g.chunk;
  t1 = t1 < hi ? t1 : hi;
  if (a.pages == 0) t1 = t0;
  if (t0 >= t1 && g.splits > 1) return;  // the same for the whole workgroup
  const uint32_t b = at.b;
  const uint32_t P = 1u << a.page_log2;
  const uint64_t page_size = (uint64_t)P * Page<BITS>::kToken;

  Share<BITS> sh;
  auto load = [&](int32_t t, int32_t page) __attribute__((always_inline)) {
    const uint8_t* p = a.cache + ((uint64_t)(page < 0 ? 0 : page) * a.heads + h) * page_size;
    load_keys<BITS>(p, P, (uint32_t)t & (P - 1u), lane, sh);
    load_values<BITS>(p, P, (uint32_t)t & (P - 1u), lane, sh);
  };
  // this wavefront's 16 tokens at t, as operands
  auto stage = [&](TreeStage& d, uint2* flags, int32_t t, int32_t page) __attribute__((always_inline)) {
    uint32_t word = page < 0 ? 0xFFFF0000u : 0u, large = 0;
    if (__builtin_amdgcn_ballot_w64(odd_scales<BITS>(most(sh.ks[0], sh.ks[1])))) {
      const int32_t tok = t + (int32_t)n;
      if (page < 0 || tok < lo || tok >= t1) sh.ks[0] = sh.ks[1] = 0u;  // a token that no row sees may hold anything
      word |= gone_keys(sh.ks) << 16;
      if (shrink<BITS>(sh.ks)) large |= 1u;
    }
    f16x8 kh[4], kl[4];
    key_operands<BITS, false>(sh, kh, kl);
#pragma unroll
    for (int j = 0; j < 4; ++j) d.k[wave][j][lane] = kh[j];
    if (__builtin_amdgcn_ballot_w64(odd_scales<BITS>(most(sh.vs[0], sh.vs[1])))) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int32_t tok = t + 4 * (int32_t)b4 + i;
        if (page < 0 || tok < lo || tok >= t1) drop_scales(sh.vs, 1u << i);
      }
      const uint32_t bad = bad_scales(sh.vs);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t votes = __builtin_amdgcn_ballot_w64((bad >> i) & 1u);
#pragma unroll
        for (int q = 0; q < 4; ++q) word |= (votes >> (16 * q)) & 0xFFFFu ? 1u << (4 * q + i) : 0u;
      }
      // a value vector with one NaN scale is NaN as a whole: its rows are poisoned, its scales count as 0
      drop_scales(sh.vs, (word >> (4 * b4)) & 15u);
      if (shrink<BITS>(sh.vs)) large |= 2u;
    }
    if (lane == 0) flags[wave] = make_uint2(word, large);
    uint32_t v[8][2];
    value_operands<BITS>(sh, v);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      reinterpret_cast<uint2*>(&d.v[wave >> 1][i][lane])[wave & 1u] = make_uint2(v[i][0], v[i][1]);
  };
  const int32_t mine = 16 * (int32_t)wave;
  int32_t t = t0, page = page_of(a, b, t + mine, t1);
  if (t < t1) load(t + mine, page);
  int32_t next = entry_of(a, b, t + kTok + mine, t1);

  uint32_t query[R];
  const bool climbs = a.window || t1 > s.back;  // as for few rows
  if (climbs) climb(a, g.parents, s, i0, last - i0 + 1u, s_tree);

  const bool cap = a.cap_in > 0.0f;
  f16x8 qh[R][4];
  float qf[R], eff[R], m[R], poison[R];
  int32_t row_lo[R];
  bool have[R];
  f32x4 o[R][8], ones[R];
#pragma unroll
  for (int q = 0; q < R; ++q) {
    const uint64_t row = (uint64_t)h * a.rows + (uint64_t)s.q0 * a.group + w0 + 16u * q + n;
    const bool some = w0 + 16u * q < rows;  // the last 16 may have rows of the next sequence among them: they see nothing
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      qh[q][j] = (f16x8)(_Float16)0.0f;
      if (some) qh[q][j] = *reinterpret_cast<const f16x8*>(a.qhi + row * kD + 8 * (4 * b4 + j));
    }
    qf[q] = some ? a.qf[row] : 1.0f;
    eff[q] = cap ? 1.0f : qf[q];  // scores are eff sc: the product with qf waits for the exponent's fma
    m[q] = kLowest;
    poison[q] = 0.0f;
    have[q] = w0 + 16u * q + n < rows;
    query[q] = have[q] ? query_of(a, w0 + 16u * q + n) - i0 : 0u;
    row_lo[q] = climbs ? tree_lo(a, s, s_tree.depth[query[q]]) : 0;
    ones[q] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 8; ++i) o[q][i] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  }
  // a new reference for the rows' exponentials
  auto raise = [&](const float* top) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const float mn = fmaxf(m[q], blocks_max(top[q]));
      const float f = __builtin_amdgcn_exp2f(m[q] - mn);
      m[q] = mn;
      ones[q] *= f;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[q][i] *= f;
    }
  };
  uint32_t buf = 0;
  if (t < t1) {
    stage(st[0], s_flags[0], t + mine, page);
    __syncthreads();
  }
  for (; t < t1; t += kTok) {
    const bool more = t + kTok < t1;
    if (more) {
      page = page_in(a, next);
      load(t + kTok + mine, page);
      next = entry_of(a, b, t + 2 * kTok + mine, t1);
    }
    const TreeStage& d = st[buf];
    // blocks of 16 tokens with a flag, asked for once and not between the products
    const uint2 flags = s_flags[buf][lane & (kAttWaves - 1)];
    const uint32_t flagged = (uint32_t)__builtin_amdgcn_ballot_w64(lane < (uint32_t)kAttWaves && (flags.x | flags.y) != 0u);
    bool whole = false;
    {
      if (!cap && !flagged && t >= all_lo && t + kTok <= all_hi && t + kTok <= t1) {
        // Every row sees every token: each step's scores are under way during the softmax of the one before.  Capped scores, a dozen
        // vector instructions more each, take the loop below (64 drafts on 32768 tokens 108 us, 78 without a cap; here they were not tried).
        f32x4 sc[2][R][2];
        auto products = [&](int w, f32x4 (*x)[2]) __attribute__((always_inline)) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int q = 0; q < R; ++q) x[q][u] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const f16x8 kh = d.k[2 * w + u][j][lane];
#pragma unroll
              for (int q = 0; q < R; ++q) x[q][u] = mfma(kh, qh[q][j], x[q][u]);
            }
          }
        };
        products(0, sc[0]);
#pragma unroll
        for (int w = 0; w < kTok / 32; ++w) {
          f32x4(*x)[2] = sc[w & 1];
          float top[R];
          bool rise = false;
#pragma unroll
          for (int q = 0; q < R; ++q) {
            top[q] = x[q][0][0];
#pragma unroll
            for (int i = 1; i < 8; ++i) top[q] = fmaxf(top[q], x[q][i >> 2][i & 3]);
            top[q] *= eff[q];
            rise |= top[q] > m[q] + kSlack;
          }
          if (__builtin_amdgcn_ballot_w64(rise)) raise(top);
          if (w + 1 < kTok / 32) products(w + 1, sc[(w + 1) & 1]);
          f16x8 pf[R];
#pragma unroll
          for (int q = 0; q < R; ++q) {
            const float base = kPScaleLog2 - m[q];
            U32x4 p;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int u = i >> 1, c = 2 * (i & 1);
              const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[q][u][c], eff[q], base));
              const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[q][u][c + 1], eff[q], base));
              p.v[i] = u2((f16x2){(_Float16)p0, (_Float16)p1});
            }
            pf[q] = frag(p);
            ones[q] = mfma((f16x8)(_Float16)1.0f, pf[q], ones[q]);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const f16x8 v = d.v[w][i][lane];
#pragma unroll
            for (int q = 0; q < R; ++q) o[q][i] = mfma(v, pf[q], o[q][i]);
          }
        }
        whole = true;
      }
    }
#pragma unroll 1
    for (int w = whole ? kTok / 32 : 0; w < kTok / 32; ++w) {
      const int32_t tw = t + 32 * w;
      if (tw >= whi || tw + 32 <= wlo || tw >= t1) continue;
      f32x4 sc[R][2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int q = 0; q < R; ++q) sc[q][u] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f16x8 kh = d.k[2 * w + u][j][lane];
#pragma unroll
          for (int q = 0; q < R; ++q) sc[q][u] = mfma(kh, qh[q][j], sc[q][u]);
        }
      }
      auto unshrink = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float k = s_flags[buf][2 * w + u].y & 1u ? kShrunk : 1.0f;
#pragma unroll
          for (int q = 0; q < R; ++q) sc[q][u] *= k;
        }
      };
      uint32_t large = 0;  // blocks of shrunk values
      if (cap) {
        if (flagged >> (2 * w) & 3u) unshrink();
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[q][u][i] = a.cap_out * tanh32(sc[q][u][i] * qf[q] * a.cap_in);
      }
      if ((flagged >> (2 * w) & 3u) || tw < all_lo || tw + 32 > all_hi || tw + 32 > t1) {
        const uint2 f0 = s_flags[buf][2 * w], f1 = s_flags[buf][2 * w + 1];
        large = uniform(f0.y >> 1 | (f1.y & 2u));
        if (!cap) unshrink();
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int32_t tok = tw + 16 * u + 4 * (int32_t)b4 + i;
              const uint32_t fl = (u ? f1.x : f0.x) >> (4 * b4 + i);
              const bool shown = have[q] & !(fl & 0x10000u) & (tok < t1) & tree_sees(s_tree, s.back, query[q], row_lo[q], tok);
              sc[q][u][i] = shown ? sc[q][u][i] : -__builtin_inff();
              poison[q] = shown & (fl & 1u) ? __builtin_nanf("") : poison[q];
            }
      }
      float top[R];
      bool rise = false;
#pragma unroll
      for (int q = 0; q < R; ++q) {
        top[q] = sc[q][0][0];
#pragma unroll
        for (int i = 1; i < 8; ++i) top[q] = fmaxf(top[q], sc[q][i >> 2][i & 3]);
        top[q] *= eff[q];
        rise |= top[q] > m[q] + kSlack;
      }
      // with shrunk values, P goes up to 2^15 against the maximum itself
      if (large || __builtin_amdgcn_ballot_w64(rise)) raise(top);
      f16x8 pf[R];
#pragma unroll
      for (int q = 0; q < R; ++q) {
        const float base = kPScaleLog2 - m[q];
        U32x4 p;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int u = i >> 1, c = 2 * (i & 1);
          const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[q][u][c], eff[q], base));
          const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[q][u][c + 1], eff[q], base));
          p.v[i] = u2((f16x2){(_Float16)p0, (_Float16)p1});
        }
        pf[q] = frag(p);
        // the sum of the rounded P, the one the output is weighted with, is one more product
        ones[q] = mfma((f16x8)(_Float16)1.0f, pf[q], ones[q]);
      }
      if (large) {
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
          for (int i = 0; i < 8; ++i) pf[q][i] *= (large >> (i >> 2)) & 1u ? (_Float16)kShrunk : (_Float16)1.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const f16x8 v = d.v[w][i][lane];
#pragma unroll
        for (int q = 0; q < R; ++q) o[q][i] = mfma(v, pf[q], o[q][i]);
      }
    }
    if (more) {
      if (R == 1) __syncthreads();
      else buf ^= 1u;
      stage(st[buf], s_flags[buf], t + kTok + mine, page);
    }
    __syncthreads();
  }

  // each wavefront's rows, 16 at a time, through its part of LDS: a row's values to 16 lanes
  __syncthreads();
  const uint64_t first_part = ((((uint64_t)b * g.tiles + at.tile) * a.heads + h) * g.splits + at.split) * kRows + wave * 16u * R;
  const LaneInverse inv = lane_inverse(K, n);
#pragma unroll
  for (int q = 0; q < R; ++q) {
    const float total = ones[q][0], bad = blocks_sum(poison[q]);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int i = 0; i < 8; i += 4)
        *reinterpret_cast<f32x4*>(&s_o[wave][n][8 * (4 * b4 + r) + i]) =
            (f32x4){o[q][i][r] + bad, o[q][i + 1][r] + bad, o[q][i + 2][r] + bad, o[q][i + 3][r] + bad};
    const uint64_t part = first_part + 16u * q;
    if (b4 == 0 && g.splits > 1) *reinterpret_cast<f32x2*>(g.pml + (part + n) * 2) = (f32x2){m[q], total};
    wave_sync();
#pragma unroll 1
    for (uint32_t k = 0; k < 4; ++k) {
      const uint32_t r = 4u * k + b4;
      if (w0 + 16u * q + 4u * k >= rows) break;
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = s_o[wave][r][8 * n + i];
      const float tr = row_get_any(total, r);
      if (g.splits == 1) {
        store_row<BITS>(a, K, K.v, s, h, w0 + 16u * q + r, n, inv, y, tr);
      } else {
        float* d = g.po + (part + r) * kD + 8 * n;
        *reinterpret_cast<f32x4*>(d) = (f32x4){y[0], y[1], y[2], y[3]};
        *reinterpret_cast<f32x4*>(d + 4) = (f32x4){y[4], y[5], y[6], y[7]};
      }
    }
    wave_sync();
  }
}

// Joins a row's splits, turns it back and stores it.  WIDE: one workgroup a row, its 16 groups of 16 lanes take
// the splits in turn and join in LDS; otherwise 16 lanes take a row and all its splits.
template <int BITS, bool WIDE>
__global__ __launch_bounds__(kAttBlock) void join_tree_kernel(AttendArgs a, TreeArgs g, Tables K, uint32_t tile_rows, uint32_t most_rows) {
  __shared__ float s_y[WIDE ? 16 : 1][kD + 4], s_m[16], s_l[16];
  const uint32_t l = threadIdx.x & 15u, k = threadIdx.x >> 4;
  const uint32_t index = WIDE ? blockIdx.x : blockIdx.x * 16u + k;
  // rows of a (sequence, head) in order; none of a wavefront's or all of its four are in a tile of the sequence
  const uint32_t r = index % most_rows, h = index / most_rows % a.heads, b = index / most_rows / a.heads;
  if (b >= a.seqs) return;
  const Seq s = seq_of(a, b);
  if ((r & ~3u) >= (uint32_t)s.m * a.group) return;
  const uint32_t tile = r / tile_rows, r0 = tile * tile_rows;
  int32_t lo, hi;
  tree_range(a, s, r0, tile_rows, &lo, &hi);
  if (a.pages == 0) hi = lo;
  const uint32_t s1 = hi > lo ? ((uint32_t)(hi - (lo & ~15)) + g.chunk - 1u) / g.chunk : 0u;
  const uint64_t first = (((uint64_t)b * g.tiles + tile) * a.heads + h) * g.splits;
  float m = kLowest, sum = 0.0f, y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = 0.0f;
  for (uint32_t i = WIDE ? k : 0u; i < s1; i += WIDE ? 16u : 1u) {
    const uint64_t p = (first + i) * tile_rows + r - r0;
    const f32x2 ml = *reinterpret_cast<const f32x2*>(g.pml + p * 2);
    const f32x4 u0 = *reinterpret_cast<const f32x4*>(g.po + p * kD + 8 * l), u1 = *reinterpret_cast<const f32x4*>(g.po + p * kD + 8 * l + 4);
    const float mn = fmaxf(m, ml[0]), f0 = __builtin_amdgcn_exp2f(m - mn), f1 = __builtin_amdgcn_exp2f(ml[0] - mn);
    m = mn;
    sum = sum * f0 + ml[1] * f1;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      y[c] = y[c] * f0 + u0[c] * f1;
      y[4 + c] = y[4 + c] * f0 + u1[c] * f1;
    }
  }
  if (WIDE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) s_y[WIDE ? k : 0][8 * l + i] = y[i];
    if (l == 0) {
      s_m[k] = m;
      s_l[k] = sum;
    }
    __syncthreads();
    if (k) return;
    m = s_m[0];
    for (int i = 1; i < 16; ++i) m = fmaxf(m, s_m[i]);
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = 0.0f;
    for (int i = 0; i < 16; ++i) {
      const float f = __builtin_amdgcn_exp2f(s_m[i] - m);
      sum += s_l[i] * f;
#pragma unroll
      for (int c = 0; c < 8; ++c) y[c] += s_y[WIDE ? i : 0][8 * l + c] * f;
    }
  }
  store_row<BITS>(a, K, K.v, s, h, r, l, lane_inverse(K, l), y, sum);
}

}  // namespace hq_kv

using namespace hq_kv;

namespace {

bool is_tree(const hq_kv_attend_args* g) { return g && g->causal && !g->weights && g->max_q <= (uint32_t)kMaxTree; }

struct TreePlan {
  uint32_t max_q, rows, all, tile_rows, tiles, splits, chunk;
  uint64_t grid, joins, pml, po, qf, qhi, bytes;
};

// HQ_OK, or an error for a call that the launches cannot take.
int plan_tree(const hq_kv_cache& c, const hq_kv_attend_args& g, TreePlan* out) {
  TreePlan p;
  const uint64_t each = g.q_start || g.seqs == 0 ? g.total_q : g.total_q / g.seqs;
  p.max_q = (uint32_t)(each < g.max_q ? each : g.max_q);
  const uint64_t rows = (uint64_t)p.max_q * (g.q_heads / c.heads), sh = (uint64_t)g.seqs * c.heads, all = g.total_q * (g.q_heads / c.heads);
  if (all > 0x7FFFFF00ull || all * c.heads > kMaxThreads / 16 || rows > 0x7FFFFF00ull / 128u) return HQ_ERR_INVALID_ARG;
  p.rows = (uint32_t)rows;
  p.all = (uint32_t)all;
  const uint64_t seen = (uint64_t)g.window + p.max_q + 15, span = g.window && seen < g.max_len ? seen : g.max_len;
  // Operands in registers, 32 rows a tile, up to 2^24 rows x tokens: LDS starts later and takes a launch for the rows.  us in
  // registers and in LDS, 4 query heads a KV head, 4 bits unless said:
  //   64 drafts, 8 heads, on 4096 tokens 32 and 40, on 8192 (2^24) 40 and 42, on 16384 57 and 51, on 32768 92 and 73; at 8 bits 33 and
  //   41, 40 and 43, 57 and 52, 90 and 73; one head, on 32768 29 and 38, 65536 (2^24) 40 and 43, 131072 58 and 53
  //   16 drafts of 16 sequences, 8 heads, on 1024 28 and 32, 2048 (2^24) 37 and 39, 4096 54 and 53, 8192 89 and 86; at 8 bits 28 and 35,
  //   38 and 42, 54 and 57
  //   16 drafts of 64 sequences on 256 34 and 33, 512 (2^24) 43 and 40, 1024 60 and 60, 2048 93 and 94
  //   100 drafts of 16 sequences, 2 heads, on 1024 49 and 61, 2048 (2^24.6) 65 and 67, 4096 101 and 104
  // It is off where rows are many and tokens few (64 drafts of 64 sequences, 8 heads, on 128 tokens (2^24) 113 and 80), and where 64-row
  // tiles are half empty (9 drafts, 36 rows, of 64 sequences on 2048 93 and 114).
  p.tile_rows = rows <= 16 ? 16 : rows <= 32 || sh * rows * span <= 1ull << 24 ? 32 : rows <= 64 ? 64 : 128;
  p.tiles = rows ? (uint32_t)((rows + p.tile_rows - 1u) / p.tile_rows) : 1u;
  // Workgroups: about three rounds of up to 16 rows, as in hq_attend.hip; of more rows, whose starts cost more, as many as the chip
  // holds at once, and half as many again where four fit a CU (16 drafts on 16 x 8192 ragged tokens, 64 rows: 68 us at 1536, 79 at
  // 1024, 81 at 2048; 64 on 32768, 128 rows a tile: 73 at 512, 84 at 768; 13 on 64 x 2001, 32 rows: 43 at 512, 54 at 768).
  // Splits count from the first token that a tile sees, at most one for each 512 tokens begun; in whole 128 tokens, of 384 or more where
  // there are several.
  // Rows are counted by max_q: 16 sequences of 16 drafts on 8192 tokens take 96 us with 16 and 364 with 256 (tiles for rows that no
  // sequence has, and no splits), one of 64 drafts among 15 of 4 342 with 64.
  const uint64_t items = sh * p.tiles, target = p.tile_rows == 16 ? 2048 : p.tile_rows == 64 ? 1536 : 512;
  uint64_t splits = items ? (target + items - 1) / items : 1;
  const uint64_t most = (span + 511) / 512;
  if (splits > most) splits = most;
  if (splits < 1) splits = 1;
  p.chunk = (uint32_t)(((span + splits - 1) / splits + 127) / 128 * 128);
  if (p.chunk == 0) p.chunk = 128;
  p.splits = (uint32_t)((span + p.chunk - 1) / p.chunk);
  if (p.splits == 0) p.splits = 1;
  p.grid = (sh * p.splits + 7) / 8 * 8 * p.tiles;
  p.joins = sh * ((rows + 15) / 16 * 16);
  if (p.grid > kMaxThreads / kAttBlock || p.joins > kMaxThreads / 16) return HQ_ERR_INVALID_ARG;
  uint64_t at = 0;
  auto take = [&](uint64_t n) {
    const uint64_t here = at;
    at = (at + n + 255) / 256 * 256;
    return here;
  };
  // 16 rows are read together from any row on
  const uint64_t parts = p.splits > 1 ? items * p.splits * p.tile_rows : 0, held = p.tile_rows > 32 ? all * c.heads + 16 : 0;
  p.pml = take(parts * 8);
  p.po = take(parts * kD * 4);
  p.qf = take(held * 4);
  p.qhi = take(held * kD * 2);
  p.bytes = at;
  *out = p;
  return HQ_OK;
}

template <int BITS, int R>
hipError_t launch_tree_many(const AttendArgs& a, const TreeArgs& g, const Tables& T, const TreePlan& p, hipStream_t st) {
  // dynamic LDS, which may be more than the default limit: asked for once per kernel (the attribute holds for every device)
  static const hipError_t set = hipFuncSetAttribute(reinterpret_cast<const void*>(&attend_tree_many_kernel<BITS, R>),
                                                    hipFuncAttributeMaxDynamicSharedMemorySize, (int)(tree_lds<R>()));
  if (set != hipSuccess) return set;
  hipLaunchKernelGGL((rotate_tree_kernel<BITS>), dim3((a.rows + 15u) / 16u * a.heads), dim3(kAttBlock), 0, st, a, T);
  hipLaunchKernelGGL((attend_tree_many_kernel<BITS, R>), dim3((uint32_t)p.grid), dim3(kAttBlock), tree_lds<R>(), st, a, g, T);
  return hipSuccess;
}

template <int BITS>
hipError_t launch_tree(const AttendArgs& a, const TreeArgs& g, const Tables& T, const TreePlan& p, hipStream_t st) {
  const dim3 grid((uint32_t)p.grid), block(kAttBlock);
  hipError_t e = hipSuccess;
  if (p.tile_rows == 16) hipLaunchKernelGGL((attend_tree_kernel<BITS, 1>), grid, block, 0, st, a, g, T);
  else if (p.tile_rows == 32) hipLaunchKernelGGL((attend_tree_kernel<BITS, 2>), grid, block, 0, st, a, g, T);
  else if (p.tile_rows == 64) e = launch_tree_many<BITS, 1>(a, g, T, p, st);
  else e = launch_tree_many<BITS, 2>(a, g, T, p, st);
  if (e != hipSuccess) return e;
  if (p.splits > 1) {
    // A workgroup a row while those are at most 16 a CU, 16 lanes a row beyond, as in hq_attend.hip.
    const uint32_t each = (p.rows + 15u) / 16u * 16u;
    if (p.joins <= 4096) hipLaunchKernelGGL((join_tree_kernel<BITS, true>), dim3((uint32_t)p.joins), block, 0, st, a, g, T, p.tile_rows, each);
    else hipLaunchKernelGGL((join_tree_kernel<BITS, false>), dim3((uint32_t)(p.joins / 16)), block, 0, st, a, g, T, p.tile_rows, each);
  }
  return hipGetLastError();
}

}  // namespace

extern "C" {

int hq_kv_attend_tree_workspace_size(const hq_kv_cache* cache, const hq_kv_attend_args* args, size_t* bytes) {
  if (!bytes || !is_tree(args)) return HQ_ERR_INVALID_ARG;
  if (int rc = check_attend(cache, args)) return rc;
  TreePlan p;
  if (int rc = plan_tree(*cache, *args, &p)) return rc;
  *bytes = p.bytes;
  return HQ_OK;
}

int hq_kv_attend_tree(const hq_kv_cache* cache, const hq_kv_attend_args* args, const int32_t* parents, void* workspace,
                      size_t workspace_bytes, hq_stream_t stream) {
  if (!is_tree(args)) return HQ_ERR_INVALID_ARG;
  if (int rc = check_attend(cache, args)) return rc;
  AttendArgs a = {};
  Tables T;
  bool nothing;
  if (int rc = attend_args(*cache, *args, &a, &T, &nothing)) return rc;
  if (nothing) return HQ_OK;
  if (!parents || ((uintptr_t)parents & 3u)) return HQ_ERR_INVALID_ARG;
  TreePlan p;
  if (int rc = plan_tree(*cache, *args, &p)) return rc;
  if (p.bytes && (!workspace || ((uintptr_t)workspace & 255u) || workspace_bytes < p.bytes)) return HQ_ERR_INVALID_ARG;
  a.max_q = p.max_q;
  a.rows = p.all;
  char* w = static_cast<char*>(workspace);
  a.qf = reinterpret_cast<float*>(w + p.qf);
  a.qhi = reinterpret_cast<_Float16*>(w + p.qhi);
  TreeArgs g;
  g.parents = parents;
  g.tiles = p.tiles;
  g.splits = p.splits;
  g.chunk = p.chunk;
  g.pml = reinterpret_cast<float*>(w + p.pml);
  g.po = reinterpret_cast<float*>(w + p.po);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const hipError_t e = cache->bits == 4 ? launch_tree<4>(a, g, T, p, st) : launch_tree<8>(a, g, T, p, st);
  return e == hipSuccess ? HQ_OK : HQ_ERR_HIP;
}

}  // extern "C"
