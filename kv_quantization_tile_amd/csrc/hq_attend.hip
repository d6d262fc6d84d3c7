// hq_attend.hip -- softmax attention over the paged SRFT cache, on the codes themselves.
//
// A cached vector is x^ = T^t y, y_c = code_c Delta_{c/8} lambda_c, with T = pack(F diag(s) .)
// orthogonal ("When quantization is free" technical summary, gist.science/ko/paper/2605.05699, section
// "Methodology").  So q . k^ = (lambda (T q)) . (code Delta), and sum_t p_t v^_t = T^t (lambda sum_t p_t
// code Delta): the query is transformed once, the output transformed back once, and no key or value
// is.  Per token and head that reads 192 bytes (4 bits; 320 at 8) instead of bf16's 512.
//
// Tiles: a row is one (query, head of the KV head's group); 16 rows are a tile.  S^t = K Q^t on
// v_mfma_f32_16x16x32_f16 leaves lane (n, b) (n = lane mod 16, b = lane / 16) the scores of row n for
// tokens 4b..4b+3 of 16; two such blocks are, register for register, the operand P^t of O^t = V^t P^t
// over 32 tokens, with V's blocks of four tokens laid out to match, so nothing crosses lanes between
// the two products.  Lane (n, b) of O^t holds row n, groups 4b..4b+3.
//
// Codes become binary16 in two steps: or-ing a code's offset bits into the mantissa of 1024.0 gives
// 1024 + c + 8 (c + 128) exactly, subtracting 1032 (1152) gives c, and the product with Delta is rounded once
// to binary16.  Delta and so c Delta are whole multiples of 2^-24, binary16's smallest step: the rounding is
// at most 2^-11 of the value however small the vector.  A step with a scale so large that c Delta would overflow
// takes its scales times 2^-7 (shrink) and undoes that in the scores and in P.
// Rows of Q are scaled by a power of two so that their largest coordinate lies in [2^14, 2^15).
// With accumulated weights asked for, scores are needed to binary32: Q and the keys go in two parts
// (hi = rounded product, lo = fma(code, Delta, -hi), exact), three products instead of one.
// Scores, maxima, sums and outputs are binary32; P is binary16, scaled by 2^8 against a running
// reference at most 2^6 below the maximum (so P <= 2^14, and terms down to 2^-22 of it stay normal).
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/hq.h"
#include "hq_attend_device.h"

namespace hq_kv {

// Where row r of a sequence lies among its head's, in [heads][rows].
__device__ __forceinline__ uint64_t row_at(const AttendArgs& a, const Seq& s, uint32_t h, uint32_t r) {
  return (uint64_t)h * a.rows + (uint64_t)s.q0 * a.group + r;
}
// The last tile of a sequence: its first row.
__device__ __forceinline__ uint32_t last_tile(const AttendArgs& a, const Seq& s) {
  const uint32_t rows = (uint32_t)s.m * a.group;
  return rows ? (rows - 1u) & ~(a.tile_rows - 1u) : 0u;  // a power of two
}

// The sequence of full tile f: the last whose tiles begin at or before it.  A wavefront looks at 64 places at a time.
__device__ __forceinline__ uint32_t seq_with(const AttendArgs& a, uint32_t f) {
  uint32_t b = 0, count = a.seqs;
  while (count > 1u) {
    const uint32_t step = (count + 63u) / 64u, i = (threadIdx.x & 63u) * step;
    const bool here = i < count && a.first[b + i] <= f;
    const uint32_t skip = ((uint32_t)__builtin_popcountll(__builtin_amdgcn_ballot_w64(here)) - 1u) * step;
    b += skip;
    count = count - skip < step ? count - skip : step;
  }
  return b;
}

// ---------------------------------------------------------------------------------------------
// Light tiles, of up to 16 rows: the single-token step, and the single tokens and last rows of a batch that has longer
// chunks too (with the full tiles they take as long as 256 rows: 181 us for 4 x 129 and 4 x 1 queries, against 107 there and
// 28 here).  A workgroup takes one split of the tokens; its four wavefronts take 32 tokens in
// turn, the next 32 already on their way, and join at the end.  The rows are a fraction of the products' 16
// columns, which costs nothing here.  The cache's bytes bound it where there are many: 16 sequences of up to
// 32768 tokens, 535 MB, in 148 us with the join (3.6 TB/s; a sum over 1 GiB reads 3.9, a 2 GiB copy moves 4.9); an extra
// wavefront a SIMD (128 registers, some spilled) took 160 us.  Scales out of the ordinary are looked for where the codes
// beside them are first used: one look at a step's scales waits for its last load (151 us).  One sequence of 301 tokens
// takes 10.5 us: about 2 until the codes are asked for, 1.5 for the rows, 4.2 for three turns, 1 for the join.
template <int BITS, bool PREC>
__global__ __launch_bounds__(kAttBlock, BITS == 4 ? 3 : 2) void attend_few_kernel(AttendArgs a, Tables K) {
  __shared__ __align__(16) float s_o[kAttWaves][16][kPad];
  __shared__ __align__(16) _Float16 s_q[PREC ? 2 : 1][16][kD + 8];
  __shared__ float s_f[16], s_m[kAttWaves][16], s_l[kAttWaves][16], s_lam[2][kD];
  const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 15u, b4 = lane >> 4;
  const uint32_t split = blockIdx.x % a.lsplits, item = blockIdx.x / a.lsplits, h = item % a.heads, b = item / a.heads;
  const Seq s = seq_of(a, b);
  const uint32_t r0 = last_tile(a, s), rows = (uint32_t)s.m * a.group - r0;  // of this tile
  if (rows == 0 || rows > 16u) return;
  int32_t lo, hi;
  rows_range(a, s, r0, 16, &lo, &hi);
  int32_t t0 = (int32_t)(split * a.lchunk), t1 = t0 + (int32_t)a.lchunk;
  t0 = t0 > (lo & ~15) ? t0 : lo & ~15;
  t1 = t1 < hi ? t1 : hi;
  if (a.pages == 0) t1 = t0;
  if (t0 >= t1 && a.lsplits > 1) return;  // the same for the whole workgroup
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
  {  // the rows: four to a wavefront, 16 lanes each
    const uint32_t r = threadIdx.x >> 4;
    float f = 0.0f;
    if ((r & ~3u) < rows) f = rotate_row<BITS>(a, K, s_lam[0], h, (uint32_t)s.q0 * a.group + r0 + r, r < rows, n, lane_forward(K, n), s_q[0][r], PREC ? s_q[PREC ? 1 : 0][r] : nullptr);
    else
      for (int i = 0; i < 8; ++i) {
        s_q[0][r][8 * n + i] = (_Float16)0.0f;
        if (PREC) s_q[PREC ? 1 : 0][r][8 * n + i] = (_Float16)0.0f;
      }
    if (n == 0) s_f[r] = f;
  }
  __syncthreads();
  f16x8 qh[4], ql[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    qh[j] = *reinterpret_cast<const f16x8*>(&s_q[0][n][8 * (4 * b4 + j)]);
    if (PREC) ql[j] = *reinterpret_cast<const f16x8*>(&s_q[PREC ? 1 : 0][n][8 * (4 * b4 + j)]);
  }
  const float qf = s_f[n];
  int32_t row_lo = 0, row_hi = 0, all_lo = hi, all_hi = lo;
  if (n < rows) visible(a, s, (int32_t)query_of(a, r0 + n), &row_lo, &row_hi);
  // the tokens every existing row sees need no mask (rows past the last are products with zero)
  if (rows) rows_common(a, s, r0, rows, &all_lo, &all_hi);

  float m = kLowest, sum = 0.0f, poison = 0.0f;
  f32x4 o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
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
    float sc[8];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (__builtin_amdgcn_ballot_w64(odd_scales<BITS>(most(cur[u].ks[0], cur[u].ks[1])))) {
        const int32_t tok = t + 16 * u + (int32_t)n;
        if (!there[u] || tok < lo || tok >= t1) cur[u].ks[0] = cur[u].ks[1] = 0u;  // a token that no row sees may hold anything
        gone |= gone_keys(cur[u].ks) << (16 * u);
        if (shrink<BITS>(cur[u].ks)) large |= 1u << u;
      }
      f16x8 kh[4], kl[4];
      key_operands<BITS, PREC>(cur[u], kh, kl);
      const f32x4 r = scores16<PREC>(kh, kl, qh, ql);
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[4 * u + i] = r[i] * qf;
    }
    if (large & 3u) {
#pragma unroll
      for (int i = 0; i < 8; ++i) sc[i] *= (large >> (i >> 2)) & 1u ? kShrunk : 1.0f;
    }
    cap_scores<8>(a, sc);
    if (gone) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if ((gone >> (4u * b4) >> (16 * (i >> 2) + (i & 3))) & 1u) sc[i] = -__builtin_inff();
    }
    if (!(there[0] && there[1] && t >= all_lo && t + 32 <= all_hi && t + 32 <= t1)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int32_t tok = t + 16 * (i >> 2) + 4 * (int32_t)b4 + (i & 3);
        if (!there[i >> 2] || tok < row_lo || tok >= row_hi || tok >= t1) sc[i] = -__builtin_inff();
      }
    }
    if (a.scores && n < rows) {
      float* d = a.scores + ((uint64_t)item * a.wrows + n) * a.wpad + (uint32_t)t + 4u * b4;
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (t + 16 * u < t1) *reinterpret_cast<f32x4*>(d + 16 * u) = (f32x4){sc[4 * u], sc[4 * u + 1], sc[4 * u + 2], sc[4 * u + 3]};
    }
    // A value vector with NaN scales makes the rows that see it NaN and no other (0 NaN in the product
    // would reach every row): its scales count as 0, and the rows are poisoned.
    if (__builtin_amdgcn_ballot_w64(odd_scales<BITS>(__builtin_elementwise_max(most(cur[0].vs[0], cur[0].vs[1]), most(cur[1].vs[0], cur[1].vs[1]))))) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t bad = bad_scales(cur[u].vs);
        uint32_t drop = bad;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int32_t tok = t + 16 * u + 4 * (int32_t)b4 + i;
          if (!there[u] || tok < lo || tok >= t1) drop |= 1u << i;  // as with the keys
          if ((bad >> i) & 1u && sc[4 * u + i] != -__builtin_inff()) poison = __builtin_nanf("");
        }
        drop_scales(cur[u].vs, drop);
        if (shrink<BITS>(cur[u].vs)) large |= 4u << u;
      }
    }
    float top = sc[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = fmaxf(top, sc[i]);
    // with shrunk values, P goes up to 2^15 against the maximum itself
    if (large >= 4u || __builtin_amdgcn_ballot_w64(top > m + kSlack)) {
      const float mn = fmaxf(m, blocks_max(top));
      const float f = __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      sum *= f;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] *= f;
    }
    const float base = m - kPScaleLog2;
    U32x4 pf;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p0 = __builtin_amdgcn_exp2f(sc[2 * i] - base), p1 = __builtin_amdgcn_exp2f(sc[2 * i + 1] - base);
      sum += p0 + p1;
      pf.v[i] = u2((f16x2){(_Float16)p0, (_Float16)p1});
    }
    if (large >= 4u) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if ((large >> (2 + (i >> 1))) & 1u) pf.v[i] = u2(h2(pf.v[i]) * (f16x2){(_Float16)kShrunk, (_Float16)kShrunk});
    }
    uint32_t v0[8][2], v1[8][2];
    value_operands<BITS>(cur[0], v0);
    value_operands<BITS>(cur[1], v1);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const U32x4 v = {{v0[i][0], v0[i][1], v1[i][0], v1[i][1]}};
      o[i] = mfma(frag(v), frag(pf), o[i]);
    }
    cur[0] = nxt[0];
    cur[1] = nxt[1];
  }

  // the wavefronts' parts, joined in order
  sum = blocks_sum(sum);
  poison = blocks_sum(poison);
  if (b4 == 0) {
    s_m[wave][n] = m;
    s_l[wave][n] = sum;
  }
  __syncthreads();
  float mm = s_m[0][n];
#pragma unroll
  for (int w = 1; w < kAttWaves; ++w) mm = fmaxf(mm, s_m[w][n]);
  const float f = __builtin_amdgcn_exp2f(m - mm);
  if (n < rows) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int i = 0; i < 8; i += 4)
        *reinterpret_cast<f32x4*>(&s_o[wave][n][8 * (4 * b4 + r) + i]) =
            (f32x4){o[i][r] * f + poison, o[i + 1][r] * f + poison, o[i + 2][r] * f + poison, o[i + 3][r] * f + poison};
  }
  __syncthreads();
  const uint32_t r = threadIdx.x >> 4;
  if (r >= rows) return;
  float total = 0.0f, mr = s_m[0][r], y[8];
#pragma unroll
  for (int w = 1; w < kAttWaves; ++w) mr = fmaxf(mr, s_m[w][r]);
#pragma unroll
  for (int w = 0; w < kAttWaves; ++w) total += s_l[w][r] * __builtin_amdgcn_exp2f(s_m[w][r] - mr);
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = s_o[0][r][8 * n + i];
#pragma unroll
  for (int w = 1; w < kAttWaves; ++w)
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] += s_o[w][r][8 * n + i];
  if (a.lsplits == 1) {
    if (n == 0) a.lse[row_at(a, s, h, r0 + r)] = mr + __builtin_amdgcn_logf(total) - kPScaleLog2;
    store_row<BITS>(a, K, s_lam[1], s, h, r0 + r, n, lane_inverse(K, n), y, total);
    return;
  }
  const uint64_t p = ((uint64_t)item * a.lsplits + split) * 16u + r;
  *reinterpret_cast<f32x4*>(a.lpo + p * kD + 8 * n) = (f32x4){y[0], y[1], y[2], y[3]};
  *reinterpret_cast<f32x4*>(a.lpo + p * kD + 8 * n + 4) = (f32x4){y[4], y[5], y[6], y[7]};
  if (n == 0) *reinterpret_cast<f32x2*>(a.lpml + p * 2) = (f32x2){mr, total};
}

// Joins a row's splits, turns it back and stores it.  WIDE: one workgroup a row, its 16 groups of 16 lanes take
// the splits in turn and join in LDS; otherwise 16 lanes take a row and all its splits.  LIGHT: the rows of light tiles,
// else of full ones.
template <int BITS, bool WIDE, bool LIGHT>
__global__ __launch_bounds__(kAttBlock) void combine_kernel(AttendArgs a, Tables K, uint32_t rows_per_tile, uint32_t all_rows) {
  __shared__ float s_y[WIDE ? 16 : 1][kD + 4], s_m[16], s_l[16];
  const uint32_t l = threadIdx.x & 15u, g = threadIdx.x >> 4;
  const uint32_t index = WIDE ? blockIdx.x : blockIdx.x * 16u + g;
  const uint32_t tile_rows = LIGHT ? 16u : a.tile_rows, splits = LIGHT ? a.lsplits : a.plan[1], chunk = LIGHT ? a.lchunk : a.plan[2];
  const float *po = LIGHT ? a.lpo : a.po, *pml = LIGHT ? a.lpml : a.pml;
  if (index >= all_rows) return;  // no part of a workgroup unless WIDE or LIGHT: tiles have 16 rows or a multiple
  const uint32_t item = index / rows_per_tile, row = index % rows_per_tile, h = item % a.heads;
  uint32_t b = item / a.heads, r0;
  if (!LIGHT) {
    if (splits == 1 || item >= a.plan[0] * a.heads) return;
    const uint32_t f = b;
    b = seq_with(a, f);
    r0 = (f - a.first[b]) * tile_rows;
  }
  const Seq s = seq_of(a, b);
  if (LIGHT) r0 = last_tile(a, s);
  const uint32_t r = r0 + row, rows = (uint32_t)s.m * a.group;
  if (r >= rows || (LIGHT && rows - r0 > 16u)) return;
  int32_t lo, hi;
  rows_range(a, s, r0, tile_rows, &lo, &hi);
  if (a.pages == 0) hi = lo;
  const uint32_t s0 = hi > lo ? (uint32_t)lo / chunk : 0u, s1 = hi > lo ? ((uint32_t)hi + chunk - 1u) / chunk : 0u;
  float m = kLowest, sum = 0.0f, y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = 0.0f;
  for (uint32_t i = s0 + (WIDE ? g : 0u); i < s1; i += WIDE ? 16u : 1u) {
    const uint64_t p = ((uint64_t)item * splits + i) * tile_rows + row;
    const f32x2 ml = *reinterpret_cast<const f32x2*>(pml + p * 2);
    const f32x4 u0 = *reinterpret_cast<const f32x4*>(po + p * kD + 8 * l), u1 = *reinterpret_cast<const f32x4*>(po + p * kD + 8 * l + 4);
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
    for (int i = 0; i < 8; ++i) s_y[WIDE ? g : 0][8 * l + i] = y[i];
    if (l == 0) {
      s_m[g] = m;
      s_l[g] = sum;
    }
    __syncthreads();
    if (g) return;
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
  if (l == 0) a.lse[row_at(a, s, h, r)] = m + __builtin_amdgcn_logf(sum) - kPScaleLog2;
  store_row<BITS>(a, K, K.v, s, h, r, l, lane_inverse(K, l), y, sum);
}

// Accumulated weights of up to 16 rows, from the stored scores: a thread owns a token.
__global__ __launch_bounds__(kAttBlock) void weights_few_kernel(AttendArgs a, uint32_t blocks) {
  const uint32_t bh = blockIdx.x / blocks, b = bh / a.heads;
  const Seq s = seq_of(a, b);
  const uint32_t rows = (uint32_t)s.m * a.group;
  const int32_t t = (int32_t)((blockIdx.x % blocks) * kAttBlock + threadIdx.x);
  int32_t lo, hi;
  rows_range(a, s, 0, 16, &lo, &hi);
  if (a.pages == 0 || t < (lo & ~15) || t >= hi) return;
  float w = 0.0f;
  for (uint32_t r = 0; r < rows; ++r) {
    const float sc = a.scores[((uint64_t)bh * a.wrows + r) * a.wpad + (uint32_t)t];
    if (sc != -__builtin_inff()) w += __builtin_amdgcn_exp2f(sc - a.lse[row_at(a, s, bh % a.heads, r)]);
  }
  a.weights[(uint64_t)bh * a.wstride + (uint32_t)t] += w;
}

// ---------------------------------------------------------------------------------------------
// Many rows: which tiles there are, by one workgroup.  A sequence's tiles of tile_rows rows are full but for a light last
// one; `first` counts them sequence after sequence, and the splits are what leaves `parts` of them in all.
__device__ void plan_tiles(const AttendArgs& a) {
  __shared__ uint32_t s_tiles[kAttWaves], s_seqs[kAttWaves];
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  uint32_t total = 0, some = 0;
  for (uint32_t b0 = 0; b0 < a.seqs; b0 += kAttBlock) {
    const uint32_t b = b0 + threadIdx.x;
    uint32_t count = 0;
    if (b < a.seqs) {
      const uint32_t rows = (uint32_t)seq_of(a, b).m * a.group;
      count = rows / a.tile_rows + (rows % a.tile_rows > (a.light ? 16u : 0u) ? 1u : 0u);
    }
    uint32_t sum = count;  // of this lane and those before it
#pragma unroll
    for (uint32_t d = 1; d < 64; d <<= 1) {
      const uint32_t down = (uint32_t)__builtin_amdgcn_ds_bpermute((int)(((lane - d) & 63u) << 2), (int)sum);
      if (lane >= d) sum += down;
    }
    if (lane == 63) s_tiles[wave] = sum;
    const uint64_t votes = __builtin_amdgcn_ballot_w64(count > 0);
    if (lane == 0) s_seqs[wave] = (uint32_t)__builtin_popcountll(votes);
    __syncthreads();
    uint32_t before = total, all = 0;
#pragma unroll
    for (uint32_t i = 0; i < kAttWaves; ++i) {
      before += i < wave ? s_tiles[i] : 0u;
      all += s_tiles[i];
      some += s_seqs[i];
    }
    // no more than there is room for, whatever the offsets say
    before += sum - count;
    if (b < a.seqs) a.first[b] = before < a.bound ? before : a.bound;
    total = total + all < a.bound ? total + all : a.bound;
    __syncthreads();
  }
  if (threadIdx.x) return;
  a.first[a.seqs] = total;
  uint32_t splits = total ? a.parts / (total * a.heads) : 1u;
  splits = splits < a.most ? splits : a.most;
  if (splits < 1u) splits = 1u;
  uint32_t chunk = ((a.max_len + splits - 1u) / splits + 127u) / 128u * 128u;
  if (chunk == 0) chunk = 128u;
  splits = (a.max_len + chunk - 1u) / chunk;
  a.plan[0] = total;
  a.plan[1] = splits ? splits : 1u;
  a.plan[2] = chunk;
  a.plan[3] = some;
}

// Many rows: the queries' rows transformed once, to the workspace; the first workgroup counts the tiles.  A workgroup
// takes `span` rows of a head, 16 at a time: 64 where that leaves four workgroups a CU, so that the twiddles are fetched
// once for four (262144 rows: 45 us, 53 us with 16; 16640 rows: 12 us with 64, 11 us with 16).
template <int BITS>
__global__ __launch_bounds__(kAttBlock) void rotate_rows_kernel(AttendArgs a, Tables K, int parts, uint32_t span) {
  __shared__ __align__(16) _Float16 s_q[2][16][kD + 8];
  __shared__ float s_lam[2][kD];
  if (blockIdx.x == 0) {
    plan_tiles(a);
    return;
  }
  stage_tables(K, s_lam);
  const uint32_t l = threadIdx.x & 15u, g = threadIdx.x >> 4, per = (a.rows + span - 1u) / span;
  const uint32_t h = (blockIdx.x - 1u) / per, begin = (blockIdx.x - 1u) % per * span;
  const LaneForward forward = lane_forward(K, l);
#pragma unroll 1
  for (uint32_t k = begin; k < begin + span && k < a.rows; k += 16u) {
    const uint32_t row = k + g;
    const float f = rotate_row<BITS>(a, K, s_lam[0], h, row, row < a.rows, l, forward, s_q[0][g], parts == 2 ? s_q[1][g] : nullptr);
    const uint64_t at = (uint64_t)h * a.rows + row;
    // a row is written and read by the same wavefront
    wave_sync();
    if (row < a.rows) {
      if (l == 0) a.qf[at] = f;
      *reinterpret_cast<f16x8*>(a.qhi + at * kD + 8 * l) = *reinterpret_cast<const f16x8*>(&s_q[0][g][8 * l]);
      if (parts == 2) *reinterpret_cast<f16x8*>(a.qlo + at * kD + 8 * l) = *reinterpret_cast<const f16x8*>(&s_q[1][g][8 * l]);
    }
    wave_sync();
  }
}

// Many rows: a workgroup of 8 wavefronts takes 128 R rows of a (sequence, head) and one split of the tokens;
// each wavefront owns 16 R rows.  128 tokens at a time are made operands once, 16 by each wavefront, into
// LDS in the order the products read them (lane after lane, 16 bytes each: no bank conflict); the next
// ones' codes are in flight meanwhile.  Two wavefronts a SIMD, so that one's softmax runs beside the
// other's products; R = 2 is what 256 registers hold (at R = 4 and one wavefront a SIMD nothing overlapped:
// 1.2 ms for a prompt of 8192 tokens).  Two stages of LDS, one with the keys in two parts (160 KB hold no more).
// A prompt of 8192 tokens, 550 GFLOP, takes 635 to 740 us (740 to 865 TFLOP/s, less the longer the card
// has been at it; a 16-bit product of 8192^3 reaches 1050 to 1100).
// A turn of 128 tokens was 12800 cycles: 4350 of matrix instructions, about 6800 of vector instructions and 4100
// of LDS a SIMD, in phases that the two wavefronts share (scores 700, softmax 700, output 750, four times; 1750
// for the operands, 1000 for the loads).  Where every row sees every token of a turn, a step's scores are now under
// way during the softmax of the one before (732 us to 689 for the call, in turn).  Priorities, an offset between the wavefronts,
// operands fetched from LDS ahead, those of the next turn made between the products, and R = 1 with four wavefronts
// a SIMD changed the rest by 3 % at most.
constexpr int kManyWaves = 8, kManyBlock = 64 * kManyWaves;
template <bool PREC>
struct Stage {
  f16x8 k[PREC ? 2 : 1][8][4][64];  // [part][16 tokens][step][lane]
  f16x8 v[4][8][64];                // [32 tokens][coordinate][lane]
};
template <bool PREC>
constexpr size_t many_lds() { return sizeof(Stage<PREC>) * (PREC ? 1 : 2); }

template <int BITS, bool PREC, int R>
__global__ __launch_bounds__(kManyBlock, 2) void attend_many_kernel(AttendArgs a, Tables K) {
  constexpr int32_t kTok = 16 * kManyWaves;
  extern __shared__ __align__(16) uint8_t raw[];
  Stage<PREC>* st = reinterpret_cast<Stage<PREC>*>(raw);
  float(*s_o)[16][kPad] = reinterpret_cast<float(*)[16][kPad]>(raw);  // [wavefront], after the last product
  // bits 0..15: tokens with NaN value scales, 16..31: tokens that take no part; bits 0 and 1: shrunk keys, values
  __shared__ uint2 s_flags[PREC ? 1 : 2][kManyWaves];
  const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 15u, b4 = lane >> 4;
  const uint32_t tiles = uniform(a.plan[0]), splits = uniform(a.plan[1]), chunk = uniform(a.plan[2]), items = tiles * a.heads;
  if (blockIdx.x >= items * splits) return;
  // The last tiles see the most tokens under the causal mask: they go first, those of all sequences in turn (of
  // sequences with as many tiles each, all the last ones, then all the ones before).  The head changes fastest, so that
  // with 8 heads an XCD reads one head's cache.
  const uint32_t split = blockIdx.x % splits, order = items - 1u - blockIdx.x / splits, h = order % a.heads, seqs = uniform(a.plan[3]);
  uint32_t f = order / a.heads;
  if (f < tiles / seqs * seqs) f = f % seqs * (tiles / seqs) + f / seqs;
  const uint32_t b = seq_with(a, f);
  const Seq s = seq_of(a, b);
  const uint32_t rows = (uint32_t)s.m * a.group, r0 = (f - a.first[b]) * a.tile_rows, w0 = r0 + wave * 16u * R;
  if (r0 >= rows) return;
  int32_t lo, hi, wlo, whi, all_lo, all_hi;
  rows_range(a, s, r0, a.tile_rows, &lo, &hi);
  rows_range(a, s, w0, 16u * R, &wlo, &whi);
  rows_common(a, s, w0, 16u * R, &all_lo, &all_hi);
  int32_t t0 = (int32_t)(split * chunk), t1 = t0 + (int32_t)chunk;
  t0 = t0 > (lo & ~15) ? t0 : lo & ~15;
  t1 = t1 < hi ? t1 : hi;
  if (a.pages == 0) t1 = t0;
  if (t0 >= t1 && splits > 1) return;
  // what the end of the kernel needs, out of the scalar registers meanwhile (a prompt of 8192 tokens: 680 us, 708 with
  // these spilled)
  __shared__ uint32_t s_keep[6];
  if (threadIdx.x == 0) {
    s_keep[0] = (uint32_t)s.q0;
    s_keep[1] = (uint32_t)s.m;
    s_keep[2] = h;
    s_keep[3] = r0;
    s_keep[4] = splits;
    s_keep[5] = ((f * a.heads + h) * splits + split) * a.tile_rows;  // the tile's rows among the split outputs
  }
  const uint32_t P = 1u << a.page_log2;
  const uint64_t page_size = (uint64_t)P * Page<BITS>::kToken;

  Share<BITS> sh;
  auto load = [&](int32_t t, int32_t page) __attribute__((always_inline)) {
    const uint8_t* p = a.cache + ((uint64_t)(page < 0 ? 0 : page) * a.heads + h) * page_size;
    load_keys<BITS>(p, P, (uint32_t)t & (P - 1u), lane, sh);
    load_values<BITS>(p, P, (uint32_t)t & (P - 1u), lane, sh);
  };
  // this wavefront's 16 tokens at t, as operands
  auto stage = [&](Stage<PREC>& d, uint2* flags, int32_t t, int32_t page) __attribute__((always_inline)) {
    uint32_t word = page < 0 ? 0xFFFF0000u : 0u, large = 0;
    if (__builtin_amdgcn_ballot_w64(odd_scales<BITS>(most(sh.ks[0], sh.ks[1])))) {
      const int32_t tok = t + (int32_t)n;
      if (page < 0 || tok < lo || tok >= t1) sh.ks[0] = sh.ks[1] = 0u;  // a token that no row sees may hold anything
      word |= gone_keys(sh.ks) << 16;
      if (shrink<BITS>(sh.ks)) large |= 1u;
    }
    f16x8 kh[4], kl[4];
    key_operands<BITS, PREC>(sh, kh, kl);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      d.k[0][wave][j][lane] = kh[j];
      if (PREC) d.k[PREC ? 1 : 0][wave][j][lane] = kl[j];
    }
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

  const bool cap = a.cap_in > 0.0f;
  f16x8 qh[R][4], ql[R][4];
  float qf[R], eff[R], m[R], sum[R], poison[R];
  int32_t row_lo[R], row_hi[R];
  f32x4 o[R][8], ones[R];
#pragma unroll
  for (int q = 0; q < R; ++q) {
    const uint64_t row = row_at(a, s, h, w0 + 16u * q + n);
    const bool have = w0 + 16u * q < rows;  // the last 16 may have rows of the next sequence among them: they see nothing
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      qh[q][j] = ql[q][j] = (f16x8)(_Float16)0.0f;
      if (have) qh[q][j] = *reinterpret_cast<const f16x8*>(a.qhi + row * kD + 8 * (4 * b4 + j));
      if (PREC && have) ql[q][j] = *reinterpret_cast<const f16x8*>(a.qlo + row * kD + 8 * (4 * b4 + j));
    }
    qf[q] = have ? a.qf[row] : 1.0f;
    eff[q] = cap ? 1.0f : qf[q];  // scores are eff sc: the product with qf waits for the exponent's fma
    m[q] = kLowest;
    sum[q] = poison[q] = 0.0f;
    row_lo[q] = row_hi[q] = 0;
    if (w0 + 16u * q + n < rows) visible(a, s, (int32_t)query_of(a, w0 + 16u * q + n), &row_lo[q], &row_hi[q]);
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
      sum[q] *= f;
      ones[q] *= f;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[q][i] *= f;
    }
  };
  uint32_t buf = 0;
  if (!PREC && t < t1) {
    stage(st[0], s_flags[0], t + mine, page);
    __syncthreads();
  }
  for (; t < t1; t += kTok) {
    const bool more = t + kTok < t1;
    if (PREC) {
      stage(st[0], s_flags[0], t + mine, page);
      __syncthreads();
    }
    if (more) {
      page = page_in(a, next);
      load(t + kTok + mine, page);
      next = entry_of(a, b, t + 2 * kTok + mine, t1);
    }
    const Stage<PREC>& d = st[buf];
    // blocks of 16 tokens with a flag, asked for once and not between the products
    const uint2 flags = s_flags[buf][lane & (kManyWaves - 1)];
    const uint32_t flagged = (uint32_t)__builtin_amdgcn_ballot_w64(lane < (uint32_t)kManyWaves && (flags.x | flags.y) != 0u);
    bool whole = false;
    if constexpr (!PREC) {
      if (!cap && !flagged && t >= all_lo && t + kTok <= all_hi && t + kTok <= t1) {
        // every row sees every token: each step's scores are under way during the softmax of the one before
        f32x4 sc[2][R][2];
        auto products = [&](int w, f32x4 (*x)[2]) __attribute__((always_inline)) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int q = 0; q < R; ++q) x[q][u] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const f16x8 kh = d.k[0][2 * w + u][j][lane];
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
    constexpr int kUnroll = PREC ? 2 : 1;  // without PREC the count depends on `whole`: such a loop is not unrolled
#pragma unroll kUnroll
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
          const f16x8 kh = d.k[0][2 * w + u][j][lane];
          if (PREC) {
            const f16x8 kl = d.k[PREC ? 1 : 0][2 * w + u][j][lane];
#pragma unroll
            for (int q = 0; q < R; ++q) {
              sc[q][u] = mfma(kl, qh[q][j], sc[q][u]);
              sc[q][u] = mfma(kh, ql[q][j], sc[q][u]);
            }
          }
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
              if ((fl & 0x10000u) || tok < row_lo[q] || tok >= row_hi[q] || tok >= t1) sc[q][u][i] = -__builtin_inff();
              else if (fl & 1u) poison[q] = __builtin_nanf("");
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
          if (PREC) sum[q] += p0 + p1;
          p.v[i] = u2((f16x2){(_Float16)p0, (_Float16)p1});
        }
        pf[q] = frag(p);
        // the sum of the rounded P, the one the output is weighted with, is one more product
        if (!PREC) ones[q] = mfma((f16x8)(_Float16)1.0f, pf[q], ones[q]);
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
    if (!PREC && more) {
      buf ^= 1u;
      stage(st[buf], s_flags[buf], t + kTok + mine, page);
    }
    __syncthreads();
  }

  // each wavefront's rows, 16 at a time, through its part of LDS: a row's values to 16 lanes
  __syncthreads();
  const Seq es = {(int64_t)uniform(s_keep[0]), (int32_t)uniform(s_keep[1]), 0, 0};
  const uint32_t eh = uniform(s_keep[2]), erows = (uint32_t)es.m * a.group, ew = uniform(s_keep[3]) + wave * 16u * R;
  const bool whole_tile = uniform(s_keep[4]) == 1u;
  const uint32_t first_part = uniform(s_keep[5]) + wave * 16u * R;
  const LaneInverse inv = lane_inverse(K, n);
#pragma unroll
  for (int q = 0; q < R; ++q) {
    const float total = PREC ? blocks_sum(sum[q]) : ones[q][0], bad = blocks_sum(poison[q]);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int i = 0; i < 8; i += 4)
        *reinterpret_cast<f32x4*>(&s_o[wave][n][8 * (4 * b4 + r) + i]) =
            (f32x4){o[q][i][r] + bad, o[q][i + 1][r] + bad, o[q][i + 2][r] + bad, o[q][i + 3][r] + bad};
    const uint32_t part = first_part + 16u * q;
    if (b4 == 0 && ew + 16u * q + n < erows) {
      if (whole_tile) a.lse[row_at(a, es, eh, ew + 16u * q + n)] = m[q] + __builtin_amdgcn_logf(total) - kPScaleLog2;
      else *reinterpret_cast<f32x2*>(a.pml + (uint64_t)(part + n) * 2) = (f32x2){m[q], total};
    }
    wave_sync();
#pragma unroll 1
    for (uint32_t k = 0; k < 4; ++k) {
      const uint32_t r = 4u * k + b4;
      if (ew + 16u * q + 4u * k >= erows) break;
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = s_o[wave][r][8 * n + i];
      const float tr = row_get_any(total, r);
      if (whole_tile) {
        store_row<BITS>(a, K, K.v, es, eh, ew + 16u * q + r, n, inv, y, tr);
      } else {
        float* d = a.po + (uint64_t)(part + r) * kD + 8 * n;
        *reinterpret_cast<f32x4*>(d) = (f32x4){y[0], y[1], y[2], y[3]};
        *reinterpret_cast<f32x4*>(d + 4) = (f32x4){y[4], y[5], y[6], y[7]};
      }
    }
    wave_sync();
  }
}

// Accumulated weights of many rows: a wavefront owns 64 tokens of a (sequence, head), keeps their keys as
// operands, forms their scores with every row again and adds the sum of exp(s - lse) over the rows, in a
// fixed order.  The four wavefronts share each 16 rows' operands through LDS, the next ones' on their way.
// 4 x 129 queries on up to 5003 tokens, 8 heads, 4 a head: 83 us (142 us with a branch a score and each wavefront
// fetching the rows by itself).  Storing the scores instead, as for few rows, would move 0.6 GB.
template <int BITS>
__global__ __launch_bounds__(kAttBlock, 2) void weights_many_kernel(AttendArgs a, uint32_t blocks) {
  __shared__ f16x8 s_q[2][2][4][64];  // [buffer][part][step][lane]
  __shared__ float s_f[2][16], s_l[2][16];
  const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 15u, b4 = lane >> 4;
  // consecutive workgroups go to the 8 XCDs in turn: those of one (sequence, head), which read the same rows, meet
  // in one XCD's L2
  const uint32_t bh = blockIdx.x / 8u / blocks * 8u + blockIdx.x % 8u, h = bh % a.heads, b = bh / a.heads;
  if (bh >= a.seqs * a.heads) return;
  const Seq s = seq_of(a, b);
  const int32_t first = (int32_t)((blockIdx.x / 8u % blocks) * 64u * kAttWaves), t = first + 64 * (int32_t)wave;
  const uint32_t rows = (uint32_t)s.m * a.group;
  if (first >= s.n || a.pages == 0) return;
  // queries [i0, i1) see some of the workgroup's tokens
  const int64_t back = s.back, last = (int64_t)first + 64 * kAttWaves - 1;
  const int64_t i0 = a.causal && first > back ? first - back : 0, i1 = a.window && last + a.window - back < s.m ? last + a.window - back : s.m;
  if (i0 >= i1) return;
  const uint32_t P = 1u << a.page_log2;
  const uint64_t page_size = (uint64_t)P * Page<BITS>::kToken;
  f16x8 kh[4][4], kl[4][4];
  uint32_t hidden = 0, some = 0;  // of the lane's 16 tokens, those that take no part; whether any of the 64 does not
  float factor[4];                // undoes a block's shrunk keys
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int32_t page = page_of(a, b, t + 16 * u, s.n);
    uint32_t gone = page < 0 ? 0xFFFFu : 0u;
    factor[u] = 1.0f;
    Share<BITS> sh;
    load_keys<BITS>(a.cache + ((uint64_t)(page < 0 ? 0 : page) * a.heads + h) * page_size, P, (uint32_t)(t + 16 * u) & (P - 1u), lane, sh);
    if (__builtin_amdgcn_ballot_w64(odd_scales<BITS>(most(sh.ks[0], sh.ks[1])))) {
      if (page < 0 || t + 16 * u + (int32_t)n >= s.n) sh.ks[0] = sh.ks[1] = 0u;
      gone |= gone_keys(sh.ks);
      if (shrink<BITS>(sh.ks)) factor[u] = kShrunk;
    }
    hidden |= (gone >> (4u * b4) & 15u) << (4 * u);
    some |= gone;
    key_operands<BITS, true>(sh, kh[u], kl[u]);
  }
  float acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
  // a thread's share of 16 rows: group threadIdx mod 16 of row threadIdx / 16, in both parts
  const uint64_t base = row_at(a, s, h, 0);
  const uint32_t lr = threadIdx.x >> 4, lg = threadIdx.x & 15u;
  f16x8 qh, ql;
  float qf = 0.0f, lse = 0.0f;
  auto fetch = [&](uint32_t r0) __attribute__((always_inline)) {
    const uint64_t row = base + r0 + lr;
    qh = *reinterpret_cast<const f16x8*>(a.qhi + row * kD + 8 * lg);
    ql = *reinterpret_cast<const f16x8*>(a.qlo + row * kD + 8 * lg);
    if (lg == 0) {
      qf = a.qf[row];
      lse = a.lse[row];
    }
  };
  const uint32_t r1 = (uint32_t)i1 * a.group;
  uint32_t buf = 0, r0 = (uint32_t)i0 * a.group & ~15u;
  fetch(r0);
  for (; r0 < r1; r0 += 16, buf ^= 1u) {
    s_q[buf][0][lg & 3u][lr + 16u * (lg >> 2)] = qh;
    s_q[buf][1][lg & 3u][lr + 16u * (lg >> 2)] = ql;
    if (lg == 0) {
      s_f[buf][lr] = qf;
      s_l[buf][lr] = lse;
    }
    __syncthreads();
    if (r0 + 16 < r1) fetch(r0 + 16);
    int32_t lo, hi, all_lo, all_hi;
    rows_range(a, s, r0, 16, &lo, &hi);
    if (t >= hi || t + 64 <= lo) continue;
    rows_common(a, s, r0, 16, &all_lo, &all_hi);
    f16x8 oh[4], ol[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      oh[j] = s_q[buf][0][j][lane];
      ol[j] = s_q[buf][1][j][lane];
    }
    const float f = s_f[buf][n], ls = s_l[buf][n];
    f32x4 raw[4];
    float sc[16];
#pragma unroll
    for (int u = 0; u < 4; ++u) raw[u] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // the four blocks in turn: no product waits for the one before
#pragma unroll
      for (int u = 0; u < 4; ++u) raw[u] = mfma(kl[u][j], oh[j], raw[u]);
#pragma unroll
      for (int u = 0; u < 4; ++u) raw[u] = mfma(kh[u][j], ol[j], raw[u]);
#pragma unroll
      for (int u = 0; u < 4; ++u) raw[u] = mfma(kh[u][j], oh[j], raw[u]);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) sc[i] = raw[i >> 2][i & 3] * (f * factor[i >> 2]);
    cap_scores<16>(a, sc);
    if (!some && t >= all_lo && t + 64 <= all_hi) {
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i] += __builtin_amdgcn_exp2f(sc[i] - ls);
    } else {
      int32_t row_lo = 0, row_hi = 0;
      if (r0 + n < rows) visible(a, s, (int32_t)query_of(a, r0 + n), &row_lo, &row_hi);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int32_t tok = t + 16 * (i >> 2) + 4 * (int32_t)b4 + (i & 3);
        const float p = __builtin_amdgcn_exp2f(sc[i] - ls);
        acc[i] += bool((tok >= row_lo) & (tok < row_hi) & !((hidden >> i) & 1u)) ? p : 0.0f;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float x = acc[i];
    x += lane_xor<1>(x);
    x += lane_xor<2>(x);
    x += lane_xor<4>(x);
    x += lane_xor<8>(x);
    const int32_t tok = t + 16 * (i >> 2) + 4 * (int32_t)b4 + (i & 3);
    if (n == 0 && tok < s.n) a.weights[(uint64_t)bh * a.wstride + (uint32_t)tok] += x;
  }
}

}  // namespace hq_kv

using namespace hq_kv;

namespace {

uint64_t align256(uint64_t v) { return (v + 255u) & ~(uint64_t)255u; }

// How a call is cut, and the workspace it takes.
struct Plan {
  uint32_t max_q, rows, tile_rows, bound, most, parts, grid, lsplits, lchunk, wrows, wpad;
  bool few, light;
  uint64_t plan, first, qhi, qlo, qf, lse, pml, po, lpml, lpo, scores, bytes;
};

// HQ_OK, or an error for a call that the launches cannot take.
int plan_of(const hq_kv_cache& c, const hq_kv_attend_args& g, Plan* out) {
  Plan p;
  const uint32_t group = g.q_heads / c.heads;
  const uint64_t each = g.q_start || g.seqs == 0 ? g.total_q : g.total_q / g.seqs, sh = (uint64_t)g.seqs * c.heads;
  p.max_q = (uint32_t)(each < g.max_q ? each : g.max_q);
  // rows of a sequence, at most, and of a head
  const uint64_t rows = (uint64_t)p.max_q * group, all = g.total_q * group;
  if (all > 0x7FFFFF00ull || all * c.heads > kMaxThreads / 16) return HQ_ERR_INVALID_ARG;
  p.rows = (uint32_t)all;
  p.few = rows <= 16;
  // up to 16 rows: one tile, split over many workgroups; beyond, 16 rows a wavefront while that covers them,
  // then 32
  p.tile_rows = p.few ? 16 : rows <= 128 ? 128 : 256;
  const uint64_t last = rows % p.tile_rows;  // of equal sequences
  p.light = !p.few && (g.q_start ? g.seqs > 1 : last > 0 && last <= 16);
  // Light tiles (all tiles of few rows): workgroups to fill 256 CUs and to even out ragged lengths, each with enough
  // tokens to be worth its start (about 5 us) and its part of the join: 2048 of at least 1024 tokens, or of 512 where that
  // leaves fewer than 512 (64 sequences of 4001 tokens: 59 us at 1024, 67 at 512; one of 32768: 31 and 30;
  // one of 301: 14 us whole, 17 in two).
  auto cut = [&](uint64_t splits, uint64_t least, uint32_t* chunk) {
    const uint64_t most = (g.max_len + least - 1) / least;
    if (splits > most) splits = most;
    if (splits < 1) splits = 1;
    *chunk = (uint32_t)(((g.max_len + splits - 1) / splits + 127) / 128 * 128);
    if (*chunk == 0) *chunk = 128;
    const uint32_t n = (g.max_len + *chunk - 1) / *chunk;
    return n ? n : 1u;
  };
  p.lsplits = p.few || p.light ? cut(sh ? (2048 + sh - 1) / sh : 1, sh * ((g.max_len + 1023) / 1024) >= 512 ? 1024 : 512, &p.lchunk) : 1;
  // Full tiles of a head: what the rows fill, and each sequence's last if it is not light.  Their number is known on the
  // device (plan_tiles), which splits them over what workgroups and split outputs there are: 1536 of at least 512 tokens,
  // unless the tiles are two a CU as they stand.  Where half of them or more may not exist, because many sequences share few
  // rows, 512 of 256 rows or 1024 of 128: two rounds of the chip or more, and 68 MB.
  const uint64_t odd = p.light ? all / 17 : all, tiles = (rows + p.tile_rows - 1) / p.tile_rows;
  uint64_t bound = all / p.tile_rows + (odd < g.seqs ? odd : g.seqs), parts = 0;
  if (tiles * g.seqs < bound) bound = tiles * g.seqs;
  if (p.few) bound = 0;
  const uint64_t items = bound * c.heads, filled = (all + p.tile_rows - 1) / p.tile_rows * c.heads;
  p.most = (g.max_len + 511) / 512;
  if (p.most > 1 && items) {
    if (2 * filled <= items) parts = filled < 512 ? 512 * 256 / p.tile_rows : 0;
    else if (items < 512) parts = items * ((1536 + items - 1) / items);
    if (parts > items * p.most) parts = items * p.most;
  }
  const uint64_t grid = items > parts ? items : parts;
  if (grid > kMaxThreads / kManyBlock || sh * p.lsplits > kMaxThreads / kAttBlock) return HQ_ERR_INVALID_ARG;
  // the weights: a thread a token
  if (g.weights && (sh + 7) * ((g.max_len + 255u) / 256u) > kMaxThreads / kAttBlock) return HQ_ERR_INVALID_ARG;
  p.bound = (uint32_t)bound;
  p.parts = (uint32_t)parts;
  p.grid = (uint32_t)grid;
  p.wrows = p.few && g.weights ? (uint32_t)rows : 0;
  p.wpad = (g.max_len + 31u) / 16u * 16u;  // whole blocks of 16 from any block's start
  uint64_t at = 0;
  auto take = [&](uint64_t n) {
    const uint64_t here = at;
    at = align256(at + n);
    return here;
  };
  // 16 rows are read together from any row on
  const uint64_t r = all * c.heads + 16, split = parts * p.tile_rows, lsplit = p.lsplits > 1 ? sh * p.lsplits * 16 : 0;
  p.plan = take(p.few ? 0 : 16);
  p.first = take(p.few ? 0 : ((uint64_t)g.seqs + 1) * 4);
  p.lse = take(r * 4);
  p.qf = take(p.few ? 0 : r * 4);
  p.qhi = take(p.few ? 0 : r * kD * 2);
  p.qlo = take(p.few || !g.weights ? 0 : r * kD * 2);
  p.pml = take(split * 8);
  p.po = take(split * kD * 4);
  p.lpml = take(lsplit * 8);
  p.lpo = take(lsplit * kD * 4);
  p.scores = take(p.wrows * sh * p.wpad * 4);
  p.bytes = at;
  *out = p;
  return HQ_OK;
}

template <int BITS, bool PREC, int R>
hipError_t launch_many(const AttendArgs& a, const Tables& T, uint32_t grid, hipStream_t st) {
  // more dynamic LDS than the default limit: asked for once per kernel (the attribute holds for every device)
  static const hipError_t set = hipFuncSetAttribute(reinterpret_cast<const void*>(&attend_many_kernel<BITS, PREC, R>),
                                                    hipFuncAttributeMaxDynamicSharedMemorySize, (int)many_lds<PREC>());
  if (set != hipSuccess) return set;
  hipLaunchKernelGGL((attend_many_kernel<BITS, PREC, R>), dim3(grid), dim3(kManyBlock), many_lds<PREC>(), st, a, T);
  return hipSuccess;
}

// The join of split tiles.  A workgroup a row while those are at most 16 a CU, 16 lanes a row beyond: 64 rows of 12 splits
// 5 us as one, 49152 rows of 3 splits 87 us against 14 us.
template <int BITS, bool LIGHT>
void launch_combine(const AttendArgs& a, const Tables& T, uint32_t tiles, uint32_t per, hipStream_t st) {
  const dim3 block(kAttBlock);
  if ((uint64_t)tiles * per <= 4096) hipLaunchKernelGGL((combine_kernel<BITS, true, LIGHT>), dim3(tiles * per), block, 0, st, a, T, per, tiles * per);
  else hipLaunchKernelGGL((combine_kernel<BITS, false, LIGHT>), dim3((tiles * per + 15) / 16), block, 0, st, a, T, per, tiles * per);
}

template <int BITS>
hipError_t launch_attend(const AttendArgs& a, const Tables& T, const Plan& p, hipStream_t st) {
  const dim3 block(kAttBlock);
  const bool prec = a.weights != nullptr;
  const uint32_t sh = a.seqs * a.heads, rows = a.max_q * a.group;
  if (!p.few) {
    const uint32_t span = (uint64_t)a.rows * a.heads / 64 >= 1024 ? 64 : 16;
    hipLaunchKernelGGL((rotate_rows_kernel<BITS>), dim3((a.rows + span - 1) / span * a.heads + 1), block, 0, st, a, T, prec ? 2 : 1, span);
  }
  if (p.few || p.light) {
    const dim3 grid(sh * a.lsplits);
    if (prec) hipLaunchKernelGGL((attend_few_kernel<BITS, true>), grid, block, 0, st, a, T);
    else hipLaunchKernelGGL((attend_few_kernel<BITS, false>), grid, block, 0, st, a, T);
    if (a.lsplits > 1) launch_combine<BITS, true>(a, T, sh, rows < 16 ? rows : 16, st);
  }
  if (p.grid) {
    const hipError_t e = a.tile_rows == 128 ? prec ? launch_many<BITS, true, 1>(a, T, p.grid, st) : launch_many<BITS, false, 1>(a, T, p.grid, st)
                                            : prec ? launch_many<BITS, true, 2>(a, T, p.grid, st) : launch_many<BITS, false, 2>(a, T, p.grid, st);
    if (e != hipSuccess) return e;
    // of split tiles there are half as many as parts
    const uint32_t items = a.bound * a.heads, per = rows < a.tile_rows ? (rows + 15) / 16 * 16 : a.tile_rows;
    if (a.parts) launch_combine<BITS, false>(a, T, items < a.parts / 2 ? items : a.parts / 2, per, st);
  }
  if (prec && a.max_len) {
    const uint32_t blocks = (a.max_len + 255u) / 256u;  // of 256 tokens
    if (p.few) hipLaunchKernelGGL(weights_few_kernel, dim3(sh * blocks), block, 0, st, a, blocks);
    else hipLaunchKernelGGL((weights_many_kernel<BITS>), dim3((sh + 7u) / 8u * 8u * blocks), block, 0, st, a, blocks);
  }
  return hipGetLastError();
}

}  // namespace

extern "C" {

int hq_kv_attend_workspace_size(const hq_kv_cache* cache, const hq_kv_attend_args* args, size_t* bytes) {
  if (!bytes) return HQ_ERR_INVALID_ARG;
  if (int rc = check_attend(cache, args)) return rc;
  Plan p;
  if (int rc = plan_of(*cache, *args, &p)) return rc;
  *bytes = p.bytes;
  return HQ_OK;
}

int hq_kv_attend(const hq_kv_cache* cache, const hq_kv_attend_args* args, void* workspace, size_t workspace_bytes,
                 hq_stream_t stream) {
  if (int rc = check_attend(cache, args)) return rc;
  AttendArgs a;
  Tables T;
  bool nothing;
  if (int rc = attend_args(*cache, *args, &a, &T, &nothing)) return rc;
  if (nothing) return HQ_OK;
  Plan p;
  if (int rc = plan_of(*cache, *args, &p)) return rc;
  if (!workspace || ((uintptr_t)workspace & 255u) || workspace_bytes < p.bytes) return HQ_ERR_INVALID_ARG;
  a.max_q = p.max_q;
  a.rows = p.rows;
  a.tile_rows = p.tile_rows;
  a.bound = p.bound;
  a.parts = p.parts;
  a.most = p.most;
  a.lsplits = p.lsplits;
  a.lchunk = p.lchunk;
  a.light = p.light;
  a.wrows = p.wrows;
  a.wpad = p.wpad;
  char* w = static_cast<char*>(workspace);
  a.plan = reinterpret_cast<uint32_t*>(w + p.plan);
  a.first = reinterpret_cast<uint32_t*>(w + p.first);
  a.qhi = reinterpret_cast<_Float16*>(w + p.qhi);
  a.qlo = reinterpret_cast<_Float16*>(w + p.qlo);
  a.qf = reinterpret_cast<float*>(w + p.qf);
  a.lse = reinterpret_cast<float*>(w + p.lse);
  a.pml = reinterpret_cast<float*>(w + p.pml);
  a.scores = p.wrows ? reinterpret_cast<float*>(w + p.scores) : nullptr;
  a.po = reinterpret_cast<float*>(w + p.po);
  a.lpml = reinterpret_cast<float*>(w + p.lpml);
  a.lpo = reinterpret_cast<float*>(w + p.lpo);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const hipError_t e = cache->bits == 4 ? launch_attend<4>(a, T, p, st) : launch_attend<8>(a, T, p, st);
  return e == hipSuccess ? HQ_OK : HQ_ERR_HIP;
}

}  // extern "C"
