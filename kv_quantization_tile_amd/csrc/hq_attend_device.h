// hq_attend_device.h -- attention over the paged SRFT cache: what its kernels share (hq_attend.hip, hq_tree.hip).  The
// mathematics and the operands' layout: hq_attend.hip.
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/hq.h"
#include "hq_kv_device.h"
#include "hq_kv_internal.h"

namespace hq_kv {

constexpr int kAttBlock = 256;
constexpr int kAttWaves = 4;
constexpr int kPad = kD + 4;         // row of a tile in LDS, in floats
constexpr float kPScaleLog2 = 8.0f;  // P is stored as p 2^8
constexpr float kSlack = 6.0f;       // the reference may lag the maximum by this much (log2)
constexpr float kLowest = -3.402823466e38f;  // the reference before the first score: no finite score is below it

struct AttendArgs {
  const uint8_t* cache;
  const void* q;
  void* out;
  const int32_t *q_start, *table, *lens;
  float* weights;
  uint64_t wstride, total_q;
  int64_t qt, qh;  // strides of q in values
  uint32_t heads, group, q_heads, pages, page_log2, width, seqs, max_q, max_len;
  uint32_t group_mul, group_shift;  // query_of
  // rows of a head: `rows` = total_q group of them, a sequence's from q0 group on, cut into tiles of tile_rows
  uint32_t rows, tile_rows, window;
  uint32_t lsplits, lchunk;     // splits of a light tile (of up to 16 rows, a sequence's last), tokens of each
  uint32_t bound, parts, most;  // full tiles of a head, at most; split tiles there is room for; splits of a full tile, at most
  uint32_t wrows, wpad;  // stored scores: rows of a (sequence, head), tokens a row
  int causal, q_f32, out_f32, vec;
  int light;  // light tiles are left to the few rows' kernel
  float scale_log2, cap_in, cap_out;  // scores in log2 units; s = cap_out tanh(cap_in s) when cap_in > 0
  // workspace
  uint32_t* plan;       // full tiles of a head, their splits, tokens of each, sequences with a full tile (plan_tiles)
  uint32_t* first;      // [seqs + 1] full tiles before a sequence
  _Float16 *qhi, *qlo;  // [heads][rows][128]
  float* qf;            // [heads][rows] factor of a row's products
  float* lse;           // [heads][rows]
  float *po, *pml;      // [full tiles][heads][splits][tile_rows], 128 and 2 values
  float *lpo, *lpml;    // [seqs][heads][lsplits][16], the same of light tiles
  float* scores;        // [seqs][heads][wrows][wpad]
};

// Query r / group of row r < 2^31: with 2^sh >= group > 2^(sh-1) and M = floor(2^(31+sh) / group) + 1 the product r M
// exceeds r 2^(31+sh) / group by less than 2^(31+sh) / group, so its quotient by 2^(31+sh) is exact.
__device__ __forceinline__ uint32_t query_of(const AttendArgs& a, uint32_t r) { return (uint32_t)(((uint64_t)r * a.group_mul) >> a.group_shift); }

struct Seq {
  int64_t q0;
  int32_t m, n;  // queries that are computed (the first max_q), cached tokens
  int32_t back;  // position of query 0: the tokens less all the sequence's queries, computed or not
};
__device__ __forceinline__ Seq seq_of(const AttendArgs& a, uint32_t b) {
  Seq s;
  int64_t all;
  if (a.q_start) {
    const int64_t x = a.q_start[b], y = a.q_start[b + 1], top = (int64_t)a.total_q;
    s.q0 = x < 0 ? 0 : x > top ? top : x;
    all = y < s.q0 ? 0 : (y > top ? top : y) - s.q0;
  } else {
    all = (int64_t)(a.total_q / a.seqs);
    s.q0 = all * b;
  }
  s.m = (int32_t)(all < (int64_t)a.max_q ? all : (int64_t)a.max_q);
  const uint64_t held = (uint64_t)a.width << a.page_log2, most = held < a.max_len ? held : a.max_len;
  const int32_t n = a.lens[b];
  s.n = n < 0 ? 0 : (uint64_t)n < most ? n : (int32_t)most;
  s.back = (int32_t)(s.n - all);
  return s;
}
// Visible tokens [lo, hi) of query i of a sequence.
__device__ __forceinline__ void visible(const AttendArgs& a, const Seq& s, int32_t i, int32_t* lo, int32_t* hi) {
  const int32_t pos = s.back + i;
  int32_t h = a.causal ? (pos + 1 < s.n ? pos + 1 : s.n) : s.n;
  if (h < 0) h = 0;
  int64_t l = a.window ? (int64_t)pos + 1 - (int64_t)a.window : 0;
  if (l < 0) l = 0;
  *lo = l > h ? h : (int32_t)l;
  *hi = h;
}
// Tokens that some row of [r0, r0 + count) sees, as one range.
__device__ __forceinline__ void rows_range(const AttendArgs& a, const Seq& s, uint32_t r0, uint32_t count, int32_t* lo, int32_t* hi) {
  const uint32_t rows = (uint32_t)s.m * a.group;
  if (r0 >= rows) {
    *lo = *hi = 0;
    return;
  }
  const uint32_t r1 = r0 + count < rows ? r0 + count - 1u : rows - 1u;
  int32_t l0, h0, l1, h1;
  visible(a, s, (int32_t)query_of(a, r0), &l0, &h0);
  visible(a, s, (int32_t)query_of(a, r1), &l1, &h1);
  *lo = l0;
  *hi = h1;
}

// Tokens that every row of [r0, r0 + count) sees; none if some of the rows do not exist.
__device__ __forceinline__ void rows_common(const AttendArgs& a, const Seq& s, uint32_t r0, uint32_t count, int32_t* lo, int32_t* hi) {
  *lo = *hi = 0;
  if (r0 + count > (uint32_t)s.m * a.group) return;
  int32_t x;
  visible(a, s, (int32_t)query_of(a, r0 + count - 1u), lo, &x);
  visible(a, s, (int32_t)query_of(a, r0), &x, hi);
}

__device__ __forceinline__ float swap16_max(float x) {
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float swap32_max(float x) {
  const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float blocks_max(float x) { return swap32_max(swap16_max(x)); }
__device__ __forceinline__ float blocks_sum(float x) {
  auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ __forceinline__ f16x2 h2(uint32_t u) { return __builtin_bit_cast(f16x2, u); }
__device__ __forceinline__ uint32_t u2(f16x2 h) { return __builtin_bit_cast(uint32_t, h); }

struct U32x4 {
  uint32_t v[4];
};
__device__ __forceinline__ f16x8 frag(const U32x4& u) { return __builtin_bit_cast(f16x8, u); }

// 8 codes (one group of one token) -> 4 registers of code pairs, exact.  Pair order:
// 4 bits (c_i, c_{i+4}), 8 bits (c_2i, c_2i+1).
template <int BITS>
__device__ __forceinline__ void code_pairs(const uint32_t* w, f16x2 out[4]) {
  if (BITS == 4) {
    const uint32_t u = w[0] ^ 0x88888888u;
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = h2(((u >> (4 * i)) & 0x000F000Fu) | 0x64006400u) - (f16x2){(_Float16)1032.0f, (_Float16)1032.0f};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = w[i >> 1] ^ 0x80808080u;
      // bytes: code, 0x64, code, 0x64
      const uint32_t p = __builtin_amdgcn_perm(u, 0x64646464u, (i & 1) ? 0x00070006u : 0x00050004u);
      out[i] = h2(p) - (f16x2){(_Float16)1152.0f, (_Float16)1152.0f};
    }
  }
}

// The same for tokens a and b: out[i] = (code_i of a, code_i of b), i = 0..7.
template <int BITS>
__device__ __forceinline__ void token_pairs(const uint32_t* a, const uint32_t* b, f16x2 out[8]) {
  if (BITS == 4) {
    const uint32_t lo = __builtin_amdgcn_perm(b[0], a[0], 0x05040100u) ^ 0x88888888u;  // codes 0..3 of a, of b
    const uint32_t hi = __builtin_amdgcn_perm(b[0], a[0], 0x07060302u) ^ 0x88888888u;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      out[i] = h2((((i < 4 ? lo : hi) >> (4 * (i & 3))) & 0x000F000Fu) | 0x64006400u) - (f16x2){(_Float16)1032.0f, (_Float16)1032.0f};
  } else {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint32_t p = __builtin_amdgcn_perm(b[w], a[w], 0x05010400u) ^ 0x80808080u;  // a0 b0 a1 b1
      const uint32_t q = __builtin_amdgcn_perm(b[w], a[w], 0x07030602u) ^ 0x80808080u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t r = __builtin_amdgcn_perm(i < 2 ? p : q, 0x64646464u, (i & 1) ? 0x00070006u : 0x00050004u);
        out[4 * w + i] = h2(r) - (f16x2){(_Float16)1152.0f, (_Float16)1152.0f};
      }
    }
  }
}

// One lane's share of 16 tokens.  Keys: token n = lane mod 16, groups 4b..4b+3.  Values: tokens 4b..4b+3,
// group n.
template <int BITS>
struct Share {
  uint32_t k[BITS], v[BITS];  // 4 x 8 codes each
  uint32_t ks[2], vs[2];      // 4 binary16 scales each
};

template <int BITS>
__device__ __forceinline__ void load_keys(const uint8_t* page, uint32_t P, uint32_t t, uint32_t lane, Share<BITS>& s) {
  const uint32_t n = lane & 15u, b = lane >> 4;
  const uint4* kc = reinterpret_cast<const uint4*>(page + Page<BITS>::k_code(P, t + n) + b * 4u * BITS);
#pragma unroll
  for (int i = 0; i < BITS / 4; ++i) {
    const uint4 u = kc[i];
    s.k[4 * i] = u.x; s.k[4 * i + 1] = u.y; s.k[4 * i + 2] = u.z; s.k[4 * i + 3] = u.w;
  }
  const uint2 u = *reinterpret_cast<const uint2*>(page + Page<BITS>::k_scale(P, t + n) + 8u * b);
  s.ks[0] = u.x;
  s.ks[1] = u.y;
}
template <int BITS>
__device__ __forceinline__ void load_values(const uint8_t* page, uint32_t P, uint32_t t, uint32_t lane, Share<BITS>& s) {
  const uint32_t n = lane & 15u, b = lane >> 4;
  const uint4* vc = reinterpret_cast<const uint4*>(page + Page<BITS>::v_code(P, t + 4u * b, n));
#pragma unroll
  for (int i = 0; i < BITS / 4; ++i) {
    const uint4 u = vc[i];
    s.v[4 * i] = u.x; s.v[4 * i + 1] = u.y; s.v[4 * i + 2] = u.z; s.v[4 * i + 3] = u.w;
  }
  const uint2 u = *reinterpret_cast<const uint2*>(page + Page<BITS>::v_scale(P, t + 4u * b, n));
  s.vs[0] = u.x;
  s.vs[1] = u.y;
}

// A lane's keys as operands: hi[j] is group 4b + j, lo[j] what rounding it left.
template <int BITS, bool PREC>
__device__ __forceinline__ void key_operands(const Share<BITS>& s, f16x8 hi[4], f16x8 lo[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f16x2 c[4];
    code_pairs<BITS>(s.k + j * (BITS / 4), c);
    const _Float16 d = __builtin_bit_cast(_Float16, (uint16_t)(s.ks[j >> 1] >> (16 * (j & 1))));
    const f16x2 dd = {d, d};
    U32x4 h, l;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f16x2 p = c[i] * dd;
      h.v[i] = u2(p);
      if (PREC) l.v[i] = u2(__builtin_elementwise_fma(c[i], dd, -p));
    }
    hi[j] = frag(h);
    if (PREC) lo[j] = frag(l);
  }
}

__device__ __forceinline__ f32x4 mfma(f16x8 a, f16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

// Raw products of 16 tokens with 16 rows: lane (n, b) gets row n, tokens 4b..4b+3.
template <bool PREC>
__device__ __forceinline__ f32x4 scores16(const f16x8 kh[4], const f16x8 kl[4], const f16x8 qh[4], const f16x8 ql[4]) {
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (PREC) {
      acc = mfma(kl[j], qh[j], acc);
      acc = mfma(kh[j], ql[j], acc);
    }
    acc = mfma(kh[j], qh[j], acc);
  }
  return acc;
}

// A lane's values as two of the four registers of the operand of 32 tokens: out[i][w], i the
// coordinate within the lane's group, w the pair of tokens.
template <int BITS>
__device__ __forceinline__ void value_operands(const Share<BITS>& s, uint32_t out[8][2]) {
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    f16x2 c[8];
    token_pairs<BITS>(s.v + (2 * w) * (BITS / 4), s.v + (2 * w + 1) * (BITS / 4), c);
    const f16x2 d = h2(s.vs[w]);
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i][w] = u2(c[i] * d);
  }
}

// Scales from here on are large: 2^13 (2^9 at 8 bits), below which 7 (127) of them stay under binary16's 65504.
template <int BITS>
constexpr uint32_t kLargeScale = BITS == 4 ? 0x7000u : 0x6000u;

// The largest bits of pairs of scales, and whether one of a pair is out of the ordinary: large, infinite, NaN, or with the
// sign that marks the key of a token that takes no part.
__device__ __forceinline__ u16x2 most(uint32_t a, uint32_t b) { return __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)); }
template <int BITS>
__device__ __forceinline__ bool odd_scales(u16x2 m) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_sub_sat(m, (u16x2)(uint16_t)(kLargeScale<BITS> - 1u))) != 0u;
}
// Takes the scales times 2^-7 if one of the wavefront's is large (and finite): what is made of them is then 2^-7 of what it
// stands for.  A scale in the same 16 tokens as a large one is then off by up to 2^-18, at most 2^-27 of the large one.
template <int BITS>
__device__ __forceinline__ bool shrink(uint32_t s[2]) {
  bool large = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = (s[i >> 1] >> (16 * (i & 1))) & 0x7FFFu;
    large |= h >= kLargeScale<BITS> && h < 0x7C00u;
  }
  if (!__builtin_amdgcn_ballot_w64(large)) return false;
#pragma unroll
  for (int i = 0; i < 2; ++i) s[i] = u2(h2(s[i]) * (f16x2){(_Float16)0x1p-7f, (_Float16)0x1p-7f});
  return true;
}
constexpr float kShrunk = 128.0f;
// Which of 16 tokens (bit 0: the first) have keys that take no part.
__device__ __forceinline__ uint32_t gone_keys(const uint32_t ks[2]) { return (uint32_t)__builtin_amdgcn_ballot_w64((ks[0] & 0x8000u) != 0u) & 0xFFFFu; }
// Which of the lane's four value scales are NaN or infinite (bit r: token 4b + r).
__device__ __forceinline__ uint32_t bad_scales(const uint32_t vs[2]) {
  uint32_t bad = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) bad |= ((vs[i >> 1] >> (16 * (i & 1))) & 0x7C00u) == 0x7C00u ? 1u << i : 0u;
  return bad;
}
// Zeroes the scales of the tokens in `mask`.
__device__ __forceinline__ void drop_scales(uint32_t vs[2], uint32_t mask) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (mask & (1u << i)) vs[i >> 1] &= (i & 1) ? 0x0000FFFFu : 0xFFFF0000u;
}

// tanh from the exponential: 1 - 2 / (e^2x + 1) away from zero, the odd series to x^7 below 2^-3 in
// magnitude (the next term, 62 x^9 / 2835, is below 2^-29 of x), so that small scores keep their relative
// precision.  NaN stays NaN (a key whose scales are NaN).
__device__ __forceinline__ float tanh32(float x) {
  const float a = fabsf(x), x2 = x * x;
  const float e = __builtin_amdgcn_exp2f((a > 20.0f ? 20.0f : a) * 2.885390081777927f);
  const float big = __builtin_fmaf(-2.0f, __builtin_amdgcn_rcpf(e + 1.0f), 1.0f);
  const float small = __builtin_fmaf(x2, __builtin_fmaf(x2, __builtin_fmaf(x2, -17.0f / 315.0f, 2.0f / 15.0f), -1.0f / 3.0f), 1.0f) * a;
  return __builtin_copysignf(a < 0.125f ? small : big, x);
}

template <int N>
__device__ __forceinline__ void cap_scores(const AttendArgs& a, float* s) {
  if (a.cap_in > 0.0f) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = a.cap_out * tanh32(s[i] * a.cap_in);
  }
}

// LDS written by some lanes of a wavefront is read by others of the same one.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ---------------------------------------------------------------------------------------------
// Row `r` of head h (zeros unless `have`), by the caller's 16 lanes: transformed, scaled by a power of two, in two
// binary16 parts in the operand's order, to hi[128] (and lo[128] unless null).  Returns the factor that turns the
// row's products into scores.
template <int BITS>
__device__ __forceinline__ float rotate_row(const AttendArgs& a, const Tables& K, const float* lam, uint32_t h, uint32_t r, bool have, uint32_t l,
                                            const LaneForward& f, _Float16* hi, _Float16* lo) {
  const uint32_t kappa = rev4(l);
  float m[8], x[8], y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t c = 2 * (kappa + 16 * i);
    m[2 * i] = packing(c) * a.scale_log2;
    m[2 * i + 1] = packing(c + 1) * a.scale_log2;
    if (K.scaled) {
      m[2 * i] *= lam[c];
      m[2 * i + 1] *= lam[c + 1];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = 0.0f;
  if (have) {
    const uint32_t i = query_of(a, r);
    const int64_t at = (int64_t)i * a.qt + (int64_t)(h * a.group + r - i * a.group) * a.qh + 8 * l;
    if (a.q_f32) {
      const float* p = static_cast<const float*>(a.q) + at;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = p[i];
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(a.q) + at;
      if (a.vec) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[2 * i] = __uint_as_float(w[i] << 16);
          x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float((uint32_t)p[i] << 16);
      }
    }
  }
  forward_row(x, y, m, l, f);
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(y[i]));
  top = fmaxf(top, lane_xor<8>(top));
  top = fmaxf(top, lane_xor<4>(top));
  top = fmaxf(top, lane_xor<2>(top));
  top = fmaxf(top, lane_xor<1>(top));
  int e = 0;
  if (top > 0.0f && __builtin_isfinite(top)) e = 15 - __builtin_amdgcn_frexp_expf(top);
  e = e < 120 ? e : 120;  // the factor 2^-e stays normal: a masked score (-inf times it) is never NaN
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t g = (kappa >> 2) + 4u * (i >> 1), c = 2u * (kappa & 3u) + (i & 1);
    const uint32_t at = 8u * g + (BITS == 8 ? c : c < 4u ? 2u * c : 2u * (c - 4u) + 1u);
    const float v = __builtin_ldexpf(y[i], e);
    const _Float16 vh = (_Float16)v;
    hi[at] = vh;
    if (lo) lo[at] = (_Float16)(v - (float)vh);
  }
  return __builtin_ldexpf(1.0f, -e);
}

// Turns a row's sum_t p_t code Delta (the lane's group, y[8]) back and stores the row.
template <int BITS>
__device__ __forceinline__ void store_row(const AttendArgs& a, const Tables& K, const float* lam, const Seq& s, uint32_t h, uint32_t r, uint32_t l,
                                          const LaneInverse& f, float y[8], float sum) {
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;  // a row that sees nothing is 0
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] *= inv;
    if (K.scaled) y[i] *= lam[8 * l + i];
  }
  inverse_row(y, x, l, f);
  if (r >= (uint32_t)s.m * a.group) return;
  const uint32_t q = query_of(a, r);
  const uint64_t at = ((uint64_t)(s.q0 + q) * a.q_heads + h * a.group + r - q * a.group) * kD;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint64_t i = at + 2u * inverse_n(l, e);
    if (a.out_f32) *reinterpret_cast<float2*>(static_cast<float*>(a.out) + i) = make_float2(x[2 * e], x[2 * e + 1]);
    else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + i) = bf16_pair(x[2 * e], x[2 * e + 1]);
  }
}

__device__ __forceinline__ uint32_t uniform(uint32_t x) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)x); }

// The table's entry for token tt (-1 past `end`), the same in every lane; and the page it names (-1: absent).  Two
// steps, so that a loop can fetch an entry in one turn and first wait for it in the next: memory answers in
// order, and waiting at once would wait for the codes asked for before it.
__device__ __forceinline__ int32_t entry_of(const AttendArgs& a, uint32_t b, int32_t tt, int32_t end) {
  return tt < end ? a.table[(uint64_t)b * a.width + ((uint32_t)tt >> a.page_log2)] : -1;
}
__device__ __forceinline__ int32_t page_in(const AttendArgs& a, int32_t entry) {
  const int32_t p = __builtin_amdgcn_readfirstlane(entry);
  return (uint32_t)p < a.pages ? p : -1;
}
__device__ __forceinline__ int32_t page_of(const AttendArgs& a, uint32_t b, int32_t tt, int32_t end) { return page_in(a, entry_of(a, b, tt, end)); }

// ---- the host's side ---------------------------------------------------------------------------

// HQ_OK for sizes that the kernels can address.
inline int check_attend(const hq_kv_cache* cache, const hq_kv_attend_args* g) {
  if (int rc = check_cache(cache)) return rc;
  if (!g || g->q_heads == 0 || g->q_heads % cache->heads || g->q_heads > 65535u * 16u) return HQ_ERR_INVALID_ARG;
  // token indices and the ends of chunks and steps past them are 32-bit
  if (g->max_len > kMaxTokens || (uint64_t)g->table_width * cache->page > 0x7FFFFFFFull) return HQ_ERR_INVALID_ARG;
  if (g->total_q > (1ull << 31) || (uint64_t)g->max_q * (g->q_heads / cache->heads) > 0x7FFFFF00ull) return HQ_ERR_INVALID_ARG;
  if ((uint64_t)g->seqs * cache->heads > kMaxThreads / kAttBlock) return HQ_ERR_INVALID_ARG;
  if (!g->q_start && g->seqs && g->total_q % g->seqs) return HQ_ERR_INVALID_ARG;
  return HQ_OK;
}

// The other checks, and the arguments that do not depend on how a call is cut.  `nothing`: there is nothing to do, and pointers are
// not looked at.
inline int attend_args(const hq_kv_cache& c, const hq_kv_attend_args& g, AttendArgs* a, Tables* T, bool* nothing) {
  if ((g.q_dtype != HQ_F32 && g.q_dtype != HQ_BF16) || (g.out_dtype != HQ_F32 && g.out_dtype != HQ_BF16)) return HQ_ERR_INVALID_ARG;
  // log2(e) times the scale and the cap, and its reciprocal, are normal binary32 numbers (NaN fails too)
  if (!(std::fabs(g.scale) <= 0x1p126f)) return HQ_ERR_INVALID_ARG;
  if (g.softcap != 0.0f && !(g.softcap >= 0x1p-125f && g.softcap <= 0x1p125f)) return HQ_ERR_INVALID_ARG;
  if (g.weights && g.weights_stride < g.max_len) return HQ_ERR_INVALID_ARG;
  if (!make_tables(c, false, T)) return HQ_ERR_INVALID_ARG;
  *nothing = g.total_q == 0 || g.seqs == 0 || g.max_q == 0;
  if (*nothing) return HQ_OK;
  if (!g.q || !g.out || !g.lens || (g.max_len && g.table_width && !g.table)) return HQ_ERR_INVALID_ARG;
  const uint32_t size = g.q_dtype == HQ_F32 ? 4u : 2u;
  if (((uintptr_t)g.q & (size - 1u)) || ((uintptr_t)g.out & 15u)) return HQ_ERR_INVALID_ARG;
  if (((uintptr_t)g.lens | (uintptr_t)g.table | (uintptr_t)g.q_start | (uintptr_t)g.weights) & 3u) return HQ_ERR_INVALID_ARG;
  a->cache = static_cast<const uint8_t*>(c.data);
  a->q = g.q;
  a->out = g.out;
  a->q_start = g.q_start;
  a->table = g.table;
  a->lens = g.lens;
  a->weights = g.weights;
  a->wstride = g.weights_stride;
  a->total_q = g.total_q;
  a->qt = g.q_stride_token;
  a->qh = g.q_stride_head;
  a->heads = c.heads;
  a->group = g.q_heads / c.heads;
  uint32_t sh = 0;
  while ((1u << sh) < a->group) ++sh;
  a->group_mul = (uint32_t)((1ull << (31u + sh)) / a->group + 1u);
  a->group_shift = 31u + sh;
  a->q_heads = g.q_heads;
  a->pages = c.pages;
  a->page_log2 = 31u - (uint32_t)__builtin_clz(c.page);
  a->width = g.table_width;
  a->seqs = g.seqs;
  a->max_len = g.max_len;
  a->window = g.window;
  a->causal = g.causal != 0;
  a->q_f32 = g.q_dtype == HQ_F32;
  a->out_f32 = g.out_dtype == HQ_F32;
  a->vec = !((uintptr_t)g.q & 15u) && !((a->qt * (int64_t)size) % 16) && !((a->qh * (int64_t)size) % 16);
  const double log2e = 1.4426950408889634074;
  a->scale_log2 = (float)(g.scale * log2e);
  a->cap_in = g.softcap > 0.0f ? (float)(1.0 / (g.softcap * log2e)) : 0.0f;
  a->cap_out = (float)(g.softcap * log2e);
  return HQ_OK;
}

}  // namespace hq_kv
