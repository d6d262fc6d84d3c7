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
// Codes become binary16 in two steps: or-ing a code's offset bits into the mantissa of 128.0 (4 bits;
// 8.0 for 8) gives 128 + (c + 8) / 8 exactly, subtracting 129 gives c / 8 (c / 128), and the product
// with Delta is rounded once to binary16 (2^-11 of the value; it cannot overflow, |c / 8| < 1).
// Rows of Q are scaled by a power of two so that their largest coordinate lies in [2^14, 2^15).
// With accumulated weights asked for, scores are needed to binary32: Q and the keys go in two parts
// (hi = rounded product, lo = fma(code, Delta, -hi), exact down to 2^-25), three products instead of one.
// Scores, maxima, sums and outputs are binary32; P is binary16, scaled by 2^8 against a running
// reference at most 2^6 below the maximum (so P <= 2^14, and terms down to 2^-22 of it stay normal).
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/hq.h"
#include "hq_kv_device.h"
#include "hq_kv_internal.h"

namespace hq_kv {

constexpr int kAttBlock = 256;
constexpr int kAttWaves = 4;
constexpr float kPScaleLog2 = 8.0f;  // P is stored as p 2^8
constexpr float kSlack = 6.0f;       // the reference may lag the maximum by this much (log2)

struct AttendArgs {
  const uint8_t* cache;
  const void* q;
  void* out;
  const int32_t *q_start, *table, *lens;
  float* weights;
  uint64_t wstride, total_q;
  int64_t qt, qh;  // strides of q in values
  uint32_t heads, group, q_heads, pages, page_log2, width, seqs, max_q, max_len;
  uint32_t tiles, splits, chunk, window;
  int causal, q_f32, out_f32, vec;
  float scale_log2, cap_in, cap_out;  // scores in log2 units; s = cap_out tanh(cap_in s) when cap_in > 0
  // workspace
  _Float16 *qhi, *qlo;  // [seqs heads tiles][16][128]
  float* qf;            // [..][16] factor of a row's products
  float* po;            // [..][splits][16][128]
  float* pml;           // [..][splits][16][2]
  float* lse;           // [..][16]
};

struct Seq {
  int64_t q0;
  int32_t m, n;  // queries, cached tokens
};
__device__ __forceinline__ Seq seq_of(const AttendArgs& a, uint32_t b) {
  Seq s;
  if (a.q_start) {
    const int64_t x = a.q_start[b], y = a.q_start[b + 1], top = (int64_t)a.total_q;
    s.q0 = x < 0 ? 0 : x > top ? top : x;
    const int64_t e = y < s.q0 ? s.q0 : y > top ? top : y;
    s.m = (int32_t)(e - s.q0 < (int64_t)a.max_q ? e - s.q0 : (int64_t)a.max_q);
  } else {
    const int64_t per = (int64_t)(a.total_q / a.seqs);
    s.q0 = per * b;
    s.m = (int32_t)(per < (int64_t)a.max_q ? per : (int64_t)a.max_q);
  }
  const uint64_t held = (uint64_t)a.width << a.page_log2, most = held < a.max_len ? held : a.max_len;
  const int32_t n = a.lens[b];
  s.n = n < 0 ? 0 : (uint64_t)n < most ? n : (int32_t)most;
  return s;
}
// Visible tokens [lo, hi) of query i of a sequence.
__device__ __forceinline__ void visible(const AttendArgs& a, const Seq& s, int32_t i, int32_t* lo, int32_t* hi) {
  const int32_t pos = s.n - s.m + i;
  int32_t h = a.causal ? (pos + 1 < s.n ? pos + 1 : s.n) : s.n;
  if (h < 0) h = 0;
  int64_t l = a.window ? (int64_t)pos + 1 - (int64_t)a.window : 0;
  if (l < 0) l = 0;
  *lo = l > h ? h : (int32_t)l;
  *hi = h;
}
// Tokens a tile's rows see, as one range.
__device__ __forceinline__ void tile_range(const AttendArgs& a, const Seq& s, uint32_t tile, int32_t* lo, int32_t* hi) {
  const uint32_t rows = (uint32_t)s.m * a.group, r0 = tile * 16u;
  if (r0 >= rows) {
    *lo = *hi = 0;
    return;
  }
  const uint32_t r1 = r0 + 15u < rows ? r0 + 15u : rows - 1u;
  int32_t l0, h0, l1, h1;
  visible(a, s, (int32_t)(r0 / a.group), &l0, &h0);
  visible(a, s, (int32_t)(r1 / a.group), &l1, &h1);
  *lo = l0;
  *hi = h1;
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

constexpr float kUnit4 = 8.0f, kUnit8 = 128.0f;  // a dequantised value is code Delta / unit
template <int BITS>
constexpr float unit() { return BITS == 4 ? kUnit4 : kUnit8; }

struct U32x4 {
  uint32_t v[4];
};
__device__ __forceinline__ f16x8 frag(const U32x4& u) { return __builtin_bit_cast(f16x8, u); }

// 8 codes (one group of one token) -> 4 registers of value pairs code / unit, exact.  Pair order:
// 4 bits (c_i, c_{i+4}), 8 bits (c_2i, c_2i+1).
template <int BITS>
__device__ __forceinline__ void code_pairs(const uint32_t* w, f16x2 out[4]) {
  if (BITS == 4) {
    const uint32_t u = w[0] ^ 0x88888888u;
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = h2(((u >> (4 * i)) & 0x000F000Fu) | 0x58005800u) - (f16x2){(_Float16)129.0f, (_Float16)129.0f};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = w[i >> 1] ^ 0x80808080u;
      // bytes: code, 0x48, code, 0x48
      const uint32_t p = __builtin_amdgcn_perm(u, 0x48484848u, (i & 1) ? 0x00070006u : 0x00050004u);
      out[i] = h2(p) - (f16x2){(_Float16)9.0f, (_Float16)9.0f};
    }
  }
}

// The same for tokens a and b: out[i] = (code_i of a, code_i of b) / unit, i = 0..7.
template <int BITS>
__device__ __forceinline__ void token_pairs(const uint32_t* a, const uint32_t* b, f16x2 out[8]) {
  if (BITS == 4) {
    const uint32_t lo = __builtin_amdgcn_perm(b[0], a[0], 0x05040100u) ^ 0x88888888u;  // codes 0..3 of a, of b
    const uint32_t hi = __builtin_amdgcn_perm(b[0], a[0], 0x07060302u) ^ 0x88888888u;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      out[i] = h2((((i < 4 ? lo : hi) >> (4 * (i & 3))) & 0x000F000Fu) | 0x58005800u) - (f16x2){(_Float16)129.0f, (_Float16)129.0f};
  } else {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint32_t p = __builtin_amdgcn_perm(b[w], a[w], 0x05010400u) ^ 0x80808080u;  // a0 b0 a1 b1
      const uint32_t q = __builtin_amdgcn_perm(b[w], a[w], 0x07030602u) ^ 0x80808080u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t r = __builtin_amdgcn_perm(i < 2 ? p : q, 0x48484848u, (i & 1) ? 0x00070006u : 0x00050004u);
        out[4 * w + i] = h2(r) - (f16x2){(_Float16)9.0f, (_Float16)9.0f};
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

// Raw products of 16 tokens with the tile's rows: lane (n, b) gets row n, tokens 4b..4b+3.
template <int BITS, bool PREC>
__device__ __forceinline__ f32x4 scores16(const Share<BITS>& s, const f16x8 qh[4], const f16x8 ql[4]) {
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f16x2 c[4];
    code_pairs<BITS>(s.k + j * (BITS / 4), c);
    const uint32_t sc = s.ks[j >> 1];
    const _Float16 d = (j & 1) ? h2(sc)[1] : h2(sc)[0];
    const f16x2 dd = {d, d};
    U32x4 hi, lo;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f16x2 p = c[i] * dd;
      hi.v[i] = u2(p);
      if (PREC) lo.v[i] = u2(__builtin_elementwise_fma(c[i], dd, -p));
    }
    if (PREC) {
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(frag(lo), qh[j], acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(frag(hi), ql[j], acc, 0, 0, 0);
    }
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(frag(hi), qh[j], acc, 0, 0, 0);
  }
  return acc;
}

// tanh from the exponential: 1 - 2 / (e^2x + 1) away from zero, the odd series below 2^-3 in magnitude
// (next term 17 x^7 / 315 < 3 10^-8 x), so that small scores keep their relative precision.
__device__ __forceinline__ float tanh32(float x) {
  const float a = fabsf(x), x2 = x * x;
  const float e = __builtin_amdgcn_exp2f(fminf(a, 20.0f) * 2.885390081777927f);
  const float big = 1.0f - 2.0f / (e + 1.0f);
  const float small = __builtin_fmaf(x2, __builtin_fmaf(x2, __builtin_fmaf(x2, -17.0f / 315.0f, 2.0f / 15.0f), -1.0f / 3.0f), 1.0f) * a;
  return __builtin_copysignf(a < 0.125f ? small : big, x);
}

__device__ __forceinline__ float capped(const AttendArgs& a, float s) { return a.cap_in > 0.0f ? a.cap_out * tanh32(s * a.cap_in) : s; }

// ---------------------------------------------------------------------------------------------
// The queries' rows, transformed: two binary16 parts and a factor each, in the operand's order.
template <int BITS>
__global__ __launch_bounds__(kAttBlock) void rotate_rows_kernel(AttendArgs a, Tables K) {
  const uint32_t lane = threadIdx.x & 63u, l = lane & 15u;
  const uint64_t rowid = (uint64_t)blockIdx.x * (kAttBlock / 16) + (threadIdx.x >> 4);  // item * 16 + row
  const uint64_t item = rowid >> 4;
  if (item >= (uint64_t)a.seqs * a.heads * a.tiles) return;
  const uint32_t tile = (uint32_t)(item % a.tiles), h = (uint32_t)(item / a.tiles % a.heads), b = (uint32_t)(item / a.tiles / a.heads);
  const Seq s = seq_of(a, b);
  const uint32_t r = tile * 16u + (uint32_t)(rowid & 15u);
  const bool have = r < (uint32_t)s.m * a.group;
  if (tile * 16u >= (uint32_t)s.m * a.group) return;
  const LaneForward f = lane_forward(K, l);
  const uint32_t kappa = rev4(l);
  float m[8], x[8], y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[2 * i] = K.k[2 * (kappa + 16 * i)];
    m[2 * i + 1] = K.k[2 * (kappa + 16 * i) + 1];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = 0.0f;
  if (have) {
    const int64_t at = (s.q0 + r / a.group) * a.qt + (int64_t)(h * a.group + r % a.group) * a.qh + 8 * l;
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
  if (top > 0.0f && __builtin_isfinite(top)) e = 14 - (__builtin_amdgcn_frexp_expf(top) - 1);
  _Float16 *hi = a.qhi + rowid * kD, *lo = a.qlo + rowid * kD;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t g = (kappa >> 2) + 4u * (i >> 1), c = 2u * (kappa & 3u) + (i & 1);
    const uint32_t at = 8u * g + (BITS == 8 ? c : c < 4u ? 2u * c : 2u * (c - 4u) + 1u);
    const float v = __builtin_ldexpf(y[i], e);
    const _Float16 vh = (_Float16)v;
    hi[at] = vh;
    lo[at] = (_Float16)(v - (float)vh);
  }
  if (l == 0) a.qf[rowid] = __builtin_ldexpf(a.scale_log2 * unit<BITS>(), -e);
}

// ---------------------------------------------------------------------------------------------
// One (sequence, head, row tile, split): the wavefronts take 32 tokens in turn.
template <int BITS, bool PREC>
__global__ __launch_bounds__(kAttBlock) void attend_kernel(AttendArgs a) {
  __shared__ float s_o[16][kD + 4];
  __shared__ float s_m[kAttWaves][16], s_l[kAttWaves][16];
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6, n = lane & 15u, b4 = lane >> 4;
  const uint32_t split = blockIdx.x % a.splits;
  const uint64_t item = blockIdx.x / a.splits;
  const uint32_t tile = (uint32_t)(item % a.tiles), h = (uint32_t)(item / a.tiles % a.heads), b = (uint32_t)(item / a.tiles / a.heads);
  const Seq s = seq_of(a, b);
  int32_t lo, hi;
  tile_range(a, s, tile, &lo, &hi);
  int32_t t0 = (int32_t)(split * a.chunk), t1 = t0 + (int32_t)a.chunk;
  t0 = t0 > (lo & ~15) ? t0 : lo & ~15;
  t1 = t1 < hi ? t1 : hi;
  if (t0 >= t1) return;  // the same for the whole workgroup
  const uint32_t P = 1u << a.page_log2;
  const uint64_t page_size = (uint64_t)P * Page<BITS>::kToken;

  f16x8 qh[4], ql[4];
  {
    const uint64_t row = item * 16 + n;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      qh[j] = *reinterpret_cast<const f16x8*>(a.qhi + row * kD + 8 * (4 * b4 + j));
      if (PREC) ql[j] = *reinterpret_cast<const f16x8*>(a.qlo + row * kD + 8 * (4 * b4 + j));
    }
  }
  const float qf = a.qf[item * 16 + n];
  int32_t row_lo = 0, row_hi = 0;
  if (tile * 16u + n < (uint32_t)s.m * a.group) visible(a, s, (int32_t)((tile * 16u + n) / a.group), &row_lo, &row_hi);
  // the tokens every row of the tile sees: no masks there
  const bool whole_tile = tile * 16u + 15u < (uint32_t)s.m * a.group;
  int32_t all_lo = 0, all_hi = 0;
  if (whole_tile) {
    int32_t x;
    visible(a, s, (int32_t)((tile * 16u + 15u) / a.group), &all_lo, &x);
    visible(a, s, (int32_t)((tile * 16u) / a.group), &x, &all_hi);
  }

  float m = -1.0e30f, sum = 0.0f;
  f32x4 o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  for (int32_t t = t0 + 32 * (int32_t)wave; t < t1; t += 32 * kAttWaves) {
    Share<BITS> sh[2];
    bool there[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int32_t tt = t + 16 * u;
      int32_t page = -1;
      if (tt < t1) page = a.table[(uint64_t)b * a.width + ((uint32_t)tt >> a.page_log2)];
      page = __builtin_amdgcn_readfirstlane(page);
      there[u] = page >= 0 && (uint32_t)page < a.pages;
      if (there[u]) {
        const uint8_t* p = a.cache + ((uint64_t)page * a.heads + h) * page_size;
        load_keys<BITS>(p, P, (uint32_t)tt & (P - 1u), lane, sh[u]);
        load_values<BITS>(p, P, (uint32_t)tt & (P - 1u), lane, sh[u]);
      } else {
#pragma unroll
        for (int i = 0; i < BITS; ++i) sh[u].k[i] = sh[u].v[i] = 0u;
        sh[u].ks[0] = sh[u].ks[1] = sh[u].vs[0] = sh[u].vs[1] = 0u;
      }
    }
    float sc[8];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const f32x4 r = scores16<BITS, PREC>(sh[u], qh, ql);
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[4 * u + i] = capped(a, r[i] * qf);
    }
    const bool plain = there[0] && there[1] && t >= all_lo && t + 32 <= all_hi;
    if (!plain) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int32_t tok = t + 16 * (i >> 2) + 4 * (int32_t)b4 + (i & 3);
        if (!there[i >> 2] || tok < row_lo || tok >= row_hi || tok >= t1) sc[i] = -__builtin_inff();
        // a token that no row sees may hold anything
        if (!there[i >> 2] || tok < lo || tok >= t1) sh[i >> 2].vs[(i >> 1) & 1] &= (i & 1) ? 0x0000FFFFu : 0xFFFF0000u;
      }
    }
    // A value vector with NaN scales makes the rows that see it NaN, and no other (0 NaN in the product
    // would reach every row): its scale becomes 0 and its scores NaN.
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = sh[i >> 1].vs[i & 1];
      if ((w & 0x7C00u) == 0x7C00u || (w & 0x7C000000u) == 0x7C000000u) {
        if ((w & 0x7C00u) == 0x7C00u) {
          if (sc[2 * i] != -__builtin_inff()) sc[2 * i] = __builtin_nanf("");
          sh[i >> 1].vs[i & 1] &= 0xFFFF0000u;
        }
        if ((w & 0x7C000000u) == 0x7C000000u) {
          if (sc[2 * i + 1] != -__builtin_inff()) sc[2 * i + 1] = __builtin_nanf("");
          sh[i >> 1].vs[i & 1] &= 0x0000FFFFu;
        }
      }
    }
    float top = sc[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = fmaxf(top, sc[i]);
    if (__builtin_amdgcn_ballot_w64(top > m + kSlack)) {
      const float mn = fmaxf(m, blocks_max(top));
      const float f = __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      sum *= f;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] *= f;
    }
    U32x4 pf;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p0 = __builtin_amdgcn_exp2f(sc[2 * i] - m + kPScaleLog2), p1 = __builtin_amdgcn_exp2f(sc[2 * i + 1] - m + kPScaleLog2);
      sum += p0 + p1;
      pf.v[i] = u2((f16x2){(_Float16)p0, (_Float16)p1});
    }
    U32x4 vf[8];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        f16x2 c[8];
        token_pairs<BITS>(sh[u].v + (2 * w) * (BITS / 4), sh[u].v + (2 * w + 1) * (BITS / 4), c);
        const f16x2 d = h2(sh[u].vs[w]);
#pragma unroll
        for (int i = 0; i < 8; ++i) vf[i].v[2 * u + w] = u2(c[i] * d);
      }
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(frag(vf[i]), frag(pf), o[i], 0, 0, 0);
  }

  // the wavefronts' parts, joined in order
  sum = blocks_sum(sum);
  if (b4 == 0) {
    s_m[wave][n] = m;
    s_l[wave][n] = sum;
  }
  __syncthreads();
  float mm = s_m[0][n];
#pragma unroll
  for (int w = 1; w < kAttWaves; ++w) mm = fmaxf(mm, s_m[w][n]);
  const float f = __builtin_amdgcn_exp2f(m - mm);
  for (uint32_t w = 0; w < kAttWaves; ++w) {
    if (w == wave) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float& d = s_o[n][8 * (4 * b4 + r) + i];
          d = w ? d + o[i][r] * f : o[i][r] * f;
        }
    }
    __syncthreads();
  }
  const uint64_t part = item * a.splits + split;
  for (uint32_t i = threadIdx.x; i < 16u * kD / 4u; i += kAttBlock) {
    const uint32_t row = i >> 5, c = 4u * (i & 31u);
    *reinterpret_cast<f32x4*>(a.po + (part * 16 + row) * kD + c) = *reinterpret_cast<const f32x4*>(&s_o[row][c]);
  }
  if (threadIdx.x < 16) {
    float l = 0.0f;
    for (int w = 0; w < kAttWaves; ++w) l += s_l[w][n] * __builtin_amdgcn_exp2f(s_m[w][n] - mm);
    a.pml[(part * 16 + n) * 2] = mm;
    a.pml[(part * 16 + n) * 2 + 1] = l;
  }
}

// Joins a row's splits, turns it back and stores it: 16 lanes a row.
template <int BITS>
__global__ __launch_bounds__(kAttBlock) void combine_kernel(AttendArgs a, Tables K) {
  const uint32_t l = threadIdx.x & 15u;
  const uint64_t rowid = (uint64_t)blockIdx.x * (kAttBlock / 16) + (threadIdx.x >> 4);
  const uint64_t item = rowid >> 4;
  if (item >= (uint64_t)a.seqs * a.heads * a.tiles) return;
  const uint32_t tile = (uint32_t)(item % a.tiles), h = (uint32_t)(item / a.tiles % a.heads), b = (uint32_t)(item / a.tiles / a.heads);
  const Seq s = seq_of(a, b);
  const uint32_t r = tile * 16u + (uint32_t)(rowid & 15u);
  if (tile * 16u >= (uint32_t)s.m * a.group) return;
  int32_t lo, hi;
  tile_range(a, s, tile, &lo, &hi);
  const uint32_t s0 = hi > lo ? (uint32_t)lo / a.chunk : 0u, s1 = hi > lo ? ((uint32_t)hi + a.chunk - 1u) / a.chunk : 0u;
  float m = -1.0e30f;
  for (uint32_t i = s0; i < s1; ++i) m = fmaxf(m, a.pml[((item * a.splits + i) * 16 + (rowid & 15u)) * 2]);
  float sum = 0.0f, y[8], x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = 0.0f;
  for (uint32_t i = s0; i < s1; ++i) {
    const uint64_t p = (item * a.splits + i) * 16 + (rowid & 15u);
    const float f = __builtin_amdgcn_exp2f(a.pml[p * 2] - m);
    sum += a.pml[p * 2 + 1] * f;
    const f32x4 u0 = *reinterpret_cast<const f32x4*>(a.po + p * kD + 8 * l), u1 = *reinterpret_cast<const f32x4*>(a.po + p * kD + 8 * l + 4);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      y[c] += u0[c] * f;
      y[4 + c] += u1[c] * f;
    }
  }
  if (l == 0) a.lse[rowid] = m + __builtin_amdgcn_logf(sum) - kPScaleLog2;
  const float inv = sum == 0.0f ? 0.0f : unit<BITS>() / sum;  // a row that sees nothing is 0
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = (y[i] * inv) * K.v[8 * l + i];
  const LaneInverse f = lane_inverse(K, l);
  inverse_row(y, x, l, f);
  if (r >= (uint32_t)s.m * a.group) return;
  const uint64_t at = ((uint64_t)(s.q0 + r / a.group) * a.q_heads + h * a.group + r % a.group) * kD;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint64_t i = at + 2u * inverse_n(l, e);
    if (a.out_f32) *reinterpret_cast<float2*>(static_cast<float*>(a.out) + i) = make_float2(x[2 * e], x[2 * e + 1]);
    else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + i) = bf16_pair(x[2 * e], x[2 * e + 1]);
  }
}

// Accumulated weights: a wavefront owns 32 tokens of a (sequence, head), forms their scores with every
// row again and adds the sum of exp(s - lse) over the rows, in a fixed order.
template <int BITS>
__global__ __launch_bounds__(kAttBlock) void weights_kernel(AttendArgs a, uint32_t blocks) {
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6, n = lane & 15u, b4 = lane >> 4;
  const uint32_t bh = blockIdx.x / blocks, h = bh % a.heads, b = bh / a.heads;
  const Seq s = seq_of(a, b);
  const int32_t t = (int32_t)((blockIdx.x % blocks) * 32u * kAttWaves + 32u * wave);
  if (t >= s.n) return;
  const uint32_t P = 1u << a.page_log2;
  const uint64_t page_size = (uint64_t)P * Page<BITS>::kToken;
  Share<BITS> sh[2];
  bool there[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int32_t tt = t + 16 * u;
    int32_t page = -1;
    if (tt < s.n) page = a.table[(uint64_t)b * a.width + ((uint32_t)tt >> a.page_log2)];
    page = __builtin_amdgcn_readfirstlane(page);
    there[u] = page >= 0 && (uint32_t)page < a.pages;
    if (there[u]) {
      load_keys<BITS>(a.cache + ((uint64_t)page * a.heads + h) * page_size, P, (uint32_t)tt & (P - 1u), lane, sh[u]);
    } else {
#pragma unroll
      for (int i = 0; i < BITS; ++i) sh[u].k[i] = 0u;
      sh[u].ks[0] = sh[u].ks[1] = 0u;
    }
  }
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
  const uint32_t rows = (uint32_t)s.m * a.group;
  for (uint32_t tile = 0; tile * 16u < rows; ++tile) {
    int32_t lo, hi;
    tile_range(a, s, tile, &lo, &hi);
    if (t >= hi || t + 32 <= lo) continue;
    const uint64_t item = ((uint64_t)b * a.heads + h) * a.tiles + tile, row = item * 16 + n;
    f16x8 qh[4], ql[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      qh[j] = *reinterpret_cast<const f16x8*>(a.qhi + row * kD + 8 * (4 * b4 + j));
      ql[j] = *reinterpret_cast<const f16x8*>(a.qlo + row * kD + 8 * (4 * b4 + j));
    }
    const float qf = a.qf[row], lse = a.lse[row];
    int32_t row_lo = 0, row_hi = 0;
    if (tile * 16u + n < rows) visible(a, s, (int32_t)((tile * 16u + n) / a.group), &row_lo, &row_hi);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const f32x4 r = scores16<BITS, true>(sh[u], qh, ql);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int32_t tok = t + 16 * u + 4 * (int32_t)b4 + i;
        const float p = __builtin_amdgcn_exp2f(capped(a, r[i] * qf) - lse);
        acc[4 * u + i] += there[u] && tok >= row_lo && tok < row_hi ? p : 0.0f;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float x = acc[i];
    x += lane_xor<1>(x);
    x += lane_xor<2>(x);
    x += lane_xor<4>(x);
    x += lane_xor<8>(x);
    const int32_t tok = t + 16 * (i >> 2) + 4 * (int32_t)b4 + (i & 3);
    if (n == 0 && tok < s.n) a.weights[((uint64_t)b * a.heads + h) * a.wstride + (uint32_t)tok] += x;
  }
}

}  // namespace hq_kv

using namespace hq_kv;

namespace {

uint64_t align256(uint64_t v) { return (v + 255u) & ~(uint64_t)255u; }

// How a call is cut: row tiles, splits of the longest sequence, and the workspace they take.
struct Plan {
  uint64_t items;
  uint32_t tiles, splits, chunk;
  uint64_t qhi, qlo, qf, po, pml, lse, bytes;
};

Plan plan_of(const hq_kv_cache& c, const hq_kv_attend_args& g) {
  Plan p;
  const uint32_t group = g.q_heads / c.heads;
  p.tiles = (uint32_t)(((uint64_t)g.max_q * group + 15) / 16);
  p.items = (uint64_t)g.seqs * c.heads * p.tiles;
  // enough workgroups for four a CU, no less than 256 tokens each
  const uint64_t want = 1024, most = (g.max_len + 255) / 256;
  uint64_t splits = p.items ? (want + p.items - 1) / p.items : 1;
  if (splits > most) splits = most;
  if (splits < 1) splits = 1;
  uint64_t chunk = (g.max_len + splits - 1) / splits;
  chunk = (chunk + 127) / 128 * 128;
  if (chunk == 0) chunk = 128;
  p.chunk = (uint32_t)chunk;
  p.splits = (uint32_t)((g.max_len + chunk - 1) / chunk);
  if (p.splits == 0) p.splits = 1;
  uint64_t at = 0;
  auto take = [&](uint64_t n) {
    const uint64_t here = at;
    at = align256(at + n);
    return here;
  };
  p.qhi = take(p.items * 16 * kD * 2);
  p.qlo = take(p.items * 16 * kD * 2);
  p.qf = take(p.items * 16 * 4);
  p.lse = take(p.items * 16 * 4);
  p.pml = take(p.items * p.splits * 16 * 8);
  p.po = take(p.items * p.splits * 16 * kD * 4);
  p.bytes = at;
  return p;
}

int check_attend(const hq_kv_cache* cache, const hq_kv_attend_args* g) {
  if (int rc = check_cache(cache)) return rc;
  if (!g || g->q_heads == 0 || g->q_heads % cache->heads || g->q_heads > 65535u * 16u) return HQ_ERR_INVALID_ARG;
  if (g->max_len > 0x7FFFFFFFu || (uint64_t)g->table_width * cache->page > 0x7FFFFFFFull) return HQ_ERR_INVALID_ARG;
  if (g->total_q > (1ull << 31) || (uint64_t)g->max_q * (g->q_heads / cache->heads) > 0x7FFFFFF0ull) return HQ_ERR_INVALID_ARG;
  if (!g->q_start && g->seqs && g->total_q % g->seqs) return HQ_ERR_INVALID_ARG;
  return HQ_OK;
}

}  // namespace

extern "C" {

int hq_kv_attend_workspace_size(const hq_kv_cache* cache, const hq_kv_attend_args* args, size_t* bytes) {
  if (!bytes) return HQ_ERR_INVALID_ARG;
  if (int rc = check_attend(cache, args)) return rc;
  *bytes = plan_of(*cache, *args).bytes;
  return HQ_OK;
}

int hq_kv_attend(const hq_kv_cache* cache, const hq_kv_attend_args* args, void* workspace, size_t workspace_bytes,
                 hq_stream_t stream) {
  if (int rc = check_attend(cache, args)) return rc;
  const hq_kv_attend_args& g = *args;
  if ((g.q_dtype != HQ_F32 && g.q_dtype != HQ_BF16) || (g.out_dtype != HQ_F32 && g.out_dtype != HQ_BF16)) return HQ_ERR_INVALID_ARG;
  if (!std::isfinite(g.scale) || !std::isfinite(g.softcap) || g.softcap < 0.0f) return HQ_ERR_INVALID_ARG;
  if (g.weights && g.weights_stride < g.max_len) return HQ_ERR_INVALID_ARG;
  Tables T;
  if (!make_tables(*cache, false, &T)) return HQ_ERR_INVALID_ARG;
  // forward multipliers of the queries: the orthogonal packing's factor times the keys' lambda
  for (int c = 0; c < kD; ++c) T.k[c] *= c < 2 ? (float)(1.0 / std::sqrt(128.0)) : 0.0625f;
  if (g.total_q == 0 || g.seqs == 0 || g.max_q == 0) return HQ_OK;
  if (!g.q || !g.out || !g.lens || (g.max_len && g.table_width && !g.table)) return HQ_ERR_INVALID_ARG;
  const uint32_t size = g.q_dtype == HQ_F32 ? 4u : 2u;
  if (((uintptr_t)g.q & (size - 1u)) || ((uintptr_t)g.out & 15u)) return HQ_ERR_INVALID_ARG;
  if (((uintptr_t)g.lens | (uintptr_t)g.table | (uintptr_t)g.q_start | (uintptr_t)g.weights) & 3u) return HQ_ERR_INVALID_ARG;
  const Plan p = plan_of(*cache, g);
  if (!workspace || ((uintptr_t)workspace & 255u) || workspace_bytes < p.bytes) return HQ_ERR_INVALID_ARG;
  if (p.items * p.splits > 0x7FFFFFFFull) return HQ_ERR_INVALID_ARG;
  AttendArgs a;
  a.cache = static_cast<const uint8_t*>(cache->data);
  a.q = g.q;
  a.out = g.out;
  a.q_start = g.q_start;
  a.table = g.table;
  a.lens = g.lens;
  a.weights = g.weights;
  a.wstride = g.weights_stride;
  a.total_q = g.total_q;
  a.qt = g.q_stride_token;
  a.qh = g.q_stride_head;
  a.heads = cache->heads;
  a.group = g.q_heads / cache->heads;
  a.q_heads = g.q_heads;
  a.pages = cache->pages;
  a.page_log2 = 31u - (uint32_t)__builtin_clz(cache->page);
  a.width = g.table_width;
  a.seqs = g.seqs;
  a.max_q = g.max_q;
  a.max_len = g.max_len;
  a.tiles = p.tiles;
  a.splits = p.splits;
  a.chunk = p.chunk;
  a.window = g.window;
  a.causal = g.causal != 0;
  a.q_f32 = g.q_dtype == HQ_F32;
  a.out_f32 = g.out_dtype == HQ_F32;
  a.vec = !((uintptr_t)g.q & 15u) && !((a.qt * (int64_t)size) % 16) && !((a.qh * (int64_t)size) % 16);
  const double log2e = 1.4426950408889634074;
  a.scale_log2 = (float)(g.scale * log2e);
  a.cap_in = g.softcap > 0.0f ? (float)(1.0 / (g.softcap * log2e)) : 0.0f;
  a.cap_out = (float)(g.softcap * log2e);
  char* w = static_cast<char*>(workspace);
  a.qhi = reinterpret_cast<_Float16*>(w + p.qhi);
  a.qlo = reinterpret_cast<_Float16*>(w + p.qlo);
  a.qf = reinterpret_cast<float*>(w + p.qf);
  a.lse = reinterpret_cast<float*>(w + p.lse);
  a.pml = reinterpret_cast<float*>(w + p.pml);
  a.po = reinterpret_cast<float*>(w + p.po);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const dim3 rows((uint32_t)p.items), grid((uint32_t)(p.items * p.splits)), block(kAttBlock);
  const bool prec = g.weights != nullptr;
  if (cache->bits == 4) hipLaunchKernelGGL(rotate_rows_kernel<4>, rows, block, 0, st, a, T);
  else hipLaunchKernelGGL(rotate_rows_kernel<8>, rows, block, 0, st, a, T);
  if (cache->bits == 4 && prec) hipLaunchKernelGGL((attend_kernel<4, true>), grid, block, 0, st, a);
  else if (cache->bits == 4) hipLaunchKernelGGL((attend_kernel<4, false>), grid, block, 0, st, a);
  else if (prec) hipLaunchKernelGGL((attend_kernel<8, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((attend_kernel<8, false>), grid, block, 0, st, a);
  if (cache->bits == 4) hipLaunchKernelGGL(combine_kernel<4>, rows, block, 0, st, a, T);
  else hipLaunchKernelGGL(combine_kernel<8>, rows, block, 0, st, a, T);
  if (prec && g.max_len) {
    const uint32_t blocks = (g.max_len + 32u * kAttWaves - 1) / (32u * kAttWaves);
    const uint64_t wg = (uint64_t)g.seqs * cache->heads * blocks;
    if (wg > 0x7FFFFFFFull) return HQ_ERR_INVALID_ARG;
    if (cache->bits == 4) hipLaunchKernelGGL(weights_kernel<4>, dim3((uint32_t)wg), block, 0, st, a, blocks);
    else hipLaunchKernelGGL(weights_kernel<8>, dim3((uint32_t)wg), block, 0, st, a, blocks);
  }
  return hipGetLastError() == hipSuccess ? HQ_OK : HQ_ERR_HIP;
}

}  // extern "C"
