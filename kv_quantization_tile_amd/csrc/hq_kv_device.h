// hq_kv_device.h -- the SRFT transform with 16 lanes a vector, and the page layout: what the paged
// cache's kernels (hq_kv.hip, hq_attend.hip) share.
//
// The transform is the flat codec's (hq_srft.hip): the same butterflies on the same values in the
// same order, each operation rounded once, so codes and decoded values are bit-identical to it.  There
// one thread holds a whole vector, which is the fewest instructions for hundreds of thousands of
// vectors; a cache also writes and reads a handful at a time, and attention needs the queries' rows
// spread over a wavefront, so here lane l of 16 holds the complex points 4l..4l+3.
//
// Six radix-2 passes; pass p combines points whose index differs in bit 5-p and leaves output bit p
// in its place.  Bits 5..2 are lane bits 3..0 (DPP exchanges), bits 1..0 a lane's registers.  The
// lane whose bit is set multiplies its point by the twiddle before the exchange, so every product
// is formed once: lower = own + other, upper = other - own.  The result of index k lies bit-reversed:
// lane l holds k = kappa + {0, 32, 16, 48} in registers 0..3, kappa = l with its 4 bits reversed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hq_device.h"

namespace hq_kv {

constexpr int kD = 128;

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// What a call's transform depends on: the sign diagonal's bits and, unless all ones, the multipliers of K's
// and V's coordinates.
struct Tables {
  uint32_t sign[4];
  int scaled;         // whether k and v hold anything but ones
  float k[kD], v[kD];
};

// The multipliers in LDS, when there are any: lanes pick their own, and vector loads from a kernel's arguments are
// slow enough (9 us over a launch of 16384 wavefronts) to be made once a workgroup of 256.
__device__ __forceinline__ void stage_tables(const Tables& K, float (*s)[kD]) {
  if (!K.scaled) return;
  s[threadIdx.x >> 7][threadIdx.x & 127u] = threadIdx.x < 128u ? K.k[threadIdx.x] : K.v[threadIdx.x - 128u];
  __syncthreads();
}

// cos and sin of 2 pi k / n, k < n / 2, rounded to binary32 from binary64 values in the first octant and
// continued by symmetry: the values of the flat codec's tables (hq_srft.hip), in device memory because a
// lane picks its own 20.  The octant's cos and sin are Taylor sums, whose remainder below 2^-60 no binary32
// rounding here sees.
struct Twiddles {
  float c64[32], s64[32], c128[64], s128[64];
};
constexpr double taylor(double x, bool sine) {
  double term = sine ? x : 1.0, sum = 0.0;
  for (int i = sine ? 1 : 0; i < 24; i += 2) {
    sum += term;
    term *= -x * x / ((i + 1.0) * (i + 2.0));
  }
  return sum;
}
constexpr void twiddle(int n, int k, float& c, float& s) {
  const double two_pi = 6.283185307179586476925286766559;
  const int quarter = n / 4, quad = k / quarter, r = k % quarter;
  const bool low = 2 * r <= quarter;
  const double a = two_pi * (low ? r : quarter - r) / n;
  const float c0 = (float)taylor(a, !low), s0 = (float)taylor(a, low);
  c = quad == 0 ? c0 : 0.0f - s0;
  s = quad == 0 ? s0 : c0;
}
constexpr Twiddles make_twiddles() {
  Twiddles t{};
  for (int k = 0; k < 32; ++k) twiddle(64, k, t.c64[k], t.s64[k]);
  for (int k = 0; k < 64; ++k) twiddle(128, k, t.c128[k], t.s128[k]);
  return t;
}
static __device__ const Twiddles kTwiddles = make_twiddles();

// ---- pages -----------------------------------------------------------------------------------
// A page of P tokens of one head: K codes [P][16][E], K scales [P][16], V codes [P/4][16][4][E],
// V scales [P/4][16][4], E = BITS bytes for a group's 8 codes.  K is read by token (its product runs
// over the coordinates), V by blocks of four tokens (its product runs over the tokens), so that in
// attention a lane's share of 16 tokens is one 16-byte (4 bits) run of each.
template <int BITS>
struct Page {
  static constexpr uint32_t kCode = 16u * BITS;        // bytes of one vector's codes
  static constexpr uint32_t kToken = 2u * (kCode + 32u);  // K and V, codes and scales
  __device__ __host__ static uint32_t k_code(uint32_t, uint32_t t) { return t * kCode; }
  __device__ __host__ static uint32_t k_scale(uint32_t P, uint32_t t) { return P * kCode + t * 32u; }
  __device__ __host__ static uint32_t v_code(uint32_t P, uint32_t t, uint32_t g) {
    return P * (kCode + 32u) + (((t >> 2) * 16u + g) * 4u + (t & 3u)) * (uint32_t)BITS;
  }
  __device__ __host__ static uint32_t v_scale(uint32_t P, uint32_t t, uint32_t g) {
    return P * (2u * kCode + 32u) + (((t >> 2) * 16u + g) * 4u + (t & 3u)) * 2u;
  }
};

// ---- exchanges within 16 lanes -----------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true));
}
template <int BIT>
__device__ __forceinline__ float lane_xor(float x) {
  if (BIT == 1) return dpp<0xB1>(x);         // quad_perm 1,0,3,2
  if (BIT == 2) return dpp<0x4E>(x);         // quad_perm 2,3,0,1
  if (BIT == 4) return dpp<0x1B>(dpp<0x141>(x));  // half-row mirror (^7), quad_perm 3,2,1,0 (^3)
  return dpp<0x128>(x);                      // row_ror 8
}
template <int BIT>
__device__ __forceinline__ uint32_t lane_xor_u(uint32_t x) {
  return __builtin_bit_cast(uint32_t, lane_xor<BIT>(__builtin_bit_cast(float, x)));
}

__device__ __forceinline__ uint32_t rev4(uint32_t l) {
  return ((l & 1u) << 3) | ((l & 2u) << 1) | ((l & 4u) >> 1) | ((l & 8u) >> 3);
}

// Value of x in lane `src` of the caller's 16 lanes (any lane pattern).
__device__ __forceinline__ float row_get(float x, uint32_t src) {
  const uint32_t lane = (threadIdx.x & 48u) | src;
  return __builtin_bit_cast(float, __builtin_amdgcn_ds_bpermute((int)(lane << 2), __builtin_bit_cast(int, x)));
}

// Value of x in lane `src` of the wavefront's first 16 lanes.
__device__ __forceinline__ float row_get_any(float x, uint32_t src) {
  return __builtin_bit_cast(float, __builtin_amdgcn_ds_bpermute((int)(src << 2), __builtin_bit_cast(int, x)));
}

// ---- the FFT -----------------------------------------------------------------------------------
// Twiddles of a lane's passes 1..5 (1 where the pass does not multiply the lane's points).
struct LaneTwiddles {
  float c[5], s[5];
};

template <bool INV>
__device__ __forceinline__ LaneTwiddles lane_twiddles(uint32_t l) {
  LaneTwiddles t;
  const uint32_t kappa = rev4(l);
  const uint32_t idx[5] = {(l & 4u) ? (kappa & 1u) * 16u : 0u, (l & 2u) ? (kappa & 3u) * 8u : 0u,
                           (l & 1u) ? (kappa & 7u) * 4u : 0u, kappa * 2u, kappa};
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    t.c[i] = kTwiddles.c64[idx[i]];
    t.s[i] = INV ? kTwiddles.s64[idx[i]] : -kTwiddles.s64[idx[i]];
  }
  return t;
}

template <int BIT, bool TWIDDLE>
__device__ __forceinline__ void fft_cross(float re[4], float im[4], uint32_t l, float c, float s) {
  const float sg = (l & BIT) ? -1.0f : 1.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float ar = re[e], ai = im[e];
    if (TWIDDLE) {
      const float tr = ar * c - ai * s, ti = ar * s + ai * c;
      ar = tr;
      ai = ti;
    }
    // fma by +-1 rounds once, as the sum or difference does
    re[e] = __builtin_fmaf(ar, sg, lane_xor<BIT>(ar));
    im[e] = __builtin_fmaf(ai, sg, lane_xor<BIT>(ai));
  }
}

__device__ __forceinline__ void butterfly(float& ar, float& ai, float& br, float& bi, float c, float s) {
  const float tr = br * c - bi * s, ti = br * s + bi * c, xr = ar, xi = ai;
  ar = xr + tr;
  ai = xi + ti;
  br = xr - tr;
  bi = xi - ti;
}

template <bool INV>
__device__ __forceinline__ void fft64_row(float re[4], float im[4], uint32_t l, const LaneTwiddles& t) {
  fft_cross<8, false>(re, im, l, 1.0f, 0.0f);
  fft_cross<4, true>(re, im, l, t.c[0], t.s[0]);
  fft_cross<2, true>(re, im, l, t.c[1], t.s[1]);
  fft_cross<1, true>(re, im, l, t.c[2], t.s[2]);
  butterfly(re[0], im[0], re[2], im[2], t.c[3], t.s[3]);
  butterfly(re[1], im[1], re[3], im[3], t.c[3], t.s[3]);
  butterfly(re[0], im[0], re[1], im[1], t.c[4], t.s[4]);
  // index kappa + 16 is kappa turned by a quarter, exact in the tables
  butterfly(re[2], im[2], re[3], im[3], INV ? -t.s[4] : t.s[4], INV ? t.c[4] : -t.c[4]);
}

// The forward transform of one vector per 16 lanes.  In: x[8], lane l's values 8l..8l+7.  Out: lane l
// holds coordinates 2k and 2k+1 of k = kappa + 16 r in y[2r], y[2r+1], times their multipliers m (of
// the same coordinates); so coordinates of group kappa / 4 + 4 r.
struct LaneForward {
  LaneTwiddles t;
  float c[4], e[4];  // W_128^k of the lane's four k
  uint32_t flip[4];  // sign bits of the lane's values, two a word (bits 31 and 15)
};
__device__ __forceinline__ uint32_t sign_word(const Tables& K, uint32_t i) {
  const uint32_t lo = (i & 1u) ? K.sign[1] : K.sign[0], hi = (i & 1u) ? K.sign[3] : K.sign[2];
  return (i & 2u) ? hi : lo;
}
// The orthogonal packing's factor of coordinate c.
__device__ __forceinline__ float packing(uint32_t c) { return c < 2u ? 0.08838834764831845f : 0.0625f; }

__device__ __forceinline__ LaneForward lane_forward(const Tables& K, uint32_t l) {
  LaneForward f;
  f.t = lane_twiddles<false>(l);
  const uint32_t kappa = rev4(l);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    f.c[r] = kTwiddles.c128[kappa + 16 * r];
    f.e[r] = -kTwiddles.s128[kappa + 16 * r];
    const uint32_t b = sign_word(K, l >> 2) >> ((8u * l + 2u * (uint32_t)r) & 31u);
    f.flip[r] = ((b & 1u) << 15) | ((b & 2u) << 30);
  }
  return f;
}

__device__ __forceinline__ void forward_row(const float x[8], float y[8], const float m[8], uint32_t l, const LaneForward& f) {
  float re[4], im[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    re[e] = __uint_as_float(__float_as_uint(x[2 * e]) ^ (f.flip[e] << 16));
    im[e] = __uint_as_float(__float_as_uint(x[2 * e + 1]) ^ (f.flip[e] & 0x80000000u));
  }
  fft64_row<false>(re, im, l, f.t);
  // natural order: registers of k = kappa + 16 r
  const float zr[4] = {re[0], re[2], re[1], re[3]}, zi[4] = {im[0], im[2], im[1], im[3]};
  const uint32_t kappa = rev4(l), mate = rev4((16u - kappa) & 15u);
  float pr[4], pi[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    pr[r] = row_get(zr[r], mate);
    pi[r] = row_get(zi[r], mate);
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    // Z_{64-k}: register 3 - r of the mate; of kappa = 0, which is its own mate, register (4 - r) mod 4
    const float mr = kappa ? pr[3 - r] : pr[(4 - r) & 3], mi = kappa ? pi[3 - r] : pi[(4 - r) & 3];
    const float er = zr[r] + mr, ei = zi[r] - mi, gr = zr[r] - mr, gi = zi[r] + mi;
    const float a = gi, b = -gr;
    const float ur = a * f.c[r] - b * f.e[r], ui = a * f.e[r] + b * f.c[r];
    y[2 * r] = (er + ur) * m[2 * r];
    y[2 * r + 1] = (ei + ui) * m[2 * r + 1];
  }
  if (kappa == 0) {  // X_0 and X_64
    y[0] = (zr[0] + zi[0]) * m[0];
    y[1] = (zr[0] - zi[0]) * m[1];
  }
}

// The inverse.  In: lane l holds y[8] = coordinates 8l..8l+7 (group l).  Out: x[2e], x[2e+1] = values 2n
// and 2n + 1 of n = inverse_n(l, e).
struct LaneInverse {
  LaneTwiddles t;
  float c[4], s[4];
  uint32_t flip[4];  // sign bits of the outputs, two a word
};
__device__ __forceinline__ uint32_t inverse_n(uint32_t l, int e) { return rev4(l) + (e == 0 ? 0u : e == 1 ? 32u : e == 2 ? 16u : 48u); }

__device__ __forceinline__ LaneInverse lane_inverse(const Tables& K, uint32_t l) {
  LaneInverse f;
  f.t = lane_twiddles<true>(l);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f.c[e] = kTwiddles.c128[4 * l + e];
    f.s[e] = kTwiddles.s128[4 * l + e];
    const uint32_t n = inverse_n(l, e), b = sign_word(K, n >> 4) >> ((2u * n) & 31u);
    f.flip[e] = ((b & 1u) << 15) | ((b & 2u) << 30);
  }
  return f;
}

__device__ __forceinline__ void inverse_row(const float y[8], float x[8], uint32_t l, const LaneInverse& f) {
  const float r2 = 1.41421353816986083984375f;  // binary32 sqrt(2)
  float re[4], im[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    // Y_{64-k}, k = 4 l + e: point 4 - e of lane 15 - l, and point 0 of lane 16 - l for e = 0
    const float mr = e ? dpp<0x140>(y[2 * ((4 - e) & 3)]) : row_get(y[0], (16u - l) & 15u);
    const float mi = e ? dpp<0x140>(y[2 * ((4 - e) & 3) + 1]) : row_get(y[1], (16u - l) & 15u);
    const float br = mr, bi = -mi;
    const float sr = y[2 * e] + br, si = y[2 * e + 1] + bi, dr = y[2 * e] - br, di = y[2 * e + 1] - bi;
    const float pr = dr * f.c[e] - di * f.s[e], pi = dr * f.s[e] + di * f.c[e];
    re[e] = sr - pi;
    im[e] = si + pr;
  }
  if (l == 0) {
    re[0] = (y[0] + y[1]) * r2;
    im[0] = (y[0] - y[1]) * r2;
  }
  fft64_row<true>(re, im, l, f.t);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(__float_as_uint(re[e] * 0.0625f) ^ (f.flip[e] << 16)) + 0.0f;
    x[2 * e + 1] = __uint_as_float(__float_as_uint(im[e] * 0.0625f) ^ (f.flip[e] & 0x80000000u)) + 0.0f;
  }
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {  // nearest even
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

}  // namespace hq_kv
