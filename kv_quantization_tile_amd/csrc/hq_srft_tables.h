// hq_srft_tables.h -- constant tables of the SRFT transform (host), shared by the flat codec
// (hq_srft.hip) and the paged cache (hq_kv.hip, hq_attend.hip).
//
// Twiddles are binary32 roundings of binary64 cos and sin over the first octant, the rest of the
// circle by exact symmetry; they travel in the kernel argument with the multipliers.
#pragma once

#include <cmath>
#include <cstdint>
#include <cstring>

namespace hq_srft {

constexpr int kD = 128;        // values per vector
constexpr int kN = 64;         // complex FFT length
constexpr int kGroups = 16;    // scale groups per vector

struct Consts {
  float w64c[32], w64s[32];    // cos, sin of 2 pi k / 64
  float w128c[64], w128s[64];  // cos, sin of 2 pi k / 128
  float m[kD];                 // encode multipliers sigma_c / lambda_c
  float lam[kD];               // decode multipliers lambda_c
};

static inline void twiddle(uint32_t n, uint32_t k, float* c, float* s) {
  const double two_pi = 6.283185307179586476925286766559;
  const uint32_t quarter = n / 4, quad = (k % n) / quarter, r = (k % n) % quarter;
  float c0, s0;
  if (2 * r <= quarter) {
    c0 = (float)std::cos(two_pi * (double)r / (double)n);
    s0 = (float)std::sin(two_pi * (double)r / (double)n);
  } else {
    c0 = (float)std::sin(two_pi * (double)(quarter - r) / (double)n);
    s0 = (float)std::cos(two_pi * (double)(quarter - r) / (double)n);
  }
  switch (quad) {
    case 0: *c = c0; *s = s0; break;
    case 1: *c = 0.0f - s0; *s = c0; break;
    case 2: *c = 0.0f - c0; *s = 0.0f - s0; break;
    default: *c = s0; *s = 0.0f - c0; break;
  }
}

// The twiddles, computed at the first call (the 192 cos and sin take longer than a small launch).
inline const Consts& twiddles() {
  static const Consts T = [] {
    Consts t{};
    for (uint32_t k = 0; k < 32; ++k) twiddle(64, k, &t.w64c[k], &t.w64s[k]);
    for (uint32_t k = 0; k < 64; ++k) twiddle(128, k, &t.w128c[k], &t.w128s[k]);
    return t;
  }();
  return T;
}

// Fills the tables; false if a lambda is not finite and positive.
static inline bool make_consts(const float* lambda, Consts* K) {
  *K = twiddles();
  const float s0 = (float)(1.0 / std::sqrt(128.0));
  for (int c = 0; c < kD; ++c) {
    const float l = lambda ? lambda[c] : 1.0f;
    if (!(l > 0.0f) || !std::isfinite(l)) return false;
    const volatile float r = 1.0f / l;  // binary32 quotient, then one rounded product
    K->m[c] = (c < 2 ? s0 : 0.0625f) * r;
    K->lam[c] = l;
  }
  return true;
}

}  // namespace hq_srft
