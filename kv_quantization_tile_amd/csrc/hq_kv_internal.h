// hq_kv_internal.h -- host checks and tables shared by the paged cache's entry points.
#pragma once

#include <stdint.h>

#include <cmath>

#include "../../include/hq.h"
#include "hq_kv_device.h"

namespace hq_kv {

constexpr uint64_t kMaxThreads = 0xFFFFFFFFull;  // of one launch
constexpr uint32_t kMaxTokens = 1u << 30;        // of one sequence

// HQ_OK for a cache the kernels can address.  P a power of two (slots split by shift and mask) and at
// least 16 (a block of 16 tokens lies in one page).
inline int check_cache(const hq_kv_cache* c) {
  if (!c || (c->bits != 4 && c->bits != 8)) return HQ_ERR_INVALID_ARG;
  if (c->page < 16u || c->page > 4096u || (c->page & (c->page - 1u))) return HQ_ERR_INVALID_ARG;
  if (c->heads == 0 || c->heads > 65535u || c->pages > 0x7FFFFFFFu) return HQ_ERR_INVALID_ARG;
  if (c->pages && (!c->data || ((uintptr_t)c->data & 15u))) return HQ_ERR_INVALID_ARG;
  return HQ_OK;
}

// The sign diagonal's 128 bits (Philox4x32-10, key = seed, counter 0), as the codecs draw them.
inline void sign_words(uint64_t seed, uint32_t w[4]) {
  uint32_t c[4] = {0, 0, 0, 0}, k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = (uint64_t)0xD2511F53u * c[0], p1 = (uint64_t)0xCD9E8D57u * c[2];
    const uint32_t n0 = (uint32_t)(p1 >> 32) ^ c[1] ^ k0, n2 = (uint32_t)(p0 >> 32) ^ c[3] ^ k1;
    c[0] = n0;
    c[1] = (uint32_t)p1;
    c[2] = n2;
    c[3] = (uint32_t)p0;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  for (int i = 0; i < 4; ++i) w[i] = c[i];
}

// False if a lambda is not finite and positive.  Encoding multiplies by binary32 1 / lambda (then by the
// packing's factor, as hq_srft_encode does), decoding by lambda.
inline bool make_tables(const hq_kv_cache& c, bool encode, Tables* T) {
  sign_words(c.seed, T->sign);
  T->scaled = c.lambda_k || c.lambda_v;
  if (!T->scaled) return true;
  for (int i = 0; i < kD; ++i) {
    const float k = c.lambda_k ? c.lambda_k[i] : 1.0f, v = c.lambda_v ? c.lambda_v[i] : 1.0f;
    if (!(k > 0.0f) || !(v > 0.0f) || !std::isfinite(k) || !std::isfinite(v)) return false;
    const volatile float rk = 1.0f / k, rv = 1.0f / v;
    T->k[i] = encode ? rk : k;
    T->v[i] = encode ? rv : v;
  }
  return true;
}

// The paged cache's transforms a vector a thread, for many tokens (hq_srft.hip).
struct ManyAppend {
  uint8_t* cache;
  const void *k, *v;
  const int64_t* slots;
  uint64_t tokens;
  int64_t kt, kh, vt, vh;  // strides in values
  uint32_t heads, pages, page_log2;
  uint32_t sides, one;     // workgroups take K and V in turn (2), or the side `one` (1); set by the launch
};
struct ManyRead {
  const uint8_t* cache;
  const int64_t* slots;
  uint64_t tokens;
  void *k, *v;  // one may be null
  uint32_t heads, pages, page_log2;
  uint32_t sides, one;
};
void launch_append_many(const hq_kv_cache& c, const ManyAppend& a, int f32_in, hipStream_t st);
void launch_read_many(const hq_kv_cache& c, const ManyRead& a, int f32_out, hipStream_t st);

}  // namespace hq_kv
