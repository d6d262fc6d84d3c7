// hq_kv_internal.h -- host checks and tables shared by the paged cache's entry points.
#pragma once

#include <stdint.h>

#include "../../include/hq.h"
#include "hq_kv_device.h"

namespace hq_kv {

inline uint32_t page_bytes(const hq_kv_cache& c) { return c.page * 2u * (16u * (uint32_t)c.bits + 32u); }

// HQ_OK for a cache the kernels can address.  P a power of two (slots split by shift and mask) and at
// least 16 (a block of 16 tokens lies in one page).
inline int check_cache(const hq_kv_cache* c) {
  if (!c || (c->bits != 4 && c->bits != 8)) return HQ_ERR_INVALID_ARG;
  if (c->page < 16u || c->page > 4096u || (c->page & (c->page - 1u))) return HQ_ERR_INVALID_ARG;
  if (c->heads == 0 || c->heads > 65535u || c->pages > 0x7FFFFFFFu) return HQ_ERR_INVALID_ARG;
  if (c->pages && (!c->data || ((uintptr_t)c->data & 15u))) return HQ_ERR_INVALID_ARG;
  return HQ_OK;
}

inline bool multipliers(const float* lambda, bool encode, float out[kD]) {
  hq_srft::Consts K;
  if (!hq_srft::make_consts(lambda, &K)) return false;
  for (int i = 0; i < kD; ++i) out[i] = encode ? K.m[i] : K.lam[i];
  return true;
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

// False if a lambda is not finite and positive.
inline bool make_tables(const hq_kv_cache& c, bool encode, Tables* T) {
  const hq_srft::Consts& w = hq_srft::twiddles();
  memcpy(T->w64c, w.w64c, sizeof(T->w64c));
  memcpy(T->w64s, w.w64s, sizeof(T->w64s));
  memcpy(T->w128c, w.w128c, sizeof(T->w128c));
  memcpy(T->w128s, w.w128s, sizeof(T->w128s));
  sign_words(c.seed, T->sign);
  return multipliers(c.lambda_k, encode, T->k) && multipliers(c.lambda_v, encode, T->v);
}

}  // namespace hq_kv
