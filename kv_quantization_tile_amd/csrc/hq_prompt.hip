// hq_prompt.hip -- softmax attention within packed prompts, on bf16 queries, keys and values.
//
//   o_i = sum_t p_it v_t,  p_it = exp(s_it - m_i) / sum_u exp(s_iu - m_i),  s_it = scale q_i.k_t (capped)
//
// in one pass over the keys: a running reference m (at most 2^6 below the running maximum, in powers of two), the
// running sum, and the output in registers.
//
// A row is one (query, head of the KV head's group), so that a tile of rows spans few queries and the causal
// mask wastes little.  A wavefront owns 32 rows; S^t = K Q^t on v_mfma_f32_32x32x16_bf16 leaves lane (n, h)
// (n = lane mod 32, h = lane / 32) the scores of row n for tokens 8 i + 4 h + 0..3 of 32: register for
// register the operand P^t of O^t = V^t P^t, if V^t is read for the same order of tokens.  K and V lie in LDS as they
// lie in memory, a token a row of 256 bytes; V^t comes out of it by transposing reads (four tokens of 16 columns to
// 16 lanes).  A row's 16-byte pieces are permuted so that a read meets every bank once: K's by the token modulo 16
// (a read takes one piece of 16 tokens), V's by the token modulo 4 (a read takes four pieces of four tokens): no bank
// conflict was counted.
//
// A workgroup has four wavefronts, 128 rows, and takes 64 tokens a step, the next ones on their way into the other half of its
// 64 KB; two workgroups share a CU, so that one's softmax, starts and ends run beside the other's products.  One workgroup of
// eight wavefronts kept all of them in one phase: 1 x 16384 tokens 2.15 ms against 2.06, 16 prompts of up to 2048 379 us against 343, one
// of 64 tokens 9.7 us against 7.2.  208 registers hold O (64), Q (32), two halves of scores (32), a step's keys (64, later
// its values) and weights (16); next step's scores under way as well took more than 256, and the spills cost all that it gave.
// One MI355X, 8 heads and 32 query heads: 16384 tokens 2.03 ms, 1080 TFLOP/s (a 16-bit product of 8192^3 reaches 1050 to 1165, and
// the clock falls to 1.8 GHz under either); matrix instructions are under way half of the cycles, LDS reads a quarter.
// Middling prompts lose to what a tile pays once (its place, Q, the first keys, the join of its halves, about 5 us of which the
// other workgroup hides a part) and to the masked step at its end: 16 of up to 2048 tokens, 345 to 369 us on several cards, 730 to 780
// TFLOP/s.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "../../include/hq.h"
#include "hq_kv_device.h"
#include "hq_kv_internal.h"

namespace hq_kv {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kPromptSlack = 6.0f;                 // the reference may lag the maximum by this much (log2)
constexpr float kPromptLowest = -3.402823466e38f;    // the reference before the first score
constexpr int kPromptTok = 64;                       // tokens of a step
constexpr int kPromptWaves = 4;                      // wavefronts of a workgroup, 32 rows each
constexpr uint32_t kPromptRows = 32u * kPromptWaves;
constexpr int64_t kPromptStride = 1 << 23;            // K's and V's rows are nearer than this, in values
constexpr uint32_t kPromptTile = kPromptTok * 256u;  // their bytes, K or V
constexpr uint32_t kPromptMany = 64;                 // tiles of more sequences than this go by place

struct PromptArgs {
  const uint16_t *q, *k, *v;
  void* out;
  const int32_t* start;
  int64_t qt, qh, kt, kh, vt, vh;
  uint64_t total;
  uint32_t heads, group, q_heads, seqs, window;
  uint32_t group_mul, group_shift;
  int by_place;  // workgroups take their tiles by place_of, not find_tile
  int causal, out_f32;
  uint32_t flip;  // of pairs of a query's values: their signs, for a scale below 0
  float scale_log2, cap_in, cap_out;
};

__device__ __forceinline__ uint32_t prompt_query(const PromptArgs& a, uint32_t r) { return (uint32_t)(((uint64_t)r * a.group_mul) >> a.group_shift); }

// Rows start[b] .. start[b + 1] - 1, cut to the rows there are.
__device__ __forceinline__ uint32_t prompt_rows(const PromptArgs& a, uint32_t b, uint32_t* first) {
  const int64_t x = a.start[b], y = a.start[b + 1], top = (int64_t)a.total;
  const int64_t s = x < 0 ? 0 : x > top ? top : x, e = y < s ? s : y > top ? top : y;
  *first = (uint32_t)s;
  return (uint32_t)(e - s);
}

// Sum over the wavefront: within 16 lanes by shifts, then the four ends.
template <int SHIFT>
__device__ __forceinline__ uint32_t add_shifted(uint32_t x) {
  return x + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x110 + SHIFT, 0xF, 0xF, true);  // row_shr, zeros from outside
}
__device__ __forceinline__ uint32_t wave_sum(uint32_t x) {
  x = add_shifted<8>(add_shifted<4>(add_shifted<2>(add_shifted<1>(x))));
  return (uint32_t)(__builtin_amdgcn_readlane((int)x, 15) + __builtin_amdgcn_readlane((int)x, 31) + __builtin_amdgcn_readlane((int)x, 47) +
                    __builtin_amdgcn_readlane((int)x, 63));
}

// The tile with the index-th most work, by the wavefront, of few sequences (each look walks all of them): tiles later in a sequence see more tokens, so of all
// sequences' tiles those of one place in their sequence form a level, the last levels first.  False if there are
// not so many tiles.  `tile`: its place in the sequence.
__device__ __forceinline__ bool find_tile(const PromptArgs& a, uint32_t index, uint32_t* seq, uint32_t* tile) {
  const uint32_t lane = threadIdx.x & 63u;
  auto tiles_of = [&](uint32_t b) {
    uint32_t first;
    return b < a.seqs ? (uint32_t)(((uint64_t)prompt_rows(a, b, &first) * a.group + kPromptRows - 1u) / kPromptRows) : 0u;
  };
  const uint32_t mine = tiles_of(lane);
  if (a.seqs == 1) {
    const uint32_t count = (uint32_t)__builtin_amdgcn_readfirstlane((int)mine);
    *seq = 0;
    *tile = count - 1u - index;
    return index < count;
  }
  // tiles at or past a level
  auto past = [&](uint32_t level) {
    uint32_t sum = mine > level ? mine - level : 0u;
    for (uint32_t b = 64u + lane; b < a.seqs; b += 64u) {
      const uint32_t n = tiles_of(b);
      sum += n > level ? n - level : 0u;
    }
    return wave_sum(sum);
  };
  if (past(0) <= index) return false;
  uint32_t lo = 0, hi = (uint32_t)((a.total * a.group + kPromptRows - 1u) / kPromptRows);  // past(lo) > index >= past(hi)
  while (hi - lo > 1u) {
    const uint32_t mid = lo + (hi - lo) / 2u;
    if (past(mid) > index) lo = mid;
    else hi = mid;
  }
  uint32_t skip = index - past(lo + 1u);
  for (uint32_t b0 = 0; b0 < a.seqs; b0 += 64u) {
    const uint32_t n = b0 ? tiles_of(b0 + lane) : mine;
    uint64_t votes = __builtin_amdgcn_ballot_w64(n > lo);
    const uint32_t here = (uint32_t)__builtin_popcountll(votes);
    if (skip < here) {
      for (; skip; --skip) votes &= votes - 1u;
      *seq = b0 + (uint32_t)__builtin_ctzll(votes);
      *tile = lo;
      return true;
    }
    skip -= here;
  }
  return false;
}

// The tile of the index-th place, by the wavefront, of many sequences.  A sequence of n rows from row s has places from
// floor(s / kPromptRows) + b on (rows of all the group's heads): as ceil(y) <= floor(x + y) - floor(x) + 1, they suffice and no two
// sequences share one.  The sequence is found among 64 offsets a look, and its last tile goes first.  False if the place has no tile.
__device__ __forceinline__ bool place_of(const PromptArgs& a, uint32_t index, uint32_t* seq, uint32_t* tile) {
  const uint32_t lane = threadIdx.x & 63u;
  uint32_t lo = 0, count = a.seqs, first;  // the last sequence that starts at or before `index` is one of `count` from lo on
  while (count > 1u) {
    const uint32_t stride = (count + 63u) / 64u, at = lane * stride;
    bool before = false;
    if (at < count) {
      prompt_rows(a, lo + at, &first);
      before = first * a.group / kPromptRows + lo + at <= index;
    }
    const uint64_t votes = __builtin_amdgcn_ballot_w64(before);
    const uint32_t k = votes ? 63u - (uint32_t)__builtin_clzll(votes) : 0u;
    lo += k * stride;
    count = count - k * stride < stride ? count - k * stride : stride;
  }
  const uint32_t tiles = (prompt_rows(a, lo, &first) * a.group + kPromptRows - 1u) / kPromptRows, place = index - (first * a.group / kPromptRows + lo);
  *seq = lo;
  *tile = tiles - 1u - place;
  return place < tiles;  // unsigned: not before the sequence's first place either
}

__device__ __forceinline__ uint32_t bf16_pack(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){lo, hi}, bf16x2));
}

// How scores are capped: not, by kCapPlain, by kCapExact.
enum { kCapNone = 0, kCapPlain = 1, kCapExact = 2 };
constexpr float kCapPlainMost = 256.0f;
// cap tanh(x) = cap - 2 cap / (e^2x + 1), of which the softmax does not see the constant: -1 / (e^2x + 1) is the score in units of
// 2 cap.  It is off by 2^-22, the capped score by 2^-21 of the cap: 2^-13 at kCapPlainMost, a 32nd of a bf16 weight's
// rounding.  Four operations where the exact form takes thirteen (2 x 4001 tokens, 28 heads, window 1024: 149 us, and 180 with the
// exact form).
__device__ __forceinline__ float cap_plain(float x2) { return __builtin_amdgcn_rcpf(-1.0f - __builtin_amdgcn_exp2f(x2)); }
// A larger cap needs small scores to their own precision: 1 - 2 / (e^2x + 1) away from zero (it saturates by itself), the
// odd series to x^5 below 2^-4 (the next term is below 2^-27 of x).
__device__ __forceinline__ float cap_exact(float x2) {
  const float x = x2 * 0.34657359027997264f, e = __builtin_amdgcn_exp2f(x2), x4 = x * x;
  const float big = __builtin_fmaf(-2.0f, __builtin_amdgcn_rcpf(e + 1.0f), 1.0f);
  const float small = x * __builtin_fmaf(x4, __builtin_fmaf(x4, 2.0f / 15.0f, -1.0f / 3.0f), 1.0f);
  return fabsf(x) < 0.0625f ? small : big;
}

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }

typedef __attribute__((address_space(3))) uint8_t lds_u8;

// Classes of instructions that sched_group_barrier names.
constexpr int kSchedVector = 0x2, kSchedMatrix = 0x8, kSchedRead = 0x100, kSchedExp = 0x400;
// x is made here, and not moved to where it is used.
__device__ __forceinline__ void keep(const bf16x8& x) { asm volatile("" ::"v"(x)); }

template <int CAP>
__global__ __launch_bounds__(64 * kPromptWaves, 2) void prompt_kernel(PromptArgs a) {
  // arrays of their own: a read of one does not wait for loads into another
  __shared__ __align__(16) uint8_t s_k0[kPromptTile], s_k1[kPromptTile], s_v0[kPromptTile], s_v1[kPromptTile];
  const uint32_t lane = threadIdx.x & 63u, wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), n32 = lane & 31u, half = lane >> 5;
  const uint32_t head = blockIdx.x % a.heads;
  uint32_t b, place;
  if (a.by_place ? !place_of(a, blockIdx.x / a.heads, &b, &place) : !find_tile(a, blockIdx.x / a.heads, &b, &place)) return;
  uint32_t first;
  const uint32_t n = prompt_rows(a, b, &first), rows = n * a.group, r0 = place * kPromptRows, w0 = r0 + 32u * wave;
  // tokens from `lo` to `hi` that some of the tile's rows see, in steps; those that all of the wavefront's see
  const uint32_t last = rows - 1u;
  auto query = [&](uint32_t x) { return (int32_t)prompt_query(a, x < last ? x : last); };
  auto from = [&](int32_t i) {  // the first token that query i sees
    const int64_t x = (int64_t)i + 1 - (int64_t)a.window;
    return a.window && x > 0 ? (int32_t)x : 0;
  };
  const int32_t lo = from(query(r0)) & ~(kPromptTok - 1), hi = a.causal ? query(r0 + kPromptRows - 1u) + 1 : (int32_t)n;
  const int32_t all_lo = from(query(w0 + 31u)), all_hi = a.causal ? query(w0) + 1 : (int32_t)n;
  // those that all of the tile's rows see
  const int32_t some_lo = from(query(r0 + kPromptRows - 1u)), some_hi = a.causal ? query(r0) + 1 : (int32_t)n;
  const int32_t steps = (hi - lo + kPromptTok - 1) / kPromptTok;

  // global to LDS: 1024 bytes, four tokens, an instruction
  constexpr int kLoads = 16 / kPromptWaves;
  const uint16_t* kbase = a.k + (int64_t)first * a.kt + (int64_t)head * a.kh;
  const uint16_t* vbase = a.v + (int64_t)first * a.vt + (int64_t)head * a.vh;
  auto load = [&](const uint16_t* base, uint32_t stride, bool keys, int32_t step, uint8_t* lds) __attribute__((always_inline)) {
    const uint32_t t = (uint32_t)(lo + kPromptTok * step), most = n - 1u - t;  // past the sequence: its last token again, masked below
    const uint8_t* from = reinterpret_cast<const uint8_t*>(base + (uint64_t)t * stride);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint32_t row0 = 4u * (wave * kLoads + i), row = row0 + (lane >> 4), piece = (lane & 15u) ^ (keys ? row & 15u : (row & 3u) << 2);
      const uint32_t at = (row < most ? row : most) * (2u * stride) + 16u * piece;  // below 2^31
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(from + at),
                                       (__attribute__((address_space(3))) void*)(lds + row0 * 256u), 16, 0, 0);
    }
  };
  auto load_k = [&](int32_t step, uint8_t* lds) __attribute__((always_inline)) { load(kbase, (uint32_t)a.kt, true, step, lds); };
  auto load_v = [&](int32_t step, uint8_t* lds) __attribute__((always_inline)) { load(vbase, (uint32_t)a.vt, false, step, lds); };
  load_k(0, s_k0);
  load_v(0, s_v0);

  // this lane's row: piece 2 s + half of its query
  bf16x8 q[8];
  const uint32_t r = w0 + n32;
  const bool have = r < rows;
  const uint32_t qi = (uint32_t)query(r), qg = (have ? r : last) - qi * a.group;
  {
    const uint16_t* p = a.q + (int64_t)(first + qi) * a.qt + (int64_t)(head * a.group + qg) * a.qh + 8u * half;
#pragma unroll
    for (int s = 0; s < 8; ++s) q[s] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(p + 16 * s) ^ a.flip);
  }
  const int32_t row_hi = a.causal ? (int32_t)qi + 1 : (int32_t)n, row_lo = from((int32_t)qi);

  uint32_t ka[8], va[4];
#pragma unroll
  for (uint32_t s = 0; s < 8; ++s) ka[s] = n32 * 256u + (((2u * s + half) ^ (lane & 15u)) * 16u);
#pragma unroll
  for (uint32_t d = 0; d < 4; ++d) {
    const uint32_t i = lane & 15u, tok = 4u * half + (i >> 2), piece = (4u * d + 2u * ((lane >> 4) & 1u) + ((i & 3u) >> 1)) ^ ((i >> 2) << 2);
    va[d] = tok * 256u + piece * 16u + (i & 1u) * 8u;
  }

  float m = kPromptLowest, sum = 0.0f, bad = 0.0f;  // bad: NaN once a masked step has met a value that is not finite
  f32x16 o[4];
#pragma unroll
  for (int d = 0; d < 4; ++d) o[d] = (f32x16)0.0f;
  const float c = CAP == kCapNone ? a.scale_log2 : a.cap_out;

  // the keys of 32 tokens, half u of a step, as operands; their raw scores
  auto keys = [&](const uint8_t* kb, int u, bf16x8* k) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) k[j] = *reinterpret_cast<const bf16x8*>(kb + u * 8192 + ka[j]);
  };
  auto scores = [&](const bf16x8* k, f32x16& s) __attribute__((always_inline)) {
    s = (f32x16)0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s = mfma32(k[j], q[j], s);
  };
  auto value = [&](const uint8_t* vb, int d, int w) __attribute__((always_inline)) {
    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(lds_u8*)(vb + va[d] + w * 4096));
    const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(lds_u8*)(vb + va[d] + w * 4096 + 2048));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto cap = [&](f32x16& s) __attribute__((always_inline)) {
    if (CAP != kCapNone) {
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = CAP == kCapPlain ? cap_plain(s[i] * a.cap_in) : cap_exact(s[i] * a.cap_in);
    }
  };
  // takes the tokens that the row does not see, of 32 from t, out
  auto hide = [&](int32_t t, f32x16& s) __attribute__((always_inline)) {
    const int32_t a0 = row_lo - t - 4 * (int32_t)half, a1 = row_hi - t - 4 * (int32_t)half;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int tok = 8 * (i >> 2) + (i & 3);
      if (tok < a0 || tok >= a1) s[i] = -__builtin_inff();
    }
  };
  // a new reference, if a score is far above the present one; whether there is
  auto raise = [&](const f32x16& s) __attribute__((always_inline)) {
    float top = s[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
    top *= c;
    const bool rise = __builtin_amdgcn_ballot_w64(top > m + kPromptSlack) != 0u;
    if (rise) {
      const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
      const float mn = fmaxf(m, fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]))), f = __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      sum *= f;
#pragma unroll
      for (int d = 0; d < 4; ++d) o[d] *= f;
    }
    return rise;
  };
  auto weigh = [&](const f32x16& s, bf16x8* p) __attribute__((always_inline)) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      u32x4 x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = 8 * w + 2 * i;
        const uint32_t pair = bf16_pack(__builtin_amdgcn_exp2f(__builtin_fmaf(s[e], c, -m)), __builtin_amdgcn_exp2f(__builtin_fmaf(s[e + 1], c, -m)));
        // the sum of the rounded weights, those that the output is made with
        sum = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, pair), __builtin_bit_cast(bf16x2, 0x3F803F80u), sum, false);
        x[i] = pair;
      }
      p[w] = __builtin_bit_cast(bf16x8, x);
    }
  };
  auto products = [&](const uint8_t* vb, int u, const bf16x8* p) __attribute__((always_inline)) {
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int d = 0; d < 4; ++d) o[d] = mfma32(value(vb, d, 2 * u + w), p[w], o[d]);
  };

  auto arrived = [&]() __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): the loads into LDS have landed
    __syncthreads();
  };
  // A step's two halves: one's weights are made among the other's products.
  auto step = [&](auto parity, int32_t j) __attribute__((always_inline)) {
    constexpr bool odd = decltype(parity)::value;
    const uint8_t *kb = odd ? s_k1 : s_k0, *vb = odd ? s_v1 : s_v0;
    arrived();
    if (j + 1 < steps) {
      load_k(j + 1, odd ? s_k0 : s_k1);
      load_v(j + 1, odd ? s_v0 : s_v1);
    }
    const int32_t t = lo + kPromptTok * j;
    const bool masked = t < all_lo || t + kPromptTok > all_hi;
    f32x16 s0, s1;
    bf16x8 k0[8], k1[8], p0[2], p1[2];
    keys(kb, 0, k0);
    keys(kb, 1, k1);
    __builtin_amdgcn_s_setprio(1);  // its products before the other workgroup's vector work (4096 tokens: 141 us against 149)
    scores(k0, s0);
    __builtin_amdgcn_s_setprio(0);
    cap(s0);
    if (masked) hide(t, s0);
    raise(s0);
    scores(k1, s1);
    const float before = sum;
    weigh(s0, p0);
    keep(p0[0]);
    keep(p0[1]);
    cap(s1);
    if (masked) hide(t + 32, s1);
    {
      const float with = sum;
      sum = before;
      if (raise(s1)) weigh(s0, p0);  // the first half's weights, not used yet, follow
      else sum = with;
    }
    __builtin_amdgcn_s_setprio(1);
    products(vb, 0, p0);
    weigh(s1, p1);
    keep(p1[0]);
    keep(p1[1]);
    products(vb, 1, p1);
    // the order of these: reads four products ahead, and an eighth of the second half's weights beside each of the first's products
    __builtin_amdgcn_sched_group_barrier(kSchedRead, 8, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedMatrix, 1, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedRead, 2, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedVector, 4, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedExp, 2, 0);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedMatrix, 1, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedRead, 2, 0);
    }
    __builtin_amdgcn_s_setprio(0);
    if (t < some_lo || t + kPromptTok > some_hi) {
      // 0 times a value that is not finite reaches rows that do not see it: such a tile is done again, below.  Each wavefront looks at
      // its share of the step's values.
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(vb + (64u * (wave * kLoads + i) + lane) * 16u);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t y = x[e];
          bad = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, y), __builtin_bit_cast(bf16x2, 0u), bad, false);
        }
      }
    }
  };

  __shared__ int s_again;
  if (threadIdx.x == 0) s_again = 0;
  for (int32_t j = 0; j < steps; j += 2) {
    step(std::false_type{}, j);
    if (j + 1 < steps) step(std::true_type{}, j + 1);
  }

  // Again, where a step that hides tokens has values that are not finite: they count as 0 in the products, and are added
  // to the rows that see them.
  if (__builtin_amdgcn_ballot_w64(bad != 0.0f)) s_again = 1;
  __syncthreads();
  if (s_again) {
    m = kPromptLowest;
    sum = 0.0f;
#pragma unroll
    for (int d = 0; d < 4; ++d) o[d] = (f32x16)0.0f;
#pragma unroll 1
    for (int32_t j = 0; j < steps; ++j) {
      const int32_t t = lo + kPromptTok * j;
      __syncthreads();
      load_k(j, s_k0);
      load_v(j, s_v0);
      arrived();
      bf16x8 p[4];
      f32x16 s[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        bf16x8 k[8];
        keys(s_k0, u, k);
        scores(k, s[u]);
        cap(s[u]);
        hide(t + 32 * u, s[u]);
        raise(s[u]);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) weigh(s[u], p + 2 * u);
#pragma unroll
      for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          u32x4 x = __builtin_bit_cast(u32x4, value(s_v0, d, w));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t y = x[i];
            x[i] = ((y & 0x7F80u) == 0x7F80u ? 0u : y & 0xFFFFu) | ((y & 0x7F800000u) == 0x7F800000u ? 0u : y & 0xFFFF0000u);
          }
          o[d] = mfma32(__builtin_bit_cast(bf16x8, x), p[w], o[d]);
        }
#pragma unroll 1
      for (int32_t tok = 0; tok < kPromptTok; ++tok) {
        const bool sees = t + tok >= row_lo && t + tok < row_hi;
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // columns 32 d + 8 e + 4 half + 0..3
            const uint32_t piece = (uint32_t)(4 * d + e) ^ (((uint32_t)tok & 3u) << 2);
            const uint2 x = *reinterpret_cast<const uint2*>(s_v0 + (uint32_t)tok * 256u + piece * 16u + half * 8u);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t y = i & 1 ? (i & 2 ? x.y : x.x) & 0xFFFF0000u : (i & 2 ? x.y : x.x) << 16;
              if (sees && (y & 0x7F800000u) == 0x7F800000u) o[d][4 * e + i] += __uint_as_float(y);
            }
          }
      }
    }
  }

  const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(sum), __float_as_uint(sum), false, false);
  const float total = __uint_as_float(x[0]) + __uint_as_float(x[1]), inv = total == 0.0f ? 0.0f : 1.0f / total;
  const uint64_t at = ((uint64_t)(first + qi) * a.q_heads + head * a.group + qg) * kD;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    o[d] *= inv;
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      // lane h has columns 8 j + 4 h + 0..3 and 8 more: half 0 takes columns 8 j .. 8 j + 7, half 1 the next eight
      if (a.out_f32) {
        if (have) {
          float* p = static_cast<float*>(a.out) + at + 32 * d + 8 * j + 4 * half;
          *reinterpret_cast<f32x4*>(p) = (f32x4){o[d][4 * j], o[d][4 * j + 1], o[d][4 * j + 2], o[d][4 * j + 3]};
          *reinterpret_cast<f32x4*>(p + 8) = (f32x4){o[d][4 * j + 4], o[d][4 * j + 5], o[d][4 * j + 6], o[d][4 * j + 7]};
        }
      } else {
        const auto y0 = __builtin_amdgcn_permlane32_swap(bf16_pack(o[d][4 * j], o[d][4 * j + 1]), bf16_pack(o[d][4 * j + 4], o[d][4 * j + 5]), false, false);
        const auto y1 = __builtin_amdgcn_permlane32_swap(bf16_pack(o[d][4 * j + 2], o[d][4 * j + 3]), bf16_pack(o[d][4 * j + 6], o[d][4 * j + 7]), false, false);
        if (have) *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.out) + at + 32 * d + 8 * j + 8 * half) = (u32x4){y0[0], y1[0], y0[1], y1[1]};
      }
    }
  }
}

}  // namespace hq_kv

using namespace hq_kv;

extern "C" int hq_attend_prompt(const hq_attend_prompt_args* g, hq_stream_t stream) {
  if (!g || g->heads == 0 || g->q_heads == 0 || g->q_heads % g->heads || g->q_heads > 65535u) return HQ_ERR_INVALID_ARG;
  if (g->dtype != HQ_BF16 || (g->out_dtype != HQ_F32 && g->out_dtype != HQ_BF16)) return HQ_ERR_INVALID_ARG;
  if (g->rows > (1ull << 30) || g->rows * g->q_heads > (1ull << 28)) return HQ_ERR_INVALID_ARG;
  // an index of a sequence goes up to 127 past the last one (find_tile)
  if (g->seqs > 0x7FFFFFFFu) return HQ_ERR_INVALID_ARG;
  if (!(std::fabs(g->scale) <= 0x1p126f)) return HQ_ERR_INVALID_ARG;
  if (g->softcap != 0.0f && !(g->softcap >= 0x1p-125f && g->softcap <= 0x1p125f)) return HQ_ERR_INVALID_ARG;
  // a stride that leads nowhere, of one row or one head, may be any
  const bool many = g->rows > 1;
  const struct {
    int64_t qt, qh, kt, kh, vt, vh;
  } st = {many ? g->q_stride[0] : 0, g->q_heads > 1 ? g->q_stride[1] : 0, many ? g->k_stride[0] : 0,
          g->heads > 1 ? g->k_stride[1] : 0, many ? g->v_stride[0] : 0, g->heads > 1 ? g->v_stride[1] : 0};
  if ((st.qt | st.qh | st.kt | st.kh | st.vt | st.vh) & 7) return HQ_ERR_INVALID_ARG;
  // a step's 64 rows lie within 2^31 bytes of each other
  if (st.kt < 0 || st.kt >= kPromptStride || st.vt < 0 || st.vt >= kPromptStride) return HQ_ERR_INVALID_ARG;
  if (g->rows == 0 || g->seqs == 0) return HQ_OK;
  if (!g->q || !g->k || !g->v || !g->out || !g->start || ((uintptr_t)g->start & 3u)) return HQ_ERR_INVALID_ARG;
  if (((uintptr_t)g->q | (uintptr_t)g->k | (uintptr_t)g->v | (uintptr_t)g->out) & 15u) return HQ_ERR_INVALID_ARG;
  PromptArgs a;
  a.q = static_cast<const uint16_t*>(g->q);
  a.k = static_cast<const uint16_t*>(g->k);
  a.v = static_cast<const uint16_t*>(g->v);
  a.out = g->out;
  a.start = g->start;
  a.qt = st.qt;
  a.qh = st.qh;
  a.kt = st.kt;
  a.kh = st.kh;
  a.vt = st.vt;
  a.vh = st.vh;
  a.total = g->rows;
  a.heads = g->heads;
  a.group = g->q_heads / g->heads;
  a.q_heads = g->q_heads;
  a.seqs = g->seqs;
  a.window = g->window;
  uint32_t sh = 0;
  while ((1u << sh) < a.group) ++sh;
  a.group_mul = (uint32_t)((1ull << (31u + sh)) / a.group + 1u);
  a.group_shift = 31u + sh;
  a.causal = g->causal != 0;
  a.out_f32 = g->out_dtype == HQ_F32;
  a.flip = g->scale < 0.0f ? 0x80008000u : 0u;
  // Hidden scores are -inf, which a factor of 0 would make NaN: a scale of 0 is 2^-126, the same for scores up to 2^100.
  const double log2e = 1.4426950408889634074, scale = std::fmax(std::fabs((double)g->scale), 0x1p-126);
  a.scale_log2 = (float)(scale * log2e);
  const bool plain = g->softcap <= kCapPlainMost;
  a.cap_in = g->softcap > 0.0f ? (float)std::fmin(2.0 * log2e * scale / g->softcap, 0x1p126) : 0.0f;  // 2 x log2 e of a raw score
  a.cap_out = (float)(g->softcap * log2e * (plain ? 2.0 : 1.0));
  const uint64_t rows = g->rows * a.group, some = g->seqs < rows ? g->seqs : rows;  // sequences with tokens, at most
  const uint64_t tiles = (rows + (kPromptRows - 1u) * some) / kPromptRows, most = kMaxThreads / (64u * kPromptWaves);
  // Tiles by level or by place, us (8 heads, 4 query heads each): 64 prompts of 100 tokens 47 and 45, 65 51 and 41, 256 252 and 151, 1024
  // 2315 and 593, 4096 32100 and 2473; 4096 of 8 tokens 6424 and 389; 100 of up to 2048 1893 and 1495; one of 8192 among 64 of 50
  // 535 and 522, first or last.  A launch has no room for a place to each of 2^24 / heads sequences, mostly empty ones: they go by level.
  const uint64_t places = rows / kPromptRows + g->seqs;
  a.by_place = g->seqs > kPromptMany && places * a.heads <= most;
  const uint64_t grid = (a.by_place ? places : tiles) * a.heads;
  if (grid > most) return HQ_ERR_INVALID_ARG;
  const hipStream_t on = static_cast<hipStream_t>(stream);
  const dim3 blocks((uint32_t)grid), block(64 * kPromptWaves);
  if (g->softcap == 0.0f) hipLaunchKernelGGL((prompt_kernel<kCapNone>), blocks, block, 0, on, a);
  else if (plain) hipLaunchKernelGGL((prompt_kernel<kCapPlain>), blocks, block, 0, on, a);
  else hipLaunchKernelGGL((prompt_kernel<kCapExact>), blocks, block, 0, on, a);
  return hipGetLastError() == hipSuccess ? HQ_OK : HQ_ERR_HIP;
}
