// hq_kv.hip -- the paged SRFT cache: appending tokens, reading them back, and evicting tokens by
// accumulated attention weight.  (Attention over the cache: hq_attend.hip.)
//
// The cache holds the SRFT codec's codes and scales ("When quantization is free" technical summary,
// gist.science/ko/paper/2605.05699, section "Methodology": per-channel lambda, 16 groups with binary16
// scales, signed int4 or int8) in pages of P tokens of one KV head (hq_kv_device.h: Page).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/hq.h"
#include "hq_kv_device.h"
#include "hq_kv_internal.h"

namespace hq_kv {

constexpr int kBlock = 256;

// absmax / L and 1 / d as the flat codec forms them (hq_srft.hip), equal to the correctly rounded
// quotients.
template <int L>
__device__ __forceinline__ float div_l(float a) {
  constexpr float c = 1.0f / (float)L;
  const float q0 = a * c;
  return __builtin_fmaf(__builtin_fmaf(-q0, (float)L, a), c, q0);
}
__device__ __forceinline__ float recip_f16_value(float d) {
  const float y0 = __builtin_amdgcn_rcpf(d);
  return __builtin_fmaf(__builtin_fmaf(-d, y0, 1.0f), y0, y0);
}

struct AppendArgs {
  uint8_t* cache;
  const void *k, *v;
  const int64_t* slots;
  uint64_t tokens;
  int64_t kt, kh, vt, vh;  // strides in values
  uint32_t heads, pages, page_log2, quads;
  int f32, vec;
};

// One vector per 16 lanes; the four rows of a wavefront take four consecutive tokens of one head and
// side (K or V), so that the V pieces (4 bytes every 16) of neighbouring tokens meet in one line, and `quads`
// such fours in turn, so that the twiddles are fetched once for all of them.  Vector instructions bound it: 516 a four
// (32768 tokens of 8 heads: 105 to 120 us, 97 % of the issue rate).  Many tokens go to the kernels with a vector a
// thread, which need 64 vectors a wavefront; a decode step's 4 tokens of 8 heads take 3.6 us here.
template <int BITS>
__global__ __launch_bounds__(kBlock) void append_kernel(AppendArgs a, Tables K) {
  __shared__ float s_mul[2][kD];
  stage_tables(K, s_mul);
  const uint32_t lane = threadIdx.x & 63u, l = lane & 15u, row = lane >> 4;
  const uint32_t item = __builtin_amdgcn_readfirstlane(blockIdx.x * (kBlock / 64) + (threadIdx.x >> 6));
  const uint32_t side = item & 1u, head = (item >> 1) % a.heads;
  uint64_t tok = (uint64_t)((item >> 1) / a.heads) * a.quads * 4u;
  if (tok >= a.tokens) return;
  const uint64_t end = tok + 4u * a.quads < a.tokens ? tok + 4u * a.quads : a.tokens;
  const uint32_t P = 1u << a.page_log2;
  const LaneForward f = lane_forward(K, l);
  const uint32_t kappa = rev4(l);
  float m[8];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const uint32_t c = 2 * (kappa + 16 * r);
    m[2 * r] = packing(c);
    m[2 * r + 1] = packing(c + 1);
    if (K.scaled) {
      m[2 * r] *= s_mul[side][c];
      m[2 * r + 1] *= s_mul[side][c + 1];
    }
  }
  for (tok += row; tok - row < end; tok += 4) {
    const int64_t slot = tok < end ? a.slots[tok] : -1;
    const bool live = slot >= 0 && slot < ((int64_t)a.pages << a.page_log2);
    float x[8], y[8];
    const int64_t off = side ? (int64_t)tok * a.vt + (int64_t)head * a.vh : (int64_t)tok * a.kt + (int64_t)head * a.kh;
    const void* src = side ? a.v : a.k;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.0f;
    if (live) {
      if (a.f32) {
        const float* p = static_cast<const float*>(src) + off + 8 * l;
        if (a.vec) {
          const float4 u0 = reinterpret_cast<const float4*>(p)[0], u1 = reinterpret_cast<const float4*>(p)[1];
          x[0] = u0.x; x[1] = u0.y; x[2] = u0.z; x[3] = u0.w;
          x[4] = u1.x; x[5] = u1.y; x[6] = u1.z; x[7] = u1.w;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = p[i];
        }
      } else {
        const uint16_t* p = static_cast<const uint16_t*>(src) + off + 8 * l;
        uint32_t w[4];
        if (a.vec) {
          const uint4 u = *reinterpret_cast<const uint4*>(p);
          w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = (uint32_t)p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[2 * i] = __uint_as_float(w[i] << 16);
          x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
      }
    }
    forward_row(x, y, m, l, f);

    // Group kappa / 4 + 4 r lies in the four lanes that share kappa / 4: l, l ^ 4, l ^ 8, l ^ 12.
    constexpr int L = BITS == 4 ? 7 : 127;
    bool bad = false;
    float delta[4];
    uint32_t hb[4], word[4], word1[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      bad |= !__builtin_isfinite(y[2 * r]) || !__builtin_isfinite(y[2 * r + 1]);
      float g = fmaxf(fabsf(y[2 * r]), fabsf(y[2 * r + 1]));
      g = fmaxf(g, lane_xor<8>(g));
      g = fmaxf(g, lane_xor<4>(g));
      const _Float16 h = (_Float16)fminf(div_l<L>(g), 65504.0f);
      delta[r] = (float)h;
      hb[r] = (uint32_t)__builtin_bit_cast(uint16_t, h);
    }
    const uint64_t votes = __builtin_amdgcn_ballot_w64(bad);
    bad = ((votes >> (lane & 48u)) & 0xFFFFu) != 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float inv = delta[r] > 0.0f ? recip_f16_value(delta[r]) : 0.0f;
      const int32_t q0 = (int32_t)__builtin_amdgcn_fmed3f(__builtin_rintf(y[2 * r] * inv), (float)-L, (float)L);
      const int32_t q1 = (int32_t)__builtin_amdgcn_fmed3f(__builtin_rintf(y[2 * r + 1] * inv), (float)-L, (float)L);
      const uint32_t j = kappa & 3u;  // the lane's pair of the group's 8 codes
      if (BITS == 4) {
        word[r] = (((uint32_t)q0 & 15u) | (((uint32_t)q1 & 15u) << 4)) << (8u * j);
        word1[r] = 0;
      } else {
        const uint32_t two = (((uint32_t)q0 & 255u) | (((uint32_t)q1 & 255u) << 8)) << (16u * (j & 1u));
        word[r] = j < 2u ? two : 0u;
        word1[r] = j < 2u ? 0u : two;
      }
      word[r] |= lane_xor_u<8>(word[r]);
      word[r] |= lane_xor_u<4>(word[r]);
      if (BITS == 8) {
        word1[r] |= lane_xor_u<8>(word1[r]);
        word1[r] |= lane_xor_u<4>(word1[r]);
      }
    }
    if (live) {
      // each of the four lanes stores one of the four groups: r = kappa mod 4
      const uint32_t r = kappa & 3u, g = (kappa >> 2) + 4u * r;
      uint32_t w0 = r == 0 ? word[0] : r == 1 ? word[1] : r == 2 ? word[2] : word[3];
      uint32_t w1 = r == 0 ? word1[0] : r == 1 ? word1[1] : r == 2 ? word1[2] : word1[3];
      uint32_t h = r == 0 ? hb[0] : r == 1 ? hb[1] : r == 2 ? hb[2] : hb[3];
      if (bad) {  // zero codes, NaN scales
        w0 = w1 = 0u;
        h = 0x7E00u;
      }
      const uint32_t t = (uint32_t)slot & (P - 1u);
      uint8_t* page = a.cache + ((uint64_t)(slot >> a.page_log2) * a.heads + head) * ((uint64_t)P * Page<BITS>::kToken);
      uint8_t* cdst = page + (side ? Page<BITS>::v_code(P, t, g) : Page<BITS>::k_code(P, t) + g * BITS);
      if (BITS == 4) *reinterpret_cast<uint32_t*>(cdst) = w0;
      else *reinterpret_cast<uint2*>(cdst) = make_uint2(w0, w1);
      *reinterpret_cast<uint16_t*>(page + (side ? Page<BITS>::v_scale(P, t, g) : Page<BITS>::k_scale(P, t) + 2u * g)) = (uint16_t)h;
    }
  }
}

struct ReadArgs {
  const uint8_t* cache;
  const int64_t* slots;
  uint64_t tokens;
  void *k, *v;
  uint32_t heads, pages, page_log2, quads;
  int f32, sides;  // bit 0 K, bit 1 V
};

template <int BITS>
__global__ __launch_bounds__(kBlock) void read_kernel(ReadArgs a, Tables K) {
  __shared__ float s_mul[2][kD];
  stage_tables(K, s_mul);
  const uint32_t lane = threadIdx.x & 63u, l = lane & 15u, row = lane >> 4;
  const uint32_t item = __builtin_amdgcn_readfirstlane(blockIdx.x * (kBlock / 64) + (threadIdx.x >> 6));
  const uint32_t side = a.sides == 3 ? item & 1u : (uint32_t)a.sides >> 1, rest = a.sides == 3 ? item >> 1 : item;
  const uint32_t head = rest % a.heads;
  uint64_t tok = (uint64_t)(rest / a.heads) * a.quads * 4u;
  if (tok >= a.tokens) return;
  const uint64_t end = tok + 4u * a.quads < a.tokens ? tok + 4u * a.quads : a.tokens;
  const uint32_t P = 1u << a.page_log2;
  const LaneInverse f = lane_inverse(K, l);
  float lam[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) lam[i] = K.scaled ? s_mul[side][8 * l + i] : 1.0f;
  for (tok += row; tok - row < end; tok += 4) {
    const bool have = tok < end;
    const int64_t slot = have ? a.slots[tok] : -1;
    const bool live = slot >= 0 && slot < ((int64_t)a.pages << a.page_log2);
    float y[8], x[8];
    uint32_t w0 = 0, w1 = 0, hb = 0;
    if (live) {
      const uint32_t t = (uint32_t)slot & (P - 1u);
      const uint8_t* page = a.cache + ((uint64_t)(slot >> a.page_log2) * a.heads + head) * ((uint64_t)P * Page<BITS>::kToken);
      const uint8_t* c = page + (side ? Page<BITS>::v_code(P, t, l) : Page<BITS>::k_code(P, t) + l * BITS);
      if (BITS == 4) {
        w0 = *reinterpret_cast<const uint32_t*>(c);
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(c);
        w0 = u.x;
        w1 = u.y;
      }
      hb = *reinterpret_cast<const uint16_t*>(page + (side ? Page<BITS>::v_scale(P, t, l) : Page<BITS>::k_scale(P, t) + 2u * l));
    }
    const float delta = (float)__builtin_bit_cast(_Float16, (uint16_t)hb);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int32_t q = BITS == 4 ? __builtin_amdgcn_sbfe(w0, 4 * i, 4) : __builtin_amdgcn_sbfe(i < 4 ? w0 : w1, 8 * (i & 3), 8);
      y[i] = (float)q * delta;
      y[i] *= lam[i];
    }
    inverse_row(y, x, l, f);
    if (have) {
      const uint64_t at = (tok * a.heads + head) * kD;
      void* out = side ? a.v : a.k;
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // each store instruction covers 64 (128) consecutive bytes a row
        const uint64_t i = at + 2u * inverse_n(l, e);
        if (a.f32) *reinterpret_cast<float2*>(static_cast<float*>(out) + i) = make_float2(x[2 * e], x[2 * e + 1]);
        else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(out) + i) = bf16_pair(x[2 * e], x[2 * e + 1]);
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------
// Eviction.  Of a (sequence, head)'s n tokens m = min(n, budget) stay: the first `sink`, the last
// `recent`, and those of most weight among the others, ties to the lowest index.
struct EvictArgs {
  uint8_t* cache;
  const int32_t *table, *lens, *dst;
  const float* weights;
  uint64_t wstride;
  int32_t *kept, *new_lens;
  float* new_weights;
  uint32_t seqs, heads, pages, page_log2, width, dst_width, max_len, budget, sink, recent;
};

// Order-preserving key of a weight: larger weight, larger key; -0 counts as 0, NaN below everything.  Keys of
// weights lie in [1, 0xFF800000]; 0 is a token past the end, all ones one that stays whatever its weight.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t b = __float_as_uint(w + 0.0f);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 1u;
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ uint32_t clamp_len(int32_t n, uint32_t most) { return n < 0 ? 0u : (uint32_t)n < most ? (uint32_t)n : most; }

// One workgroup per (sequence, head): the m-th largest key by three counting passes of 11, 11 and 10 bits (most
// significant first), then one ordered pass that numbers the tokens that stay.  A wavefront owns a run of
// tokens, PER of them a lane as keys in registers (the weights are read once, for up to 1024 PER tokens), so
// the ordered pass needs the counts of the wavefronts before it and no exchange within.  With PER == 0 the
// weights are read again in each pass.  Vector instructions bound it: one compute unit works on a row.
constexpr int kSelect = 1024, kSelectWaves = kSelect / 64, kHeldFew = 8, kHeld = 32, kBins = 2048;

template <int PER>
__global__ __launch_bounds__(kSelect) void evict_select_kernel(EvictArgs a) {
  __shared__ __align__(16) uint32_t hist[kBins], s_wave[kSelectWaves], s_tie[kSelectWaves];
  __shared__ uint32_t s_prefix, s_left;
  const uint32_t b = blockIdx.x / a.heads, h = blockIdx.x % a.heads, tid = threadIdx.x;
  const uint32_t lane = tid & 63u, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t width_tokens = a.width << a.page_log2;
  const uint32_t n = clamp_len(a.lens[b], a.max_len < width_tokens ? a.max_len : width_tokens);
  const uint32_t m = n < a.budget ? n : a.budget;
  const float* w = a.weights + ((uint64_t)b * a.heads + h) * a.wstride;
  const uint32_t lo = a.sink < n ? a.sink : n, rest = n - (a.recent < n ? a.recent : n), hi = rest > lo ? rest : lo;
  // the wavefront's run of tokens: `steps` times 64 from `first`
  const uint32_t steps = (n + kSelect - 1) / kSelect, first = wave * steps * 64u + lane;
  auto key_at = [&](uint32_t t) __attribute__((always_inline)) {
    return t >= n ? 0u : t < lo || t >= hi ? 0xFFFFFFFFu : weight_key(w[t]);
  };
  uint32_t held[PER ? PER : 1];
  if (PER) {
    float raw[PER ? PER : 1];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      raw[PER ? i : 0] = 0.0f;
      if ((uint32_t)i < steps && first + 64u * i < n) raw[PER ? i : 0] = w[first + 64u * i];
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint32_t t = first + 64u * i;
      held[PER ? i : 0] = t >= n ? 0u : t < lo || t >= hi ? 0xFFFFFFFFu : weight_key(raw[PER ? i : 0]);
    }
  }
  auto each = [&](auto&& body) __attribute__((always_inline)) {
    if (PER) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if ((uint32_t)i < steps) body(first + 64u * i, held[PER ? i : 0]);
    } else {
      for (uint32_t i = 0; i < steps; ++i) body(first + 64u * i, key_at(first + 64u * i));
    }
  };
  if (tid == 0 && h == 0) a.new_lens[b] = (int32_t)m;

  // tokens with keys above `prefix` stay, and of those with it the first `left`
  uint32_t prefix = m == n ? 0u : 0xFFFFFFFFu, left = 0;
  if (m > 0 && m < n) {
    prefix = 0;
    left = m;
    hist[2 * tid] = hist[2 * tid + 1] = 0;
    __syncthreads();
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t above = pass == 0 ? 0u : pass == 1 ? 0xFFE00000u : 0xFFFFFC00u, mask = pass == 2 ? 1023u : 2047u;
      each([&](uint32_t, uint32_t key) {
        const bool in = (key & above) == prefix;
        const uint64_t votes = __builtin_amdgcn_ballot_w64(in);
        if (!votes) return;
        // the first lane's bin is counted with one addition, so that many equal keys do not queue up
        const uint32_t bin = (key >> shift) & mask, lead = (uint32_t)__builtin_ctzll(votes);
        const bool same = in && bin == (uint32_t)__builtin_amdgcn_readlane((int)bin, (int)lead);
        const uint32_t count = (uint32_t)__builtin_popcountll(__builtin_amdgcn_ballot_w64(same));
        if (in && (!same || lane == lead)) atomicAdd(&hist[bin], same ? count : 1u);
      });
      __syncthreads();
      // tokens in this thread's two bins and all above them
      const uint32_t c1 = hist[2 * tid + 1], c0 = hist[2 * tid];
      hist[2 * tid] = hist[2 * tid + 1] = 0;
      uint32_t sum = c0 + c1;
#pragma unroll
      for (uint32_t d = 1; d < 64; d <<= 1) {
        const uint32_t up = (uint32_t)__builtin_amdgcn_ds_bpermute((int)(((lane + d) & 63u) << 2), (int)sum);
        if (lane + d < 64u) sum += up;
      }
      if (lane == 0) s_wave[wave] = sum;
      __syncthreads();
#pragma unroll
      for (uint32_t i = 0; i < kSelectWaves; ++i) sum += i > wave ? s_wave[i] : 0u;
      const uint32_t before = sum - c0 - c1;  // in the bins above
      if (before < left && left <= sum) {     // one thread
        const bool upper = left <= before + c1;
        s_prefix = prefix | (2 * tid + (upper ? 1u : 0u)) << shift;
        s_left = upper ? left - before : left - before - c1;
      }
      __syncthreads();
      prefix = s_prefix;
      left = s_left;
    }
  }

  uint32_t sure = 0, ties = 0;
  each([&](uint32_t, uint32_t key) {
    sure += (uint32_t)__builtin_popcountll(__builtin_amdgcn_ballot_w64(key > prefix));
    ties += (uint32_t)__builtin_popcountll(__builtin_amdgcn_ballot_w64(key == prefix));
  });
  __syncthreads();
  if (lane == 0) {
    s_wave[wave] = sure;
    s_tie[wave] = ties;
  }
  __syncthreads();
  uint32_t kept = 0, eq = 0;  // tokens that stay, and ties, of the wavefronts before
#pragma unroll
  for (uint32_t i = 0; i < kSelectWaves; ++i) {
    const uint32_t room = left > eq ? left - eq : 0u, tie = i < wave ? s_tie[i] : 0u;
    kept += (i < wave ? s_wave[i] : 0u) + (tie < room ? tie : room);
    eq += tie;
  }
  int32_t* dst = a.kept + ((uint64_t)b * a.heads + h) * a.budget;
  float* wd = a.new_weights ? a.new_weights + ((uint64_t)b * a.heads + h) * a.budget : nullptr;
  const uint64_t below = (1ull << lane) - 1ull;
  each([&](uint32_t t, uint32_t key) {
    const bool tie = key == prefix;
    const uint64_t vt = __builtin_amdgcn_ballot_w64(tie);
    const bool take = key > prefix || (tie && eq + (uint32_t)__builtin_popcountll(vt & below) < left);
    eq += (uint32_t)__builtin_popcountll(vt);
    const uint64_t vk = __builtin_amdgcn_ballot_w64(take);
    if (!vk) return;
    const uint32_t at = kept + (uint32_t)__builtin_popcountll(vk & below);
    kept += (uint32_t)__builtin_popcountll(vk);
    if (take && at < a.budget) {
      dst[at] = (int32_t)t;
      if (wd) wd[at] = w[t];
    }
  });
  for (uint32_t j = m + tid; j < a.budget; j += kSelect) {
    dst[j] = -1;
    if (wd) wd[j] = 0.0f;
  }
}

// Moves the tokens that stay: 16 lanes take four consecutive destination tokens, which are one block of V, so
// that a lane stores its group's codes and scales of all four at once.  Values lie by blocks of four tokens,
// so where a quarter of the tokens stay nearly all of V is read; that traffic bounds the kernel.  A token of an
// absent page that stays gets zeros, with the sign set in its keys' scales: it takes no part where it goes either.
template <int BITS>
__global__ __launch_bounds__(kBlock) void evict_move_kernel(EvictArgs a, uint32_t blocks) {
  const uint32_t l = threadIdx.x & 15u, bh = blockIdx.x / blocks, b = bh / a.heads, h = bh % a.heads;
  const uint32_t j = ((blockIdx.x % blocks) * (kBlock / 16) + (threadIdx.x >> 4)) * 4u;
  if (j >= a.budget) return;
  const int32_t* kept = a.kept + (uint64_t)bh * a.budget;
  const uint32_t P = 1u << a.page_log2, to = j & (P - 1u);
  const int32_t dp = a.dst[(uint64_t)b * a.dst_width + (j >> a.page_log2)];
  if ((uint32_t)dp >= a.pages) return;
  const uint64_t size = (uint64_t)P * Page<BITS>::kToken;
  uint8_t* d = a.cache + ((uint64_t)dp * a.heads + h) * size;
  int32_t src[4];  // -1: absent; -2: no token
  const uint8_t* page[4];
  bool whole = true;
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i) {
    src[i] = j + i < a.budget ? kept[j + i] : -1;
    if (src[i] < 0) src[i] = -2;
    const int32_t sp = src[i] >= 0 ? a.table[(uint64_t)b * a.width + ((uint32_t)src[i] >> a.page_log2)] : -1;
    if (src[i] >= 0 && (uint32_t)sp >= a.pages) src[i] = -1;
    page[i] = a.cache + ((uint64_t)(src[i] < 0 ? 0 : sp) * a.heads + h) * size;
    whole &= src[i] != -2;
  }
  typedef uint32_t piece __attribute__((ext_vector_type(BITS / 4)));
  piece v[4];
  uint32_t s[4];
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i) {
    const uint32_t so = (uint32_t)(src[i] < 0 ? 0 : src[i]) & (P - 1u);
    v[i] = *reinterpret_cast<const piece*>(page[i] + Page<BITS>::v_code(P, so, l));
    s[i] = *reinterpret_cast<const uint16_t*>(page[i] + Page<BITS>::v_scale(P, so, l));
    if (src[i] < 0) {
      v[i] = (piece)0u;
      s[i] = 0u;
    }
  }
  // keys: the lane's quarter of one of the four vectors
  const uint32_t which = l >> 2, part = l & 3u;
  const int32_t ks = which == 0 ? src[0] : which == 1 ? src[1] : which == 2 ? src[2] : src[3];
  const uint8_t* kp = which == 0 ? page[0] : which == 1 ? page[1] : which == 2 ? page[2] : page[3];
  const uint32_t ko = (uint32_t)(ks < 0 ? 0 : ks) & (P - 1u);
  const uint4* kc = reinterpret_cast<const uint4*>(kp + Page<BITS>::k_code(P, ko) + part * 4u * BITS);
  uint4 k0 = kc[0], k1 = kc[BITS / 8];
  uint2 kscale = *reinterpret_cast<const uint2*>(kp + Page<BITS>::k_scale(P, ko) + 8u * part);
  if (ks < 0) {
    k0 = k1 = make_uint4(0u, 0u, 0u, 0u);
    kscale = make_uint2(0x80008000u, 0x80008000u);
  }
  if (ks != -2) {
    uint4* kd = reinterpret_cast<uint4*>(d + Page<BITS>::k_code(P, to + which) + part * 4u * BITS);
    kd[0] = k0;
    if (BITS == 8) kd[1] = k1;
    *reinterpret_cast<uint2*>(d + Page<BITS>::k_scale(P, to + which) + 8u * part) = kscale;
  }
  uint8_t *vd = d + Page<BITS>::v_code(P, to, l), *sd = d + Page<BITS>::v_scale(P, to, l);
  if (whole) {
    uint32_t w[BITS];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < BITS / 4; ++c) w[i * (BITS / 4) + c] = v[i][c];
#pragma unroll
    for (int i = 0; i < BITS / 4; ++i) reinterpret_cast<uint4*>(vd)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    *reinterpret_cast<uint2*>(sd) = make_uint2(s[0] | s[1] << 16, s[2] | s[3] << 16);
  } else {
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i)
      if (src[i] != -2) {
        reinterpret_cast<piece*>(vd)[i] = v[i];
        reinterpret_cast<uint16_t*>(sd)[i] = (uint16_t)s[i];
      }
  }
}

}  // namespace hq_kv

using namespace hq_kv;

static uint32_t log2_of(uint32_t v) { return 31u - (uint32_t)__builtin_clz(v); }

// Workgroups of append and read, and the fours of tokens a wavefront takes in turn: as many as leave the chip
// 16384 wavefronts (256 CUs of 4 SIMDs, 16 each), at most 32.
static uint64_t transform_grid(uint64_t tokens, uint64_t rows, uint32_t* quads) {
  const uint64_t all = (tokens + 3) / 4;
  const uint64_t per = all * rows / 16384;
  *quads = (uint32_t)(per < 1 ? 1 : per > 32 ? 32 : per);
  const uint64_t items = (all + *quads - 1) / *quads * rows;
  return (items + kBlock / 64 - 1) / (kBlock / 64);
}

// A vector a thread (hq_srft.hip) takes 2.5 times fewer instructions than 16 lanes a vector, once it fills the chip:
// 32768 tokens of 8 heads append in 74 us against 105 and read in 44 against 67, 8192 in 26 against 33 and 18
// against 23, 4096 (at 8 bits) in 19 against 20 and 15 against 13.  K and V with lambdas are launches of their
// own, so that each has to fill it.
constexpr uint64_t kManyVectors = 1u << 17;  // of a launch
static bool many_vectors(const hq_kv_cache& c, uint64_t tokens, uint32_t sides) {
  const uint64_t vectors = tokens * c.heads * (c.lambda_k || c.lambda_v ? 1u : sides);
  return vectors >= kManyVectors && (tokens + 255) / 256 * c.heads * sides <= kMaxThreads / 256;
}

extern "C" {

int hq_kv_append(const hq_kv_cache* cache, const void* k, const void* v, int32_t dtype, uint64_t tokens,
                 const int64_t strides[4], const int64_t* slots, hq_stream_t stream) {
  if (int rc = check_cache(cache)) return rc;
  if ((dtype != HQ_F32 && dtype != HQ_BF16) || !strides || tokens > (1ull << 31)) return HQ_ERR_INVALID_ARG;
  if (tokens && (!k || !v || !slots || ((uintptr_t)slots & 7u))) return HQ_ERR_INVALID_ARG;
  const uint32_t size = dtype == HQ_F32 ? 4u : 2u;
  if (((uintptr_t)k | (uintptr_t)v) & (size - 1u)) return HQ_ERR_INVALID_ARG;
  AppendArgs a;
  Tables T;
  if (!make_tables(*cache, true, &T)) return HQ_ERR_INVALID_ARG;
  if (tokens == 0 || cache->pages == 0) return HQ_OK;
  a.cache = static_cast<uint8_t*>(cache->data);
  a.k = k;
  a.v = v;
  a.slots = slots;
  a.tokens = tokens;
  a.kt = strides[0];
  a.kh = strides[1];
  a.vt = strides[2];
  a.vh = strides[3];
  a.heads = cache->heads;
  a.pages = cache->pages;
  a.page_log2 = log2_of(cache->page);
  a.f32 = dtype == HQ_F32;
  // 16-byte loads where every row starts on 16 bytes, single values otherwise
  const int64_t per = 16 / size;
  a.vec = !(((uintptr_t)k | (uintptr_t)v) & 15u) && !(a.kt % per) && !(a.kh % per) && !(a.vt % per) && !(a.vh % per);
  const uint64_t grid = transform_grid(tokens, cache->heads * 2, &a.quads);
  if (grid > kMaxThreads / kBlock) return HQ_ERR_INVALID_ARG;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (a.vec && many_vectors(*cache, tokens, 2)) {
    const ManyAppend many = {a.cache, k, v, slots, tokens, a.kt, a.kh, a.vt, a.vh, a.heads, a.pages, a.page_log2, 0, 0};
    launch_append_many(*cache, many, a.f32, st);
    return hipGetLastError() == hipSuccess ? HQ_OK : HQ_ERR_HIP;
  }
  if (cache->bits == 4) hipLaunchKernelGGL(append_kernel<4>, dim3((uint32_t)grid), dim3(kBlock), 0, st, a, T);
  else hipLaunchKernelGGL(append_kernel<8>, dim3((uint32_t)grid), dim3(kBlock), 0, st, a, T);
  return hipGetLastError() == hipSuccess ? HQ_OK : HQ_ERR_HIP;
}

int hq_kv_read(const hq_kv_cache* cache, const int64_t* slots, uint64_t tokens, void* k, void* v, int32_t out_dtype,
               hq_stream_t stream) {
  if (int rc = check_cache(cache)) return rc;
  if ((out_dtype != HQ_F32 && out_dtype != HQ_BF16) || tokens > (1ull << 31)) return HQ_ERR_INVALID_ARG;
  if (tokens && ((!k && !v) || !slots || ((uintptr_t)slots & 7u))) return HQ_ERR_INVALID_ARG;
  if (((uintptr_t)k | (uintptr_t)v) & 15u) return HQ_ERR_INVALID_ARG;
  Tables T;
  if (!make_tables(*cache, false, &T)) return HQ_ERR_INVALID_ARG;
  if (tokens == 0) return HQ_OK;
  ReadArgs a;
  a.cache = static_cast<const uint8_t*>(cache->data);
  a.slots = slots;
  a.tokens = tokens;
  a.k = k;
  a.v = v;
  a.heads = cache->heads;
  a.pages = cache->pages;
  a.page_log2 = log2_of(cache->page);
  a.f32 = out_dtype == HQ_F32;
  a.sides = (k ? 1 : 0) | (v ? 2 : 0);
  const uint64_t grid = transform_grid(tokens, cache->heads * (a.sides == 3 ? 2 : 1), &a.quads);
  if (grid > kMaxThreads / kBlock) return HQ_ERR_INVALID_ARG;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (many_vectors(*cache, tokens, a.sides == 3 ? 2 : 1)) {
    const ManyRead many = {a.cache, slots, tokens, k, v, a.heads, a.pages, a.page_log2, 0, 0};
    launch_read_many(*cache, many, a.f32, st);
    return hipGetLastError() == hipSuccess ? HQ_OK : HQ_ERR_HIP;
  }
  if (cache->bits == 4) hipLaunchKernelGGL(read_kernel<4>, dim3((uint32_t)grid), dim3(kBlock), 0, st, a, T);
  else hipLaunchKernelGGL(read_kernel<8>, dim3((uint32_t)grid), dim3(kBlock), 0, st, a, T);
  return hipGetLastError() == hipSuccess ? HQ_OK : HQ_ERR_HIP;
}

int hq_kv_evict(const hq_kv_cache* cache, const hq_kv_evict_args* e, hq_stream_t stream) {
  if (int rc = check_cache(cache)) return rc;
  if (!e || e->max_len > kMaxTokens || e->budget > 0x7FFFFFFFu) return HQ_ERR_INVALID_ARG;
  if ((uint64_t)e->sink + e->recent > e->budget) return HQ_ERR_INVALID_ARG;
  if ((uint64_t)e->table_width * cache->page > 0x7FFFFFFFull || (uint64_t)e->dst_width * cache->page < e->budget) return HQ_ERR_INVALID_ARG;
  if (e->weights_stride < e->max_len) return HQ_ERR_INVALID_ARG;
  if ((uint64_t)e->seqs * cache->heads > kMaxThreads / kSelect) return HQ_ERR_INVALID_ARG;
  if (e->seqs == 0) return HQ_OK;
  if (!e->lens || !e->new_lens || (e->max_len && (!e->weights || !e->table)) || (e->budget && (!e->kept || !e->dst_table))) return HQ_ERR_INVALID_ARG;
  if (((uintptr_t)e->lens | (uintptr_t)e->new_lens | (uintptr_t)e->weights | (uintptr_t)e->table | (uintptr_t)e->kept |
       (uintptr_t)e->dst_table | (uintptr_t)e->new_weights) & 3u)
    return HQ_ERR_INVALID_ARG;
  EvictArgs a;
  a.cache = static_cast<uint8_t*>(cache->data);
  a.table = e->table;
  a.lens = e->lens;
  a.dst = e->dst_table;
  a.weights = e->weights;
  a.wstride = e->weights_stride;
  a.kept = e->kept;
  a.new_lens = e->new_lens;
  a.new_weights = e->new_weights;
  a.seqs = e->seqs;
  a.heads = cache->heads;
  a.pages = cache->pages;
  a.page_log2 = log2_of(cache->page);
  a.width = e->table_width;
  a.dst_width = e->dst_width;
  a.max_len = e->max_len;
  a.budget = e->budget;
  a.sink = e->sink;
  a.recent = e->recent;
  // 64 destination tokens a workgroup
  const uint32_t blocks = (e->budget + kBlock / 4 - 1) / (kBlock / 4);
  const uint64_t grid = (uint64_t)e->seqs * cache->heads * blocks;
  if (grid > kMaxThreads / kBlock) return HQ_ERR_INVALID_ARG;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const dim3 select(e->seqs * cache->heads);
  // 8 keys a lane where they hold the tokens: every pass is unrolled over them, and fetching skipped code costs (1040
  // tokens: 8.6 us against 12.3 with 32 keys a lane).  Keys in LDS: 8.4 us for 1040, but 47 against 34 for 32768.
  if (e->max_len <= kSelect * kHeldFew) hipLaunchKernelGGL(evict_select_kernel<kHeldFew>, select, dim3(kSelect), 0, st, a);
  else if (e->max_len <= kSelect * kHeld) hipLaunchKernelGGL(evict_select_kernel<kHeld>, select, dim3(kSelect), 0, st, a);
  else hipLaunchKernelGGL(evict_select_kernel<0>, select, dim3(kSelect), 0, st, a);
  if (grid && cache->pages) {
    if (cache->bits == 4) hipLaunchKernelGGL(evict_move_kernel<4>, dim3((uint32_t)grid), dim3(kBlock), 0, st, a, blocks);
    else hipLaunchKernelGGL(evict_move_kernel<8>, dim3((uint32_t)grid), dim3(kBlock), 0, st, a, blocks);
  }
  return hipGetLastError() == hipSuccess ? HQ_OK : HQ_ERR_HIP;
}

}  // extern "C"
