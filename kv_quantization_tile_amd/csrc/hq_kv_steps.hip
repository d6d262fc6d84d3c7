// hq_kv_steps.hip -- what a serving step needs around the paged SRFT cache: places for its tokens (pages taken from
// and returned to a stack, block tables, slots), and the acceptance of drafted tokens.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/hq.h"
#include "hq_kv_device.h"
#include "hq_kv_internal.h"

namespace hq_kv {

constexpr int kStepBlock = 256;

// ---- places ------------------------------------------------------------------------------------

constexpr int kPlan = 1024, kPlanWaves = kPlan / 64;

struct ReserveArgs {
  int32_t *table, *lens;
  const int32_t* counts;
  int32_t *free, *free_count;
  int64_t* slots;
  int32_t *positions, *q_start, *granted;
  uint64_t tokens;
  uint32_t seqs, width, pages, page_log2;
  int here;  // the plan's workgroup writes the slots too
};

// x of this lane and those before it.
__device__ __forceinline__ uint64_t wave_scan(uint64_t x, uint32_t lane) {
  uint32_t lo = (uint32_t)x, hi = (uint32_t)(x >> 32);
#pragma unroll
  for (uint32_t d = 1; d < 64; d <<= 1) {
    const int from = (int)(((lane - d) & 63u) << 2);
    const uint64_t y = (uint64_t)(uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)lo) |
                       (uint64_t)(uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)hi) << 32;
    if (lane >= d) x += y;
    lo = (uint32_t)x;
    hi = (uint32_t)(x >> 32);
  }
  return x;
}
// Sum of x over the threads up to this one, and over the workgroup.  s: kPlanWaves words that nothing else uses.
__device__ __forceinline__ uint64_t block_scan(uint64_t x, uint64_t* s, uint64_t* all) {
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  uint64_t sum = wave_scan(x, lane), total = 0;
  __syncthreads();
  if (lane == 63) s[wave] = sum;
  __syncthreads();
#pragma unroll
  for (uint32_t i = 0; i < (uint32_t)kPlanWaves; ++i) {
    if (i < wave) sum += s[i];
    total += s[i];
  }
  *all = total;
  return sum;
}
// The last of `count` ascending starts that is at or below x (0 if none is).
__device__ __forceinline__ uint32_t last_at(const uint32_t* start, uint32_t count, uint32_t x) {
  uint32_t lo = 0;
  while (count > 1) {
    const uint32_t half = count / 2;
    if (start[lo + half] <= x) {
      lo += half;
      count -= half;
    } else {
      count = half;
    }
  }
  return lo;
}

__device__ __forceinline__ uint32_t pages_of(const ReserveArgs& a, uint64_t tokens) {
  return (uint32_t)((tokens + (1u << a.page_log2) - 1u) >> a.page_log2);
}
__device__ __forceinline__ uint32_t held_tokens(const ReserveArgs& a, uint32_t b) {
  const int32_t n = a.lens[b];
  const uint32_t most = a.width << a.page_log2;
  return n < 0 ? 0u : (uint32_t)n < most ? (uint32_t)n : most;
}
__device__ __forceinline__ void place(const ReserveArgs& a, uint64_t i, uint32_t b, uint32_t t, bool grown) {
  int64_t slot = -1;
  if (grown) {
    const int32_t page = a.table[(uint64_t)b * a.width + (t >> a.page_log2)];
    if ((uint32_t)page < a.pages) slot = ((int64_t)page << a.page_log2) + (t & ((1u << a.page_log2) - 1u));
  }
  a.slots[i] = slot;
  if (a.positions) a.positions[i] = (int32_t)t;
}

// One workgroup: sums over the sequences say where each one's pages and tokens begin, and a sequence's share
// of them is spread over all threads, so that one long sequence costs no more than many short ones.  What it moves is a few
// kilobytes: the chain of loads, sums and barriers bounds it (4 sequences 6.2 us, 333 sequences with 34000 tokens 9.7 us and 2.9 for
// their places), and several workgroups would need a launch between returning pages and taking them.
__global__ __launch_bounds__(kPlan) void reserve_kernel(ReserveArgs a) {
  __shared__ uint64_t s_wave[kPlanWaves];
  __shared__ uint32_t s_start[kPlan], s_first[kPlan], s_tokens[kPlan], s_old[kPlan];
  __shared__ uint8_t s_grown[kPlan];
  const uint32_t tid = threadIdx.x;
  const int32_t fc = *a.free_count;
  uint32_t top = fc < 0 ? 0u : (uint32_t)fc < a.pages ? (uint32_t)fc : a.pages;
  uint64_t all;

  // pages that return: sequences from the last, each one's pages from its last
  for (uint32_t b0 = 0; b0 < a.seqs; b0 += kPlan) {
    const uint32_t k = b0 + tid, b = a.seqs - 1u - k;
    uint32_t gone = 0, last = 0;
    if (k < a.seqs) {
      const int32_t c = a.counts[b];
      if (c < 0) {
        const uint32_t old = held_tokens(a, b), drop = 0u - (uint32_t)c;
        last = pages_of(a, old);
        gone = last - pages_of(a, old > drop ? old - drop : 0u);
      }
    }
    const uint64_t end = block_scan(gone, s_wave, &all);
    if (all == 0) continue;
    s_start[tid] = (uint32_t)(end - gone);
    s_first[tid] = last;
    __syncthreads();
    for (uint32_t r0 = 0; r0 < (uint32_t)all; r0 += kPlan) {
      const uint32_t r = r0 + tid;
      int32_t page = -1;
      if (r < (uint32_t)all) {
        const uint32_t i = last_at(s_start, kPlan, r);
        int32_t* entry = a.table + (uint64_t)(a.seqs - 1u - (b0 + i)) * a.width + (s_first[i] - 1u - (r - s_start[i]));
        page = *entry;
        *entry = -1;
      }
      const bool back = (uint32_t)page < a.pages;
      uint64_t count;
      const uint64_t upto = block_scan(back ? 1u : 0u, s_wave, &count);
      if (back && top + upto <= a.pages) a.free[top + upto - 1u] = page;
      top = top + count < a.pages ? (uint32_t)(top + count) : a.pages;
    }
    __syncthreads();
  }
  __threadfence_block();
  __syncthreads();

  // pages that are taken, and the tokens' places
  uint64_t needs = 0, tokens = 0;  // of the sequences before
  uint32_t taken = 0;
  for (uint32_t b0 = 0; b0 < a.seqs; b0 += kPlan) {
    const uint32_t b = b0 + tid;
    uint32_t need = 0, old = 0;
    int32_t c = 0;
    bool fits = false;
    if (b < a.seqs) {
      c = a.counts[b];
      old = held_tokens(a, b);
      fits = c > 0 && (uint64_t)old + (uint32_t)c <= (uint64_t)a.width << a.page_log2;
      if (fits) need = pages_of(a, (uint64_t)old + (uint32_t)c) - pages_of(a, old);
    }
    uint64_t all_needs, all_tokens;
    const uint64_t need_end = needs + block_scan(need, s_wave, &all_needs);
    const uint64_t token_end = tokens + block_scan(c > 0 ? (uint64_t)c : 0u, s_wave, &all_tokens);
    const bool grown = fits && need_end <= top;
    const uint64_t token_start = token_end - (c > 0 ? (uint64_t)c : 0u);
    constexpr uint64_t kMost = 0x7FFFFFFFu;
    if (b < a.seqs) {
      const int32_t change = grown ? c : c < 0 ? ((uint32_t)(0u - (uint32_t)c) < old ? c : -(int32_t)old) : 0;
      a.granted[b] = change;
      if (change) a.lens[b] = (int32_t)(old + (uint32_t)change);
      a.q_start[b] = (int32_t)(token_start < kMost ? token_start : kMost);
      if (b == a.seqs - 1u) a.q_start[a.seqs] = (int32_t)(token_end < kMost ? token_end : kMost);
    }
    s_start[tid] = (uint32_t)(need_end - need - needs);
    s_first[tid] = pages_of(a, old);
    s_tokens[tid] = (uint32_t)(token_start < kMost ? token_start : kMost);
    s_old[tid] = old;
    s_grown[tid] = grown ? 1 : 0;
    // pages of those that grow: they come first
    uint64_t got;
    block_scan(grown ? need : 0u, s_wave, &got);  // the barriers within let the others' words be read
    for (uint32_t r = tid; r < (uint32_t)got; r += kPlan) {
      const uint32_t i = last_at(s_start, kPlan, r);
      a.table[(uint64_t)(b0 + i) * a.width + s_first[i] + (r - s_start[i])] = a.free[top - 1u - (uint32_t)needs - r];
    }
    taken += (uint32_t)got;
    if (a.here) {
      __threadfence_block();
      __syncthreads();
      const uint64_t stop = tokens + all_tokens < a.tokens ? tokens + all_tokens : a.tokens;
      for (uint64_t i = tokens + tid; i < stop; i += kPlan) {
        const uint32_t k = last_at(s_tokens, kPlan, (uint32_t)i);
        place(a, i, b0 + k, s_old[k] + ((uint32_t)i - s_tokens[k]), s_grown[k]);
      }
    }
    needs += all_needs;
    tokens += all_tokens;
    __syncthreads();
  }
  if (a.here) {
    for (uint64_t i = tokens + tid; i < a.tokens; i += kPlan) {
      a.slots[i] = -1;
      if (a.positions) a.positions[i] = 0;
    }
  }
  if (tid == 0) {
    *a.free_count = (int32_t)(top - taken);
    if (a.seqs == 0) a.q_start[0] = 0;
  }
}

// The places of many tokens, a thread each, where one workgroup would write them for too long (hq_kv_reserve).
__global__ __launch_bounds__(kStepBlock) void slots_kernel(ReserveArgs a) {
  const uint64_t i = (uint64_t)blockIdx.x * kStepBlock + threadIdx.x;
  if (i >= a.tokens) return;
  const uint32_t* start = reinterpret_cast<const uint32_t*>(a.q_start);
  if (i >= start[a.seqs]) {
    a.slots[i] = -1;
    if (a.positions) a.positions[i] = 0;
    return;
  }
  const uint32_t b = last_at(start, a.seqs, (uint32_t)i);
  const int32_t change = a.granted[b];
  place(a, i, b, held_tokens(a, b) - (uint32_t)change + ((uint32_t)i - start[b]), change > 0);
}

// ---- acceptance --------------------------------------------------------------------------------

constexpr int kDrafts = 256;

struct AcceptArgs {
  uint8_t* cache;
  const int32_t *table, *lens, *q_start, *tokens, *target, *parents;
  int32_t *path, *accepted, *next, *change;
  uint64_t total_q;
  uint32_t seqs, heads, pages, page_log2, width, max_q;
};

// Where 56 of a wavefront's lanes find a token's pieces: E bytes of K codes (16 lanes), of V codes (16), binary16
// scales of V (16), pairs of K's (8).
template <int BITS>
struct Piece {
  uint32_t at, bytes;
  __device__ __forceinline__ Piece(uint32_t P, uint32_t t, uint32_t lane) {
    const uint32_t g = lane & 15u;
    at = lane < 16u ? Page<BITS>::k_code(P, t) + g * BITS : lane < 32u ? Page<BITS>::v_code(P, t, g)
       : lane < 48u ? Page<BITS>::v_scale(P, t, g) : Page<BITS>::k_scale(P, t) + 4u * (g & 7u);
    bytes = lane < 32u ? BITS : lane < 48u ? 2u : lane < 56u ? 4u : 0u;
  }
};

// A workgroup takes a head of a sequence.  Its first wavefront follows the accepted drafts (64 candidates a
// look), which costs less than a launch of its own; then the wavefronts move the drafts' bytes, 16 at a time,
// all of them read before one is written: a draft moves towards the front, so what a turn overwrites no later
// one reads.  Latency bounds it, a chain of four loads and a few looks: 5.5 us for one sequence's 8 drafts and 8 heads, 9.2 us for
// 64 sequences' 64 drafts at 8 bits, 512 workgroups that move 2.6 MB.
template <int BITS>
__global__ __launch_bounds__(kStepBlock) void accept_kernel(AcceptArgs a) {
  __shared__ int32_t s_token[kDrafts], s_target[kDrafts], s_parent[kDrafts], s_path[kDrafts];
  __shared__ uint32_t s_count;
  const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t h = blockIdx.x % a.heads, b = blockIdx.x / a.heads;
  int64_t q0, all;
  if (a.q_start) {
    const int64_t x = a.q_start[b], y = a.q_start[b + 1], top = (int64_t)a.total_q;
    q0 = x < 0 ? 0 : x > top ? top : x;
    all = y < q0 ? 0 : (y > top ? top : y) - q0;
  } else {
    all = (int64_t)(a.total_q / a.seqs);
    q0 = all * b;
  }
  const uint32_t m = (uint32_t)(all < (int64_t)a.max_q ? all : (int64_t)a.max_q);
  for (uint32_t i = threadIdx.x; i < m; i += kStepBlock) {
    const int32_t p = a.parents[q0 + i];
    s_parent[i] = p >= 0 && p < (int32_t)i ? p : -1;
    s_token[i] = a.tokens[q0 + i];
    s_target[i] = a.target[q0 + i];
  }
  __syncthreads();
  if (wave == 0) {
    uint32_t count = m ? 1u : 0u, at = 0;
    if (lane == 0) s_path[0] = 0;
    while (count && count < m) {
      const int32_t want = s_target[at];
      uint32_t found = m;
      for (uint32_t i0 = (at + 1u) & ~63u; i0 < m && found == m; i0 += 64u) {
        const uint32_t i = i0 + lane;
        const uint64_t votes = __builtin_amdgcn_ballot_w64(i < m && s_parent[i < m ? i : 0] == (int32_t)at && s_token[i < m ? i : 0] == want);
        if (votes) found = i0 + (uint32_t)__builtin_ctzll(votes);
      }
      if (found == m) break;
      if (lane == 0) s_path[count] = (int32_t)found;
      at = found;
      ++count;
    }
    if (lane == 0) s_count = count;
  }
  __syncthreads();
  const uint32_t count = s_count;
  if (h == 0) {
    for (uint32_t i = threadIdx.x; i < a.max_q; i += kStepBlock) a.path[(uint64_t)b * a.max_q + i] = i < count ? s_path[i] : -1;
    if (threadIdx.x == 0) {
      a.accepted[b] = (int32_t)count;
      a.next[b] = count ? s_target[s_path[count - 1u]] : -1;
      a.change[b] = (int32_t)((int64_t)count - all);
    }
  }

  const uint64_t held = (uint64_t)a.width << a.page_log2;
  const int32_t n0 = a.lens[b];
  const int64_t n = n0 < 0 ? 0 : (uint64_t)n0 < held ? (int64_t)n0 : (int64_t)held, back = n - all;
  const uint32_t P = 1u << a.page_log2;
  const uint64_t page_size = (uint64_t)P * Page<BITS>::kToken;
  // a token's page of this head, or null
  auto page_at = [&](int64_t t) __attribute__((always_inline)) -> uint8_t* {
    if (t < 0 || (uint64_t)t >= held) return nullptr;
    const int32_t p = a.table[(uint64_t)b * a.width + ((uint32_t)t >> a.page_log2)];
    return (uint32_t)p < a.pages ? a.cache + ((uint64_t)p * a.heads + h) * page_size : nullptr;
  };
  constexpr int kEach = 4;  // drafts of a wavefront in a turn
  for (uint32_t i0 = 0; i0 < count; i0 += kEach * (kStepBlock / 64)) {
    uint64_t x[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const uint32_t i = i0 + kEach * wave + e;
      x[e] = lane >= 48u ? 0x80008000u : 0u;  // of a draft that is not there
      if (i < count) {
        const int64_t t = back + s_path[i];
        const uint8_t* p = page_at(t);
        if (p) {
          const Piece<BITS> s(P, (uint32_t)t & (P - 1u), lane);
          if (s.bytes == 8u) x[e] = *reinterpret_cast<const uint64_t*>(p + s.at);
          else if (s.bytes == 4u) x[e] = *reinterpret_cast<const uint32_t*>(p + s.at);
          else if (s.bytes == 2u) x[e] = *reinterpret_cast<const uint16_t*>(p + s.at);
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const uint32_t i = i0 + kEach * wave + e;
      if (i >= count || s_path[i] == (int32_t)i) continue;
      const int64_t t = back + i;
      uint8_t* p = page_at(t);
      if (!p) continue;
      const Piece<BITS> s(P, (uint32_t)t & (P - 1u), lane);
      if (s.bytes == 8u) *reinterpret_cast<uint64_t*>(p + s.at) = x[e];
      else if (s.bytes == 4u) *reinterpret_cast<uint32_t*>(p + s.at) = (uint32_t)x[e];
      else if (s.bytes == 2u) *reinterpret_cast<uint16_t*>(p + s.at) = (uint16_t)x[e];
    }
    __syncthreads();
  }
}

}  // namespace hq_kv

using namespace hq_kv;

extern "C" {

int hq_kv_reserve(const hq_kv_reserve_args* g, hq_stream_t stream) {
  if (!g || g->page < 16u || g->page > 4096u || (g->page & (g->page - 1u))) return HQ_ERR_INVALID_ARG;
  if (g->tokens > (1ull << 31) || g->pages > 0x7FFFFFFFu || (uint64_t)g->table_width * g->page > 0x7FFFFFFFull ||
      (uint64_t)g->seqs * g->table_width > 0x7FFFFFFFull || g->seqs > 0x7FFFFFFEu)
    return HQ_ERR_INVALID_ARG;
  if (!g->q_start || !g->free_count || (g->pages && !g->free) || (g->tokens && !g->slots)) return HQ_ERR_INVALID_ARG;
  if (g->seqs && (!g->lens || !g->counts || !g->granted || (g->table_width && !g->table))) return HQ_ERR_INVALID_ARG;
  if (((uintptr_t)g->table | (uintptr_t)g->lens | (uintptr_t)g->counts | (uintptr_t)g->free | (uintptr_t)g->free_count |
       (uintptr_t)g->positions | (uintptr_t)g->q_start | (uintptr_t)g->granted) & 3u)
    return HQ_ERR_INVALID_ARG;
  if ((uintptr_t)g->slots & 7u) return HQ_ERR_INVALID_ARG;
  ReserveArgs a;
  a.table = g->table;
  a.lens = g->lens;
  a.counts = g->counts;
  a.free = g->free;
  a.free_count = g->free_count;
  a.slots = g->slots;
  a.positions = g->positions;
  a.q_start = g->q_start;
  a.granted = g->granted;
  a.tokens = g->tokens;
  a.seqs = g->seqs;
  a.width = g->table_width;
  a.pages = g->pages;
  a.page_log2 = 31u - (uint32_t)__builtin_clz(g->page);
  // One launch or two, us a call: 512 tokens 8.2 and 10.1, 2048 8.7 and 10.2, 4096 9.9 and 10.2, 8192 12.0 and 10.2.
  a.here = g->tokens <= 4096;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  hipLaunchKernelGGL(reserve_kernel, dim3(1), dim3(kPlan), 0, st, a);
  if (!a.here) hipLaunchKernelGGL(slots_kernel, dim3((uint32_t)((a.tokens + kStepBlock - 1) / kStepBlock)), dim3(kStepBlock), 0, st, a);
  return hipGetLastError() == hipSuccess ? HQ_OK : HQ_ERR_HIP;
}

int hq_kv_accept(const hq_kv_cache* cache, const hq_kv_accept_args* g, hq_stream_t stream) {
  if (int rc = check_cache(cache)) return rc;
  if (!g || g->max_q > (uint32_t)kDrafts || g->total_q > (1ull << 31)) return HQ_ERR_INVALID_ARG;
  if ((uint64_t)g->table_width * cache->page > 0x7FFFFFFFull || (uint64_t)g->seqs * cache->heads > kMaxThreads / kStepBlock) return HQ_ERR_INVALID_ARG;
  if (!g->q_start && g->seqs && g->total_q % g->seqs) return HQ_ERR_INVALID_ARG;
  if (g->seqs == 0) return HQ_OK;
  if (!g->lens || !g->accepted || !g->next || !g->change || (g->max_q && !g->path) || (g->table_width && !g->table)) return HQ_ERR_INVALID_ARG;
  if (g->total_q && g->max_q && (!g->tokens || !g->target || !g->parents)) return HQ_ERR_INVALID_ARG;
  if (((uintptr_t)g->table | (uintptr_t)g->lens | (uintptr_t)g->q_start | (uintptr_t)g->tokens | (uintptr_t)g->target | (uintptr_t)g->parents |
       (uintptr_t)g->path | (uintptr_t)g->accepted | (uintptr_t)g->next | (uintptr_t)g->change) & 3u)
    return HQ_ERR_INVALID_ARG;
  AcceptArgs a;
  a.cache = static_cast<uint8_t*>(cache->data);
  a.table = g->table;
  a.lens = g->lens;
  a.q_start = g->q_start;
  a.tokens = g->tokens;
  a.target = g->target;
  a.parents = g->parents;
  a.path = g->path;
  a.accepted = g->accepted;
  a.next = g->next;
  a.change = g->change;
  a.total_q = g->total_q;
  a.seqs = g->seqs;
  a.heads = cache->heads;
  a.pages = cache->pages;
  a.page_log2 = 31u - (uint32_t)__builtin_clz(cache->page);
  a.width = g->table_width;
  a.max_q = g->max_q;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const dim3 grid(g->seqs * cache->heads), block(kStepBlock);
  if (cache->bits == 4) hipLaunchKernelGGL(accept_kernel<4>, grid, block, 0, st, a);
  else hipLaunchKernelGGL(accept_kernel<8>, grid, block, 0, st, a);
  return hipGetLastError() == hipSuccess ? HQ_OK : HQ_ERR_HIP;
}

}  // extern "C"
