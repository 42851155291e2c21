// The token table of the repetition, frequency and presence penalties: one
// int16 word per (request, token), sign bit = in the prompt, low 15 bits = the
// number of occurrences in the output, held at 32767.
//
// Build: a CTA per request, range of the vocabulary and part of the request's tokens
// keeps the range's counts (16 bits) and prompt bits in shared memory; the parts of a
// range are one cluster, whose CTAs add up the counts through distributed shared memory
// and write every word of the row once.  The tokens are read once per range, from L2.
// Updates of the table itself are far slower: one per token took 1162 us for 128
// requests of 1024 .. 131072 tokens, one per token and 4096 tokens (gathered in a hash
// table first) 45 us, because the updates of a frequent token queue up.
// Accept: one thread per token that the step has put out.
#include <algorithm>

#include "common.cuh"
#include "head.h"

namespace mtpsd {

constexpr int BUILD_THREADS = 1024;
constexpr int MAX_RANGE = 100352;             // tokens of a range: 196 KB of counts, 12 KB of bits
constexpr int MAX_PARTS = 8;
// Counts are cut to the limit after every 32768 tokens, so that none passes 32767 + 32768 before
constexpr int BLOCK = 32768;
constexpr int build_smem(int range) { return range * 2 + range / 8; }
static_assert(build_smem(MAX_RANGE) <= 232448 - 1024 && MAX_RANGE % 128 == 0, "shared memory per CTA");

// Adds n occurrences to the 16-bit word t of a row, held at 32767.  The words are updated through the
// aligned 32-bit word that holds two of them, by compare and swap, so that a count at its limit never
// carries into its neighbour; adding with a limit is order-independent.
__device__ __forceinline__ void add_word(int16_t* row, int64_t t, uint32_t n) {
  uint32_t* w = (uint32_t*)(row + (t & ~(int64_t)1));
  const int sh = (t & 1) ? 16 : 0;
  uint32_t old = *(volatile uint32_t*)w;
  for (;;) {
    const uint32_t v = (old >> sh) & 0xffffu;
    const uint32_t c = min((v & 0x7fffu) + n, 0x7fffu) | (v & 0x8000u);
    if (c == v) return;
    const uint32_t got = atomicCAS(w, old, (old & ~(0xffffu << sh)) | (c << sh));
    if (got == old) return;
    old = got;
  }
}

// The table row of request b, or -1: none, or outside the table.
__device__ __forceinline__ int64_t table_row(const int32_t* rows, int b, int n_rows, int32_t* status) {
  const int64_t row = rows ? rows[b] : b;
  if (row < -1 || row >= n_rows) {
    flag_status(status, MTPSD_STATUS_ROW_RANGE);
    return -1;
  }
  return row;
}

// The same for a whole CTA; -1 too for a row that an earlier request has (flagged).
__device__ __forceinline__ int64_t own_table_row(const int32_t* rows, int b, int n_rows, int32_t* status) {
  const int64_t row = table_row(rows, b, n_rows, threadIdx.x == 0 ? status : nullptr);
  bool taken = false;
  if (rows && row >= 0)
    for (int i = threadIdx.x; i < b; i += blockDim.x) taken = taken || rows[i] == row;
  if (__syncthreads_or(taken)) {
    if (threadIdx.x == 0) flag_status(status, MTPSD_STATUS_INDEX_RANGE);
    return -1;
  }
  return row;
}

__device__ __forceinline__ uint4 ld_peer(const void* p, uint32_t rank) {
  uint32_t a;
  uint4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_peer_u8(const void* p, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The two counts of a word, each cut to the limit.
__device__ __forceinline__ uint32_t limit2(uint32_t w) { return min(w & 0xffffu, 0x7fffu) | min(w >> 16, 0x7fffu) << 16; }

// Marks (PROMPT) or counts those of m tokens that lie in the range [base, base + span) of the vocabulary.  *high
// gathers the upper halves of the tokens and *most the largest lower half: the tokens outside the vocabulary show there.
// aligned: at is 16-byte aligned.
template <bool PROMPT>
__device__ __forceinline__ void scan(const int64_t* __restrict__ at, int m, bool aligned, uint32_t base, uint32_t span,
                                     uint32_t* cnt, uint32_t* seen, uint32_t* high, uint32_t* most) {
  auto take = [&](uint32_t lo) {
    const uint32_t c = lo - base;
    *most = max(*most, lo);
    if (c < span) {
      if (PROMPT) {
        atomicOr(&seen[c >> 5], 1u << (c & 31));   // looking first whether it is set: 36 us for the 128 requests, against 24
      } else {
        atomicAdd(&cnt[c >> 1], 1u << (c << 4 & 16));
      }
    }
  };
  auto single = [&](uint32_t lo, uint32_t hi) {
    *high |= hi;
    if (hi == 0) take(lo);
  };
  int done = 0;
  if (aligned) {
    constexpr int U = 4;                      // pairs of tokens a thread has on their way
    const uint4* two = (const uint4*)at + threadIdx.x;
    for (; done + 2 * U * BUILD_THREADS <= m; done += 2 * U * BUILD_THREADS, two += U * BUILD_THREADS) {
      uint4 t[U];
#pragma unroll
      for (int u = 0; u < U; ++u) t[u] = __ldg(two + u * BUILD_THREADS);
      uint32_t any = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) any |= t[u].y | t[u].w;
      if (any == 0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          take(t[u].x);
          take(t[u].z);
        }
      } else {
#pragma unroll 1
        for (int u = 0; u < U; ++u) {         // some token is no 32-bit number: read again, one by one
          const uint4 v = __ldg(two + u * BUILD_THREADS);
          single(v.x, v.y);
          single(v.z, v.w);
        }
      }
    }
  }
#pragma unroll 4
  for (int i = done + threadIdx.x; i < m; i += BUILD_THREADS) {
    const uint2 v = __ldg((const uint2*)at + i);
    single(v.x, v.y);
  }
}

__global__ void __launch_bounds__(BUILD_THREADS, 1) token_counts_build_kernel(
    const int64_t* __restrict__ tokens, int64_t S, const uint32_t* __restrict__ offsets,
    const int64_t* __restrict__ n_prompt, int64_t V, int16_t* __restrict__ counts, int64_t ld, int n_rows,
    const int32_t* __restrict__ rows, int range, int ranges, int parts, int32_t* status) {
  extern __shared__ __align__(16) uint32_t smem[];
  uint32_t* cnt = smem;                       // [range / 2]: two counts a word
  uint32_t* seen = smem + range / 2;          // [range / 32]: tokens of the prompt
  const int tid = threadIdx.x;
  const int part = (int)(blockIdx.x % parts), which = (int)(blockIdx.x / parts % ranges), b = (int)(blockIdx.x / parts / ranges);
  for (int i = tid; i < build_smem(range) / 16; i += BUILD_THREADS) ((uint4*)smem)[i] = make_uint4(0, 0, 0, 0);
  griddep_wait();                // the previous kernel's writes are visible from here on
  griddep_launch_dependents();
  const bool first_cta = which == 0 && part == 0;
  const int64_t row = own_table_row(rows, b, n_rows, first_cta ? status : nullptr);
  const int64_t first = offsets[b], stop = offsets[b + 1], end = min(stop, S);
  if (first_cta && tid == 0 && stop > S) flag_status(status, MTPSD_STATUS_ROW_RANGE);
  if (row < 0) return;           // the whole cluster
  const int64_t n = max(end - first, (int64_t)0), cut = n_prompt ? first + min(max(n_prompt[b], (int64_t)0), n) : end;
  const int64_t j0 = first + n * part / parts, j1 = first + n * (part + 1) / parts;
  const int64_t base = (int64_t)which * range;
  __syncthreads();
  const uint32_t base32 = (uint32_t)base, span = (uint32_t)min((int64_t)range, V - base);      // V < 2^31
  const bool pairs = (uintptr_t)tokens % 16 == 0;
  bool counted = false;                       // outputs since the counts were cut
  uint32_t high = 0, most = 0;                // tokens outside the vocabulary show in them
  // The tokens of the block that starts at `at` on their way into L2, by the request's first range: a CTA's own loads
  // keep 64 KB in flight, so that from memory the longest request set the pace (128 requests on cold tokens: 41 us)
  auto prefetch = [&](int64_t at) {
    if (which != 0 || tid != 0 || at >= j1) return;
    const uintptr_t lo = ((uintptr_t)(tokens + at) + 15) & ~(uintptr_t)15, hi = (uintptr_t)(tokens + min(at + BLOCK, j1)) & ~(uintptr_t)15;
    if (lo < hi)
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(__cvta_generic_to_global((const void*)lo)), "r"((uint32_t)(hi - lo)) : "memory");
  };
  prefetch(j0);
  prefetch(j0 + BLOCK);
  for (int64_t block = j0; block < j1; block += BLOCK) {
    const int64_t stop_at = min(block + BLOCK, j1);
    prefetch(block + 2 * BLOCK);
    const int m = (int)(stop_at - block), before = (int)min(max(cut - block, (int64_t)0), (int64_t)BLOCK);
    if (counted) {
      __syncthreads();
      for (int i = tid; i < range / 8; i += BUILD_THREADS) {
        uint4 v = ((uint4*)cnt)[i];
        v.x = limit2(v.x); v.y = limit2(v.y); v.z = limit2(v.z); v.w = limit2(v.w);
        ((uint4*)cnt)[i] = v;
      }
      __syncthreads();
    }
    counted = before < m;
    // the block's prompt tokens, then its outputs
    if (before > 0) scan<true>(tokens + block, min(before, m), pairs && block % 2 == 0, base32, span, cnt, seen, &high, &most);
    if (before < m)
      scan<false>(tokens + block + before, m - before, pairs && (block + before) % 2 == 0, base32, span, cnt, seen, &high, &most);
  }
  if (which == 0 && (high != 0 || most >= (uint64_t)V)) flag_status(status, MTPSD_STATUS_INDEX_RANGE);
  // the words of this CTA's share of the range: eight a thread and step
  if (parts > 1) cluster_sync();
  else __syncthreads();
  const int64_t width = min((int64_t)range, ld - base);            // <= 0: a range past the row
  const int g0 = (int)(max(width, (int64_t)0) / 8 * part / parts), g1 = (int)(max(width, (int64_t)0) / 8 * (part + 1) / parts);
  auto word8 = [&](int g, const uint4* v, const uint32_t* k, int most) {
    uint32_t sum[4] = {0, 0, 0, 0}, bits = 0;
#pragma unroll
    for (int r = 0; r < MAX_PARTS; ++r) {
      if (r >= most || r >= parts) break;
      const uint32_t c[4] = {v[r].x, v[r].y, v[r].z, v[r].w};
      bits |= k[r];
      // each half at most 32767 before and after, so that a sum stays within 16 bits
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] = limit2(sum[e] + limit2(c[e]));
    }
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = sum[e] | (bits >> (2 * e) & 1u) << 15 | (bits >> (2 * e + 1) & 1u) << 31;
    *(uint4*)(counts + row * ld + base + 8 * (int64_t)g) = make_uint4(w[0], w[1], w[2], w[3]);
  };
  if (parts == 1) {
    for (int g = tid; g < g1; g += BUILD_THREADS) {
      const uint4 v = ((const uint4*)cnt)[g];
      const uint32_t k = ((const uint8_t*)seen)[g];
      word8(g, &v, &k, 1);
    }
  } else {
    for (int g = g0 + tid; g < g1; g += BUILD_THREADS) {
      uint4 v[MAX_PARTS];
      uint32_t k[MAX_PARTS];
#pragma unroll
      for (int r = 0; r < MAX_PARTS; ++r) {   // every part's words on their way at once
        if (r >= parts) break;
        v[r] = r == part ? ((const uint4*)cnt)[g] : ld_peer((const uint4*)cnt + g, r);
        k[r] = r == part ? ((const uint8_t*)seen)[g] : ld_peer_u8((const uint8_t*)seen + g, r);
      }
      word8(g, v, k, MAX_PARTS);
    }
  }
  // a row wider than the vocabulary: zeros
  if (which == ranges - 1)
    for (int64_t c = (int64_t)ranges * range + 8 * (part * BUILD_THREADS + tid); c < ld; c += 8 * (int64_t)parts * BUILD_THREADS)
      *(uint4*)(counts + row * ld + c) = make_uint4(0, 0, 0, 0);
  if (parts > 1) cluster_sync();              // no CTA leaves while another reads its counts
}

__global__ void __launch_bounds__(256) token_counts_accept_kernel(const int64_t* __restrict__ draft,
                                                                  const int32_t* __restrict__ n_acc,
                                                                  const int64_t* __restrict__ next, int B, int K,
                                                                  int64_t V, int16_t* __restrict__ counts, int64_t ld,
                                                                  int n_rows, const int32_t* __restrict__ rows,
                                                                  int32_t* status) {
  griddep_wait();                // the previous kernel's writes are visible from here on
  griddep_launch_dependents();
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int b = (int)(i / (K + 1)), j = (int)(i % (K + 1));
  if (b >= B) return;
  if (j < K && j >= n_acc[b]) return;
  const int64_t row = table_row(rows, b, n_rows, status);
  if (row < 0) return;
  const int64_t t = j < K ? draft[(int64_t)b * K + j] : next[b];
  if (t < 0 || t >= V) flag_status(status, MTPSD_STATUS_INDEX_RANGE);
  else add_word(counts + row * ld, t, 1);
}

int launch_token_counts_build(const int64_t* tokens, int64_t S, const uint32_t* offsets, const int64_t* n_prompt, int B,
                              int64_t V, int16_t* counts, int64_t ld, int n_rows, const int32_t* rows, int32_t* status,
                              cudaStream_t st) {
  static std::atomic<uint64_t> attr;
  if (!set_smem_limit_once(token_counts_build_kernel, build_smem(MAX_RANGE), attr)) {
    set_error("token_counts_build: cudaFuncSetAttribute failed");
    return MTPSD_ECUDA;
  }
  const int ranges = (int)ceil_div(V, MAX_RANGE);
  const int range = (int)(ceil_div(ceil_div(V, ranges), 128) * 128);
  // parts of a request's tokens: while every part finds an SM of its own and has 4096 tokens (joining the parts costs
  // about 10000 cycles: 128 requests on two parts took 45 us)
  int parts = 1;
  while (parts < MAX_PARTS && (int64_t)B * ranges * parts * 2 <= num_sms() && S / (2 * parts) >= 4096) parts *= 2;
  const int64_t grid = (int64_t)B * ranges * parts;
  if (grid > 0x7fffffffLL) {
    set_error("token_counts_build: too many requests for this vocabulary");
    return MTPSD_EUNSUPPORTED;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(BUILD_THREADS);
  cfg.dynamicSmemBytes = build_smem(range);
  cfg.stream = st;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = parts;
  attrs[1].val.clusterDim.y = 1;
  attrs[1].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = parts > 1 ? 2 : 1;
  cudaLaunchKernelEx(&cfg, token_counts_build_kernel, tokens, S, offsets, n_prompt, V, counts, ld, n_rows, rows, range, ranges,
                     parts, status);
  return check_launch("token_counts_build");
}

int launch_token_counts_accept(const int64_t* draft, const int32_t* n_acc, const int64_t* next, int B, int K, int64_t V,
                               int16_t* counts, int64_t ld, int n_rows, const int32_t* rows, int32_t* status,
                               cudaStream_t st) {
  const int64_t n = (int64_t)B * (K + 1);
  launch_k(token_counts_accept_kernel, (unsigned)ceil_div(n, 256), 256, 0, st, draft, n_acc, next, B, K, V, counts, ld,
           n_rows, rows, status);
  return check_launch("token_counts_accept");
}

}  // namespace mtpsd
