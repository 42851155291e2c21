// Penalties, biases and the grammar mask on the verify rows' logits, the greedy
// token and the target distribution ([P1] "阶段 3:拒绝采样与 Bitmask").
//
// Memory bound: every logit is read once and every probability written once.  A
// cluster of 1, 2, 4 or 8 CTAs works on one row at a time, each CTA on a chunk of
// the vocabulary; the launch has as many clusters as run at once, and each takes an
// equal run of consecutive rows.
// For a request (its rows share the table row, the biases and the drafts):
// 1. The chunk's table words are scanned once: a bitmap and a list of the tokens
//    with a word (about 1 in 100).  Looking at the words in every row, and computing
//    the penalties where they were found, cost 29 instructions per token (768 rows of
//    154880 bf16 logits, argmax only: 166 us).
// 2. The tokens of the drafts and the biases are put down with their words.
// For a row:
// 3. One bulk copy brings the chunk's logits into shared memory (rows that are not
//    16-byte aligned: element copies); the next row's are prefetched into L2.
// 4. The row's drafts and the biases are marked in a second bitmap.
// 5. The chunk streams through, 16 bytes of logits per thread and step: -inf where
//    the mask bit is 0; every thread keeps its largest group of values, without the
//    tokens of either bitmap.  Those follow, one per thread.
// 6. The chunk's largest value m_c (and its lowest position) and, over shared
//    memory, s_c = sum exp((x - m_c) / T) are exchanged within the cluster once
//    (each CTA stores its three words into the others' shared memory): the row's
//    maximum is m = max m_c and its sum s = sum_c s_c exp((m_c - m) / T).
// 7. The chunk's probabilities exp((x - m_c) / T) * (exp((m_c - m) / T) / s) are written.
// All values, the maximum and the sums are float32; the sums add at most chunk /
// 256 values per thread before the tree, in an order fixed by the sizes.  The
// exponentials are 2^y, y = (x - m_c) (log2 e / T): three roundings and the constant's own, 3 2^-24 + 2^-26.2 < 2^-22.3 of
// its value where log2 e / T is a normal float (T of 1e-38 .. 1e38).
// Every mbarrier wait is bounded (2 s): on expiry the kernel flags MTPSD_STATUS_WAIT_TIMEOUT, the cluster leaves its rows
// from there on, and each CTA waits for its copies in flight before it returns.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "head.h"
#include "head_wait.cuh"

namespace mtpsd {
namespace lgt {

constexpr int MAX_CHUNK = 49152;              // 192 KB of values
constexpr int MAX_CLUSTER = 8;
static_assert((int64_t)MAX_CHUNK * MAX_CLUSTER == 393216, "the vocabulary that the call allows");
static_assert(MAX_CHUNK <= 65536, "list entries hold 16-bit positions");
constexpr int LIST = 2048;                    // tokens with a table word in the list (with more, the bitmap is walked)
constexpr int ENTRIES = 512;                  // drafts and biases put down in shared memory (more are read again)
constexpr int REPEATS = 64;                   // entries of a row whose token another entry has too (with more, every entry counts as one)

// shared memory: list, entries (position, word, bias), the two bitmaps, the row's mask, the logits or values
constexpr int OFF_ENT = LIST * 4;
constexpr int OFF_BITS = OFF_ENT + ENTRIES * 12;
constexpr int smem_bytes(int chunk, int per_token) { return OFF_BITS + chunk / 8 * 3 + chunk * per_token; }
static_assert(smem_bytes(MAX_CHUNK, 4) <= 232448 - 1024, "shared memory per CTA");

struct Params {
  mtpsd_logits_args a;
  int chunk;              // tokens per CTA (a multiple of 128)
  int cluster;            // CTAs per row
  int vec_in;             // logits rows are 16-byte aligned
  int vec_out;            // out_logits rows can be written 16 bytes at a time
  int vec_probs;          // probs rows likewise
};

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// the same of two bf16 pairs
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Each byte of the result is the sign of one byte of v, spread over it (selector nibble: 8 + that byte).
template <int SEL>
__device__ __forceinline__ uint32_t sign_bytes(uint32_t v) {
  uint32_t r;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(v), "n"(SEL));
  return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The barriers of the exchange exist before a peer stores into this CTA (their initialisation was released by
// fence.mbarrier_init).
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t saddr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint32_t map_rank(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ float exp2_fast(float y) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
  return r;
}

// The request of the current rows; in shared memory.
struct Request {
  const uint16_t* word;     // table row or NULL
  const int64_t* draft;
  const int32_t* bt;
  const float* bv;
  int K, nb;                // drafts, biases
  float rep, freq, pres, temp;
};

// The penalties of a token with table word w and `extra` more outputs (each step rounded to float32, as documented).
__device__ __noinline__ float penalise(const Request* r, float x, uint32_t w, int extra) {
  const int n = (int)(w & 32767u) + extra;
  if ((w & 32768u) || n > 0) x = x > 0.f ? __fdiv_rn(x, r->rep) : __fmul_rn(x, r->rep);
  if (n > 0) x = __fsub_rn(__fsub_rn(x, __fmul_rn(r->freq, (float)n)), r->pres);
  return x;
}

// THREADS: 384 with two CTAs per SM (a row's reductions and barriers cost every warp the same: 768 rows of 154880, argmax
// only, take 104 us, with 512 threads 112 and with 256 120), or 256 with four for short chunks.
template <bool BF16, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? 4 : 2) process_logits_kernel(const __grid_constant__ Params p) {
  constexpr int WARPS = THREADS / 32;
  constexpr int G = 8;                    // tokens per thread and step: a byte of each bitmap
  constexpr int ES = BF16 ? 2 : 4;
  constexpr uint32_t ALL = (1u << G) - 1;
  const mtpsd_logits_args& a = p.a;
  extern __shared__ __align__(16) char smem[];
  __shared__ Request R;
  __shared__ float s_red[WARPS];
  __shared__ unsigned s_idx;
  __shared__ int s_rep[REPEATS], s_reps, s_list;
  __shared__ int s_abort, s_told;                          // a wait of this CTA has expired; the CTA leaves
  __shared__ __align__(16) float4 s_peer[2][MAX_CLUSTER];   // (maximum, sum, position) of every CTA, by the row's parity
  __shared__ float4 s_row;                                  // the row's (maximum, sum, position)
  __shared__ __align__(8) uint64_t s_bar[2], s_in;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = p.cluster > 1 ? cluster_rank() : 0;
  uint32_t* list = (uint32_t*)smem;                    // position in the chunk | table word << 16
  int32_t* ent_pos = (int32_t*)(smem + OFF_ENT);       // drafts, then biases: position in the chunk, -1 outside it
  uint32_t* ent_word = (uint32_t*)ent_pos + ENTRIES;
  float* ent_bias = (float*)ent_word + ENTRIES;
  uint32_t* skip = (uint32_t*)(smem + OFF_BITS);       // [chunk / 32]: tokens that the stream leaves out: those with a
                                                       // table word and the row's marked ones
  uint32_t* marks = skip + p.chunk / 32;               // [chunk / 32]: tokens of the row's drafts and the biases
  uint32_t* mask = marks + p.chunk / 32;               // [chunk / 32]: the row's mask
  float* xs = (float*)(mask + p.chunk / 32);           // [chunk]
  // the logits as they come: float32 in place; bf16 in the upper half of xs (widened step by step: a step's float32
  // end at or below where the next step's bf16 begin), or alone when no probabilities are wanted
  char* raw = (char*)xs + (BF16 && a.probs ? p.chunk * 2 : 0);
  const int64_t start = (int64_t)rank * p.chunk;
  const int len = (int)max((int64_t)0, min((int64_t)p.chunk, a.V - start));
  const int bulk = p.vec_in ? len * ES & ~15 : 0;
  if (tid == 0) {
    s_abort = 0;
    s_told = 0;
    for (int i = 0; i < 2; ++i) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(saddr(&s_bar[i])));
      expect_tx(&s_bar[i], p.cluster * 16);
    }
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(saddr(&s_in)));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  for (int i = tid; i < p.chunk / 16; i += THREADS) skip[i] = 0;    // marks too
  griddep_wait();                // the previous kernel's writes are visible from here on
  griddep_launch_dependents();
  // this cluster's rows: an equal run of those of the requests (rows behind the last one stay as they are)
  const int64_t row0 = a.row_offsets[0], row_end = min((int64_t)a.row_offsets[a.B], (int64_t)a.R);
  const int64_t n_rows = max(row_end - row0, (int64_t)0);
  const int64_t clusters = gridDim.x / p.cluster, me = blockIdx.x / p.cluster;
  const int64_t r0 = row0 + me * n_rows / clusters, r1 = row0 + (me + 1) * n_rows / clusters;
  if ((int64_t)a.row_offsets[a.B] > a.R && blockIdx.x == 0 && tid == 0) flag_status(a.dev_status, MTPSD_STATUS_ROW_RANGE);
  if (r0 >= r1) return;          // the whole cluster
  if (p.cluster > 1) {
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  }

  auto source = [&](int64_t r) { return (const char*)a.logits + (r * a.ld + start) * ES; };
  // the chunk of row r, with its mask, into shared memory
  auto stage = [&](int64_t r, const uint8_t* rm) {
    const char* src = source(r);
    if (tid == 0) {
      expect_tx(&s_in, bulk);
      if (bulk)
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(saddr(raw)),
                     "l"((uint64_t)src), "r"(bulk), "r"(saddr(&s_in))
                     : "memory");
    }
    if (rm)
      for (int i = tid; i < (len + 31) / 32; i += THREADS)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(saddr(mask + i)), "l"((uint64_t)(rm + 4 * i)) : "memory");
    // what the bulk copy leaves: the last elements, or all of an unaligned row
    if constexpr (BF16) {
#pragma unroll 8
      for (int c = bulk / ES + tid; c < len; c += THREADS) ((uint16_t*)raw)[c] = ((const uint16_t*)src)[c];
    } else {
      for (int c = bulk / ES + tid; c < len; c += THREADS)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(saddr((float*)raw + c)), "l"((uint64_t)(src + 4 * c))
                     : "memory");
    }
  };
  auto staged = [&](int c) -> float {
    return BF16 ? __bfloat162float(((const __nv_bfloat16*)raw)[c]) : ((const float*)raw)[c];
  };
  auto bit = [](const uint32_t* m, int c) { return (m[c >> 5] >> (c & 31) & 1) != 0; };

  // the chunk's part of mask m, or NULL
  auto mask_at = [&](int64_t m) -> const uint8_t* {
    if (!a.bitmask) return nullptr;
    if (m >= 0 && m < a.n_masks) return (const uint8_t*)(a.bitmask + m * ((a.V + 31) / 32)) + (start >> 3);
    if (m != -1 && rank == 0 && tid == 0) flag_status(a.dev_status, MTPSD_STATUS_ROW_RANGE);
    return nullptr;
  };
  auto mask_index = [&](int64_t r) -> int64_t { return a.mask_rows ? (int64_t)a.mask_rows[r] : r; };
  int b = request_of_row_warp(a.row_offsets, a.B, (uint32_t)r0);
  int64_t first_row = 0, next_row = 0;                 // of the request, of the next one
  const uint16_t* next_word = nullptr;                 // its table row
  const uint8_t* rm_next = mask_at(a.bitmask ? mask_index(r0) : -1);
  int parity = 0, in_phase = 0, bar_phase = 0, entries = 0;
  const int steps = (len + THREADS * G - 1) / (THREADS * G);
  stage(r0, rm_next);
  for (int64_t r = r0; r < r1; ++r) {
    if (r >= next_row) {
      while (r >= (int64_t)a.row_offsets[b + 1]) ++b;  // r < row_offsets[B]
      // ---- the request
      if (warp == 0) {           // the request's numbers in one round of loads, a lane each
        int64_t v = 0;
        if (lane == 0) v = a.count_rows ? a.count_rows[b] : b;
        if (lane == 1 && a.bias_offsets) v = a.bias_offsets[b];
        if (lane == 2 && a.bias_offsets) v = a.bias_offsets[b + 1];
        float f = lane == 5 || lane == 6 ? 0.f : 1.f;
        const float* src = lane == 4 ? a.repetition : lane == 5 ? a.frequency : lane == 6 ? a.presence : lane == 7 ? a.temperature : nullptr;
        if (src) f = src[b];
        const int64_t row = __shfl_sync(0xffffffffu, v, 0), lo = __shfl_sync(0xffffffffu, v, 1);
        const int64_t hi = __shfl_sync(0xffffffffu, v, 2), end = min(hi, (int64_t)a.n_bias);
        const float rep = __shfl_sync(0xffffffffu, f, 4), freq = __shfl_sync(0xffffffffu, f, 5);
        const float pres = __shfl_sync(0xffffffffu, f, 6), temp = __shfl_sync(0xffffffffu, f, 7);
        if (lane == 0) {
          R.word = nullptr;
          if (a.counts) {
            if (row >= 0 && row < a.counts_rows) R.word = (const uint16_t*)a.counts + row * a.counts_ld;
            else if (row != -1 && rank == 0) flag_status(a.dev_status, MTPSD_STATUS_ROW_RANGE);
          }
          R.draft = a.draft ? a.draft + (int64_t)b * a.K : nullptr;
          R.K = a.draft ? a.K : 0;
          if (a.bias_offsets && hi > a.n_bias && rank == 0) flag_status(a.dev_status, MTPSD_STATUS_INDEX_RANGE);
          R.bt = a.bias_tokens + lo;
          R.bv = a.bias_values + lo;
          R.nb = a.bias_offsets && end > lo ? (int)(end - lo) : 0;
          R.rep = rep;
          R.freq = freq;
          R.pres = pres;
          R.temp = temp;
          s_list = 0;
        }
      }
      __syncthreads();
      entries = R.K + R.nb;
      const uint16_t* w = R.word;
      first_row = (int64_t)a.row_offsets[b];
      next_row = (int64_t)a.row_offsets[b + 1];
      next_word = nullptr;
      if (a.counts && next_row < r1) {
        const int64_t row = a.count_rows ? a.count_rows[b + 1] : b + 1;
        if (row >= 0 && row < a.counts_rows) next_word = (const uint16_t*)a.counts + row * a.counts_ld;
      }
      auto token = [&](int e) { return e < R.K ? R.draft[e] : (int64_t)R.bt[e - R.K]; };
      const int64_t t0 = tid < entries ? token(tid) : 0;     // on its way during the scan
      if (w) {
        // eight words per thread and step: one byte of the bitmap (a row's words reach past V to a multiple of 8)
        constexpr int U = 5;
        for (int g0 = tid; g0 - lane < (len + 7) / 8; g0 += U * THREADS) {
          uint4 k[U];
          uint32_t nz[U];
          int n = 0;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int g = g0 + u * THREADS;
            k[u] = 8 * g < len ? *(const uint4*)(w + start + 8 * g) : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int g = g0 + u * THREADS;
            const uint32_t kk[4] = {k[u].x, k[u].y, k[u].z, k[u].w};
            nz[u] = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // bit 15 of each half where its 16 bits are not all zero
              const uint32_t h = ((kk[e] & 0x7fff7fffu) + 0x7fff7fffu) | kk[e];
              nz[u] |= (h >> 15 & 1u | h >> 30 & 2u) << 2 * e;
            }
            if (len - 8 * g < 8) nz[u] &= len > 8 * g ? (1u << (len - 8 * g)) - 1 : 0u;
            if (8 * g < p.chunk) ((uint8_t*)skip)[g] = (uint8_t)nz[u];
            n += __popc(nz[u]);
          }
          int before = n;                              // places in the list: a scan over the warp, one addition for it
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += y;
          }
          const int all = __shfl_sync(0xffffffffu, before, 31);
          int at = 0;
          if (lane == 0 && all) at = atomicAdd(&s_list, all);
          at = __shfl_sync(0xffffffffu, at, 0) + before - n;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            while (nz[u]) {
              const int e = __ffs(nz[u]) - 1;
              const uint32_t pair = e < 4 ? (e < 2 ? k[u].x : k[u].y) : (e < 6 ? k[u].z : k[u].w);
              if (at < LIST) list[at] = (uint32_t)(8 * (g0 + u * THREADS) + e) | (e & 1 ? pair >> 16 : pair & 0xffffu) << 16;
              ++at;
              nz[u] &= nz[u] - 1;
            }
          }
        }
      }
      else {
        for (int i = tid; i < p.chunk / 32; i += THREADS) skip[i] = 0;
      }
      for (int e = tid; e < entries; e += THREADS) {
        const int64_t t = e == tid ? t0 : token(e), c = t - start;
        const bool in = c >= 0 && c < len;
        if ((t < 0 || t >= a.V) && rank == 0) flag_status(a.dev_status, MTPSD_STATUS_INDEX_RANGE);
        if (e < ENTRIES) {
          ent_pos[e] = in ? (int)c : -1;
          ent_word[e] = in && w ? w[t] : 0u;
          ent_bias[e] = e < R.K ? 0.f : R.bv[e - R.K];
        }
      }
    }
    const uint16_t* const rw = R.word;
    const uint8_t* const rm = rm_next;
    const int nd = (int)min(r - first_row, (int64_t)R.K);    // drafts that the row follows
    const float temp = R.temp;
    const bool onehot = !(temp > 0.f);
    const bool keep = a.probs != nullptr && !onehot;   // the values stay in shared memory for the probabilities
    float* out = a.out_logits ? a.out_logits + r * a.out_ld + start : nullptr;
    const bool special = nd + R.nb > 0;
    if (tid == 0) {
      s_idx = 0xffffffffu;
      s_reps = 0;
      if (r + 1 < r1 && bulk)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"((uint64_t)source(r + 1)), "r"(bulk) : "memory");
    }
    const int64_t mask_next = a.bitmask && r + 1 < r1 ? mask_index(r + 1) : -1;      // used after the stream
    if (r + 1 < r1) {            // the logits of unaligned rows too, and a new request's words
      if (!bulk && len > 0)
        for (int i = tid * 128; i < len * ES; i += THREADS * 128)
          asm volatile("prefetch.global.L2 [%0];" ::"l"((uint64_t)(source(r + 1) + i)));
      if (r + 1 >= next_row && next_word)
        for (int i = tid * 64; i < len; i += THREADS * 64)
          asm volatile("prefetch.global.L2 [%0];" ::"l"((uint64_t)(next_word + start + i)));
    }
    __syncthreads();
    // position of entry e, -1: not in the chunk or not one of this row's
    auto position = [&](int e) -> int {
      if (e >= nd && e < R.K) return -1;
      if (e < ENTRIES) return ent_pos[e];
      const int64_t c = (e < R.K ? R.draft[e] : (int64_t)R.bt[e - R.K]) - start;
      return c >= 0 && c < len ? (int)c : -1;
    };
    if (special) {
      for (int e = tid; e < entries; e += THREADS) {
        const int c = position(e);
        if (c < 0) continue;
        if (atomicOr(&marks[c >> 5], 1u << (c & 31)) >> (c & 31) & 1) {
          const int i = atomicAdd(&s_reps, 1);
          if (i < REPEATS) s_rep[i] = c;
        }
        atomicOr(&skip[c >> 5], 1u << (c & 31));
      }
    }
    // the thread's largest value: of the step's group at bg (-1: none yet), or of a single token (si: its position + 1, as
    // in s_idx: 0 is an expired wait)
    float best = -INFINITY, sbest = -INFINITY;
    int bg = -1;
    unsigned si = 0xffffffffu;
    auto open = [&](int c) { return !rm || bit(mask, c); };
    auto single = [&](int c, float x) {                // a token computed on its own
      if (!open(c)) x = -INFINITY;
      const unsigned t = (unsigned)(start + c) + 1;
      if (keep) xs[c] = x;
      if (out) out[c] = x;
      // NaN above everything, then the larger value, then the lower position
      const bool above = x != x ? !(sbest != sbest) || t < si : x > sbest || (x == sbest && t < si);
      if (above) {
        sbest = x;
        si = t;
      }
    };

    // ---- the chunk
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (warp == 0 && !mbar::wait_head<false>(&s_in, in_phase, &s_abort, a.dev_status)) {
      mbar::drain<false>(&s_in, in_phase, a.dev_status);     // nothing of the copy is in flight when the CTA leaves
      if (p.cluster == 1) s_told = 1;
    }
    in_phase ^= 1;
    __syncthreads();                                   // the chunk is staged, the marks are set
    // When a wait of a CTA has expired, here or in the exchange of the row before, the CTA goes through the row with what is
    // there but stores nothing, and the exchange tells the cluster: none of its CTAs stores the row's argmax and
    // probabilities, and all leave here in the next row, with no copy of theirs and no peer's values in flight.  (Leaving
    // behind the exchange took 107.7 us for 768 rows of 154880, argmax only, where 106.0 are reached and 105.8 without any
    // of this.)
    if (__builtin_expect(s_told, 0)) return;
    if (out && s_abort) out = nullptr;
#pragma unroll 2
    for (int s = 0; s < steps; ++s) {
      const int c = (s * THREADS + tid) * G;
      // the group's logits: eight float32, or four pairs of bf16
      uint32_t v[ES * 2];
#pragma unroll
      for (int i = 0; i < ES / 2; ++i) {
        const uint4 k = c < len ? *(const uint4*)(raw + c * ES + 16 * i) : make_uint4(0, 0, 0, 0);
        v[4 * i] = k.x; v[4 * i + 1] = k.y; v[4 * i + 2] = k.z; v[4 * i + 3] = k.w;
      }
      if (BF16 && keep) __syncthreads();             // to widen: every thread has read the step before any writes it
      if (c >= len) continue;
      const uint32_t sp = ((const uint8_t*)skip)[c >> 3];      // these come later, one by one
      uint32_t mk = rm ? ((const uint8_t*)mask)[c >> 3] : ALL;
      if (len - c < G) mk &= (1u << (len - c)) - 1;  // whatever lies past the end counts as masked
      auto strike = [&](uint32_t left) {             // -inf where the bit is 0
        // the bits at the tops of bytes, spread over the values by byte permutes that replicate a sign
        const uint32_t lo = (left & 15u) * 0x10204080u, hi = (left >> 4) * 0x10204080u;
        if constexpr (BF16) {
          const uint32_t m[4] = {sign_bytes<0x9988>(lo), sign_bytes<0xbbaa>(lo), sign_bytes<0x9988>(hi),
                                 sign_bytes<0xbbaa>(hi)};
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = (v[i] & m[i]) | (0xff80ff80u & ~m[i]);
        } else {
          const uint32_t m[8] = {sign_bytes<0x8888>(lo), sign_bytes<0x9999>(lo), sign_bytes<0xaaaa>(lo),
                                 sign_bytes<0xbbbb>(lo), sign_bytes<0x8888>(hi), sign_bytes<0x9999>(hi),
                                 sign_bytes<0xaaaa>(hi), sign_bytes<0xbbbb>(hi)};
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = (v[i] & m[i]) | (0xff800000u & ~m[i]);
        }
      };
      const bool stay = keep || out != nullptr;      // the masked values are wanted, not only the maximum
      if (stay && mk != ALL) strike(mk);
      auto value8 = [&](int e) { return __uint_as_float(!BF16 ? v[e] : (e & 1) ? v[e / 2] & 0xffff0000u : v[e / 2] << 16); };
      if (keep && (BF16 || mk != ALL)) {
#pragma unroll
        for (int e = 0; e < G; e += 4)
          *(float4*)(xs + c + e) = make_float4(value8(e), value8(e + 1), value8(e + 2), value8(e + 3));
      }
      if (out && p.vec_out) {
        if (!sp && c + G <= len) {
#pragma unroll
          for (int e = 0; e < G; e += 4)
            *(float4*)(out + c + e) = make_float4(value8(e), value8(e + 1), value8(e + 2), value8(e + 3));
        } else {
#pragma unroll
          for (int e = 0; e < G; ++e)
            if (!(sp >> e & 1) && c + e < len) out[c + e] = value8(e);
        }
      }
      const uint32_t left = stay ? ~sp & ALL : ~sp & mk;
      if (left != ALL) strike(left);
      float gm;
      if constexpr (BF16) {
        const uint32_t h = max_nan2(max_nan2(v[0], v[1]), max_nan2(v[2], v[3]));
        gm = max_nan(__uint_as_float(h << 16), __uint_as_float(h & 0xffff0000u));
      } else {
        gm = __uint_as_float(v[0]);
#pragma unroll
        for (int e = 1; e < G; ++e) gm = max_nan(gm, __uint_as_float(v[e]));
      }
      if (!(gm <= best) && best == best) {           // the first group with the largest value; a NaN stays
        best = gm;
        bg = c;
      }
    }
    rm_next = mask_at(mask_next);
    const bool later = out && !p.vec_out;              // out_logits rows that cannot be written 16 bytes at a time
    if (rw || special || later) {
      __syncthreads();                                 // the stream's values are written
      auto value = [&](int c) { return keep ? xs[c] : staged(c); };
      // consecutive threads write consecutive tokens (a thread's eight one by one: 76 us for 68 rows of 50001 from memory)
      if (later)
        for (int c = tid; c < len; c += THREADS)
          if (!bit(skip, c)) out[c] = keep || open(c) ? value(c) : -INFINITY;
      if (rw) {
        const int n = s_list;
        if (n <= LIST) {
          for (int i = tid; i < n; i += THREADS) {
            const int c = (int)(list[i] & 0xffffu);
            if (!bit(marks, c)) single(c, penalise(&R, value(c), list[i] >> 16, 0));
          }
        } else {
          for (int i = tid; i < (len + 31) / 32; i += THREADS) {
            uint32_t left = skip[i] & ~marks[i];
            while (left) {
              const int c = 32 * i + __ffs(left) - 1;
              left &= left - 1;
              single(c, penalise(&R, value(c), rw[start + c], 0));
            }
          }
        }
      }
      if (special) {
        const int reps = s_reps;
        const bool all = reps > REPEATS;
        auto word = [&](int e, int c) { return e < ENTRIES ? ent_word[e] : rw ? (uint32_t)rw[start + c] : 0u; };
        auto bias = [&](int e) { return e < ENTRIES ? ent_bias[e] : R.bv[e - R.K]; };
        for (int e = THREADS - 1 - tid; !all && e < entries; e += THREADS) {     // from the last warps: the first have the list
          const int c = position(e);
          bool repeated = c < 0;
          for (int i = 0; i < reps; ++i) repeated = repeated || s_rep[i] == c;
          if (repeated) continue;
          float x = penalise(&R, value(c), word(e, c), e < R.K ? 1 : 0);
          if (e >= R.K) x = __fadd_rn(x, bias(e));
          single(c, x);
        }
        // a token with several entries: a warp looks through them (300 biases with one pair among them, a thread
        // each through all of them: 70 us instead of 23 for the 68 rows of 50001)
        auto candidate = [&](int i) { return all ? position(i) : s_rep[i]; };
        for (int i = warp; i < (all ? entries : reps); i += WARPS) {
          const int c = candidate(i);
          bool again = c < 0;
          for (int k = lane; k < i; k += 32) again = again || candidate(k) == c;
          if (__any_sync(0xffffffffu, again)) continue;
          int extra = 0, first = entries;
          for (int k = lane; k < nd; k += 32)
            if (position(k) == c) {
              ++extra;
              first = min(first, k);
            }
          extra = __reduce_add_sync(0xffffffffu, extra);
          for (int k = R.K + lane; k < entries; k += 32)
            if (position(k) == c) first = min(first, k);
          first = __reduce_min_sync(0xffffffffu, first);
          float x = penalise(&R, value(c), word(first, c), extra);
          for (int k0 = R.K; k0 < entries; k0 += 32) {               // its biases, in order
            uint32_t hit = __ballot_sync(0xffffffffu, k0 + lane < entries && position(k0 + lane) == c);
            for (; hit; hit &= hit - 1) x = __fadd_rn(x, bias(k0 + __ffs(hit) - 1));
          }
          if (lane == 0) single(c, x);
        }
      }
    }

    // ---- the chunk's maximum and its lowest position
    float m = max_nan(best, sbest);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) s_red[warp] = m;
    __syncthreads();
    m = s_red[0];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) m = max_nan(m, s_red[w]);
    const bool nan = m != m;
    if (m != -INFINITY) {
      unsigned idx = 0xffffffffu;
      if (nan ? sbest != sbest : sbest == m) idx = si;
      if (bg >= 0 && (nan ? best != best : best == m)) {
        // the group's first token with that value
        uint32_t eq = 0;
#pragma unroll
        for (int e = 0; e < G; ++e) {
          const float x = bg + e < len ? (keep ? xs[bg + e] : staged(bg + e)) : -INFINITY;
          eq |= (uint32_t)(nan ? x != x : x == m) << e;
        }
        eq &= ~(uint32_t)((const uint8_t*)skip)[bg >> 3] & (rm ? (uint32_t)((const uint8_t*)mask)[bg >> 3] : ALL);
        if (eq) idx = min(idx, (unsigned)(start + bg + __ffs(eq)));
      }
      if (idx != 0xffffffffu) atomicMin(&s_idx, idx);
    }
    // ---- the chunk's sum of exponentials, kept in place of the values
    // log2(e) / T, finite so that equal values give 2^0 and positive so that a masked one gives 0 (T = inf: the least float;
    // the quotient of every finite T lies above it)
    const float c2 = onehot ? 0.f : fminf(fmaxf(__fdiv_rn(1.44269504f, temp), 1.4e-45f), 3.4e38f);
    auto expo = [&](float x, float top) { return exp2_fast((x - top) * c2); };
    float sum = 0.f;
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();                                   // the values above are read; s_red too
    if (keep) {
      const int n4 = len / 4;
      if (m != INFINITY) {
#pragma unroll 2
        for (int i = tid; i < n4; i += THREADS) {
          float4 v = ((float4*)xs)[i];
          v.x = expo(v.x, m); v.y = expo(v.y, m); v.z = expo(v.z, m); v.w = expo(v.w, m);
          ((float4*)xs)[i] = v;
          sum += (v.x + v.y) + (v.z + v.w);
        }
        if (tid < len - 4 * n4) {
          const float v = expo(xs[4 * n4 + tid], m);
          xs[4 * n4 + tid] = v;
          sum += v;
        }
      } else {                                         // +inf entries share the mass
        for (int i = tid; i < len; i += THREADS) {
          const float v = xs[i] == INFINITY ? 1.f : 0.f;
          xs[i] = v;
          sum += v;
        }
      }
      if (m == -INFINITY) sum = 0.f;                   // nothing allowed in the chunk
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) s_red[warp] = sum;
      __syncthreads();
      sum = s_red[0];
#pragma unroll
      for (int w = 1; w < WARPS; ++w) sum += s_red[w];
    } else if (r + 1 < r1) {
      stage(r + 1, rm_next);                           // the logits are not needed any more
    }
    for (int e = tid; special && e < entries; e += THREADS) {
      const int c = position(e);
      if (c < 0) continue;
      marks[c >> 5] = 0;
      if (!(e < ENTRIES ? ent_word[e] : rw ? (uint32_t)rw[start + c] : 0u)) atomicAnd(&skip[c >> 5], ~(1u << (c & 31)));
    }
    // ---- the row: one exchange within the cluster
    float top = m, total = sum;
    unsigned arg = s_idx;
    if (p.cluster > 1) {
      if (warp == 0) {           // one warp exchanges and waits; the others sleep at the block's barrier
        if (s_abort) {           // a NaN passes every other maximum, a position of 0 every other NaN
          m = NAN;
          arg = 0;
        }
        if (lane < p.cluster)
          asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                           map_rank(&s_peer[parity][rank], lane)),
                       "r"(__float_as_uint(m)), "r"(__float_as_uint(sum)), "r"(arg), "r"(0u), "r"(map_rank(&s_bar[parity], lane))
                       : "memory");
        __syncwarp();
        // where the wait expires, the peers' values may still come: they are not to find a CTA that has left
        const bool here = mbar::wait_head<true>(&s_bar[parity], bar_phase, &s_abort, a.dev_status) ||
                          mbar::drain<true>(&s_bar[parity], bar_phase, a.dev_status);
        __syncwarp();
        // armed for the row after the next before this CTA's next values let a peer get there
        if (lane == 0) expect_tx(&s_bar[parity], p.cluster * 16);
        float cm = -INFINITY, cs = 0.f;
        unsigned ci = 0xffffffffu;
        if (lane < p.cluster) {
          const float4 v = s_peer[parity][lane];
          cm = v.x;
          cs = v.y;
          ci = __float_as_uint(v.z);
        }
        if (!here) {
          cm = NAN;
          ci = 0;
        }
        float t = cm;
#pragma unroll
        for (int o = 4; o; o >>= 1) t = max_nan(t, __shfl_xor_sync(0xffffffffu, t, o));
        t = __shfl_sync(0xffffffffu, t, 0);
        if (!(t != t ? cm != cm : cm == t)) ci = 0xffffffffu;
        cs = cs == 0.f ? 0.f : cs * (cm == t ? 1.f : expo(cm, t));
#pragma unroll
        for (int o = 4; o; o >>= 1) {
          ci = min(ci, __shfl_xor_sync(0xffffffffu, ci, o));
          cs += __shfl_xor_sync(0xffffffffu, cs, o);
        }
        if (lane == 0) s_row = make_float4(t, cs, __uint_as_float(ci), 0.f);
        if (lane == 0 && ci == 0) s_told = 1;
      }
      __syncthreads();
      top = s_row.x;
      total = s_row.y;
      arg = __float_as_uint(s_row.z);
      bar_phase ^= parity;
      parity ^= 1;
    }
    const bool empty = top == -INFINITY;
    if (rank == 0 && tid == 0 && arg != 0) {
      if (a.argmax) a.argmax[r] = empty ? -1 : (int64_t)arg - 1;
      if (empty) flag_status(a.dev_status, MTPSD_STATUS_EMPTY_ROW);
    }
    // ---- the chunk's probabilities
    if (a.probs && arg != 0) {
      float* o = a.probs + r * a.probs_ld + start;
      const bool stored = keep && !empty;              // else zeros, and one at the greedy token
      // a NaN maximum makes every probability NaN
      const float f = !stored ? 0.f : (m == top ? 1.f : m == -INFINITY ? 0.f : expo(m, top));
      const float scale = stored ? __fdiv_rn(f, total) : 0.f;
      const bool bad = stored && top != top;
      auto prob = [&](int c) -> float {
        if (bad) return NAN;
        if (stored) return m == -INFINITY ? 0.f : xs[c] * scale;
        return onehot && !empty && (unsigned)(start + c) + 1 == arg ? 1.f : 0.f;
      };
      if (p.vec_probs) {
        const int n4 = len / 4;
        if (stored && !bad && m != -INFINITY) {
#pragma unroll 2
          for (int i = tid; i < n4; i += THREADS) {
            float4 v = ((float4*)xs)[i];
            v.x *= scale; v.y *= scale; v.z *= scale; v.w *= scale;
            ((float4*)o)[i] = v;
          }
        } else {
          for (int i = tid; i < n4; i += THREADS)
            ((float4*)o)[i] = make_float4(prob(4 * i), prob(4 * i + 1), prob(4 * i + 2), prob(4 * i + 3));
        }
        if (tid < len - 4 * n4) o[4 * n4 + tid] = prob(4 * n4 + tid);
      } else {
        for (int c = tid; c < len; c += THREADS) o[c] = prob(c);
      }
    }
    if (r + 1 < r1) {
      if (keep) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();                               // the values are read and may be overwritten
        stage(r + 1, rm_next);
      } else {
        __syncthreads();                               // s_idx and s_reps are read, the marks are cleared
      }
    }
  }
}

using Kernel = void (*)(const Params);

cudaLaunchConfig_t config(unsigned grid, int cluster, int threads, int smem, cudaStream_t st, cudaLaunchAttribute* attrs) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = cluster;
  attrs[1].val.clusterDim.y = 1;
  attrs[1].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cfg;
}

// Shared memory of a CTA when n of them share an SM.
constexpr int share(int n) { return (n == 4 ? 55 : n == 2 ? 110 : 220) * 1024; }

// Clusters that run at once with n CTAs per SM; cached per device.
int resident_clusters(Kernel kern, int bf16, int cluster, int n_cta, int threads) {
  static std::atomic<int> cache[kMaxCachedDevices][2][5][MAX_CLUSTER + 1];
  const int dev = current_device();
  const bool cacheable = dev >= 0 && dev < kMaxCachedDevices;
  if (cacheable) {
    const int v = cache[dev][bf16][n_cta][cluster].load(std::memory_order_relaxed);
    if (v) return v;
  }
  int n = 0;
  cudaLaunchAttribute attrs[2];
  cudaLaunchConfig_t cfg = config((unsigned)cluster, cluster, threads, share(n_cta), 0, attrs);
  if (cudaOccupancyMaxActiveClusters(&n, (void*)kern, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();            // not a fault of the call: a guess
    n = std::max(1, num_sms() * n_cta / cluster);
  }
  if (cacheable) cache[dev][bf16][n_cta][cluster].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace lgt

int launch_process_logits(const mtpsd_logits_args& a, cudaStream_t st) {
  using namespace lgt;
  const bool bf16 = a.dtype == MTPSD_BF16;
  const int per_token = bf16 && !a.probs ? 2 : 4;
  Params p;
  p.a = a;
  // CTAs per row: chunks that leave room for two CTAs per SM (where the vocabulary allows), and enough CTAs for every
  // SM twice, but no chunk below 4096 tokens (its share of the launch and the exchange would exceed its reads)
  const int two = (share(2) - smem_bytes(0, 0)) * 8 / (3 + 8 * per_token) / 128 * 128;
  p.cluster = 1;
  while (p.cluster < MAX_CLUSTER) {
    const int64_t chunk = ceil_div(a.V, p.cluster);
    if (chunk <= std::min(two, MAX_CHUNK) && ((int64_t)a.R * p.cluster >= 2 * num_sms() || chunk <= 4096)) break;
    p.cluster *= 2;
  }
  p.chunk = (int)(ceil_div(ceil_div(a.V, p.cluster), 128) * 128);
  p.vec_in = (uintptr_t)a.logits % 16 == 0 && a.ld * (bf16 ? 2 : 4) % 16 == 0;
  p.vec_out = (uintptr_t)a.out_logits % 16 == 0 && a.out_ld % 4 == 0;
  p.vec_probs = (uintptr_t)a.probs % 16 == 0 && a.probs_ld % 4 == 0;
  const int smem = smem_bytes(p.chunk, per_token);
  // few and short chunks: CTAs of 256 threads, so that more rows run at once (68 rows of 50001 took 29 us, with two of 512 36)
  const int n_cta = smem <= share(4) ? 4 : smem <= share(2) ? 2 : 1;
  const int threads = n_cta == 4 ? 256 : 384;
  static std::atomic<uint64_t> attr[4];
  Kernel kern = bf16 ? (threads == 256 ? process_logits_kernel<true, 256> : process_logits_kernel<true, 384>)
                     : (threads == 256 ? process_logits_kernel<false, 256> : process_logits_kernel<false, 384>);
  if (!set_smem_limit_once(kern, smem_bytes(MAX_CHUNK, 4), attr[2 * bf16 + (threads == 256)])) {
    set_error("process_logits: cudaFuncSetAttribute failed");
    return MTPSD_ECUDA;
  }
  const int clusters = std::min(a.R, resident_clusters(kern, bf16, p.cluster, n_cta, threads));
  cudaLaunchAttribute attrs[2];
  cudaLaunchConfig_t cfg = config((unsigned)(clusters * p.cluster), p.cluster, threads, smem, st, attrs);
  cudaLaunchKernelEx(&cfg, kern, p);
  return check_launch("process_logits");
}

}  // namespace mtpsd
