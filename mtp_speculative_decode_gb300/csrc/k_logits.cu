// Penalties, biases and the grammar mask on the verify rows' logits, the greedy
// token and the target distribution ([P1] "阶段 3:拒绝采样与 Bitmask").
//
// Memory bound: every logit is read once and every probability written once.  A
// cluster of 1, 2, 4 or 8 CTAs takes a row, each a chunk of the vocabulary.
// 1. The tokens of the row's drafts and of the request's biases are marked in a
//    bitmap.
// 2. The chunk streams through, 16 bytes of logits per thread and step: -inf
//    where the mask bit is 0; a token whose table word is not zero goes to its
//    warp's queue (they are about 1 in 100, but a warp's step would nearly always
//    have one: with the penalties computed in place 192 rows of 154880 took 124 us
//    and 768 rows, argmax only, 192 us); the others' values go to shared memory when
//    probabilities are wanted, and every thread keeps its largest group.
// 3. The queues are worked off with every lane busy, then the marked tokens, one per thread.
// 4. The chunk's largest value m_c (and its lowest position) and, over shared
//    memory, s_c = sum exp((x - m_c) / T) are exchanged within the cluster once
//    (each CTA stores its three words into the others' shared memory): the row's
//    maximum is m = max m_c and its sum s = sum_c s_c exp((m_c - m) / T).
// 5. The chunk's probabilities exp((x - m_c) / T) * (exp((m_c - m) / T) / s) are written.
// All values, the maximum and the sums are float32; the sums add at most chunk /
// 512 values per thread before the tree, in an order fixed by the sizes.  The
// exponentials are 2^y, y = (x - m_c) (log2 e / T): y is off by less than 2^-22.5 of its value.
#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"
#include "mbar.cuh"

namespace mtpsd {
namespace lgt {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int MAX_CHUNK = 49152;              // 192 KB of values
constexpr int MAX_CLUSTER = 8;
static_assert((int64_t)MAX_CHUNK * MAX_CLUSTER == 393216, "the vocabulary that the call allows");

constexpr int STEP = 512;                     // most tokens of a warp between two looks at its queue
constexpr int QUEUE = STEP + 64;              // positions in a warp's queue
constexpr int QUEUE_BYTES = WARPS * QUEUE * 2;
static_assert(MAX_CHUNK <= 65536, "a queue holds 16-bit positions");

struct Params {
  mtpsd_logits_args a;
  int chunk;              // tokens per CTA (a multiple of 128)
  int cluster;            // CTAs per row
  int vec_out;            // out_logits rows can be written 16 bytes at a time
  int vec_probs;          // probs rows likewise
};

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The barriers of the exchange exist before a peer stores into this CTA (their initialisation was released by
// fence.mbarrier_init); arriving early and waiting late hides the barrier behind the chunk.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t map_rank(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ float exp2_fast(float y) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
  return r;
}

// What one row of the call reads (request b, local row i); in shared memory.
struct Row {
  const void* x;
  const uint16_t* word;     // table row or NULL
  const uint8_t* mask;      // mask row (bytes) or NULL
  const int64_t* draft;
  const int32_t* bt;
  const float* bv;
  int nd;                   // drafts that the row follows
  int nb;                   // biases
  float rep, freq, pres, temp;
};

template <bool BF16>
__device__ __forceinline__ float raw_logit(const void* x, int64_t t) {
  return BF16 ? __bfloat162float(((const __nv_bfloat16*)x)[t]) : ((const float*)x)[t];
}

// The penalties of a token with table word w and `extra` more outputs (each step rounded to float32, as documented).
__device__ __noinline__ float penalise(const Row* r, float x, uint32_t w, int extra) {
  const int n = (int)(w & 32767u) + extra;
  if ((w & 32768u) || n > 0) x = x > 0.f ? __fdiv_rn(x, r->rep) : __fmul_rn(x, r->rep);
  if (n > 0) x = __fsub_rn(__fsub_rn(x, __fmul_rn(r->freq, (float)n)), r->pres);
  return x;
}

// x of token t outside the stream.  own_bias: entry j of the biases is its only one; scan: the chunk has tokens with
// more than one entry, so every bias of the list is looked through, in order.
template <bool BF16>
__device__ __noinline__ float token_value(const Row* r, int64_t t, int own_bias, bool scan) {
  int extra = 0;
  for (int j = 0; j < r->nd; ++j) extra += r->draft[j] == t;
  float x = penalise(r, raw_logit<BF16>(r->x, t), r->word ? r->word[t] : 0u, extra);
  if (scan) {
    for (int j = 0; j < r->nb; ++j)
      if (r->bt[j] == t) x = __fadd_rn(x, r->bv[j]);
  } else if (own_bias >= 0) {
    x = __fadd_rn(x, r->bv[own_bias]);
  }
  return !r->mask || ((r->mask[t >> 3] >> (t & 7)) & 1) ? x : -INFINITY;
}

// G: tokens per thread and step: 16 bytes of logits, or 1 when the rows are not 16-byte aligned.
template <bool BF16, int G>
__global__ void __launch_bounds__(THREADS, 2) process_logits_kernel(const __grid_constant__ Params p) {
  const mtpsd_logits_args& a = p.a;
  extern __shared__ __align__(16) float smem[];
  __shared__ Row R;
  __shared__ float s_red[WARPS];
  __shared__ unsigned s_idx;
  __shared__ int s_dup, s_abort;
  __shared__ __align__(16) float4 s_peer[MAX_CLUSTER];   // (maximum, sum, position) of every CTA of the cluster
  __shared__ float4 s_row;               // the row's (maximum, sum, position)
  __shared__ __align__(8) uint64_t s_bar;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = p.cluster > 1 ? cluster_rank() : 0;
  const uint32_t r = blockIdx.x / p.cluster;
  uint16_t* queue = (uint16_t*)smem + warp * QUEUE;    // of this warp: positions in the chunk
  uint32_t* bits = (uint32_t*)smem + QUEUE_BYTES / 4;  // [chunk / 32]: tokens of the drafts and the biases
  float* xs = (float*)bits + p.chunk / 32;             // [chunk]
  if (tid == 0) {
    s_idx = 0xffffffffu;
    s_dup = s_abort = 0;
    if (p.cluster > 1) {
      const uint32_t bar = (uint32_t)__cvta_generic_to_shared(&s_bar);
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar));
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(p.cluster * 16) : "memory");
    }
  }
  for (int i = tid; i < p.chunk / 32; i += THREADS) bits[i] = 0;
  griddep_wait();                // the previous kernel's writes are visible from here on
  griddep_launch_dependents();
  if (r < a.row_offsets[0] || r >= a.row_offsets[a.B]) return;   // a padded batch (the whole cluster leaves)
  __syncwarp();
  if (p.cluster > 1) cluster_arrive();
  const int64_t start = (int64_t)rank * p.chunk;
  const int len = (int)max((int64_t)0, min((int64_t)p.chunk, a.V - start));
  const bool first = rank == 0 && tid == 0;
  if (warp == 0) {
    const int b = request_of_row_warp(a.row_offsets, a.B, r);
    if (lane == 0) {
      R.x = (const char*)a.logits + (int64_t)r * a.ld * (BF16 ? 2 : 4);
      R.word = nullptr;
      if (a.counts) {
        const int64_t row = a.count_rows ? a.count_rows[b] : b;
        if (row >= 0 && row < a.counts_rows) R.word = (const uint16_t*)a.counts + row * a.counts_ld;
        else if (row != -1 && rank == 0) flag_status(a.dev_status, MTPSD_STATUS_ROW_RANGE);
      }
      R.mask = nullptr;
      if (a.bitmask) {
        const int64_t m = a.mask_rows ? (int64_t)a.mask_rows[r] : (int64_t)r;
        if (m >= 0 && m < a.n_masks) R.mask = (const uint8_t*)(a.bitmask + m * ((a.V + 31) / 32));
        else if (m != -1 && rank == 0) flag_status(a.dev_status, MTPSD_STATUS_ROW_RANGE);
      }
      R.draft = a.draft ? a.draft + (int64_t)b * a.K : nullptr;
      R.nd = a.draft ? (int)min((int64_t)r - a.row_offsets[b], (int64_t)a.K) : 0;
      R.bt = nullptr;
      R.bv = nullptr;
      R.nb = 0;
      if (a.bias_offsets) {
        const uint32_t lo = a.bias_offsets[b], hi = a.bias_offsets[b + 1], end = (uint32_t)a.n_bias;
        if (hi > end && rank == 0) flag_status(a.dev_status, MTPSD_STATUS_INDEX_RANGE);
        R.bt = a.bias_tokens + lo;
        R.bv = a.bias_values + lo;
        R.nb = min(hi, end) > lo ? (int)(min(hi, end) - lo) : 0;
      }
      R.rep = a.repetition ? a.repetition[b] : 1.f;
      R.freq = a.frequency ? a.frequency[b] : 0.f;
      R.pres = a.presence ? a.presence[b] : 0.f;
      R.temp = a.temperature ? a.temperature[b] : 1.f;
    }
  }
  __syncthreads();
  const float temp = R.temp;
  const bool onehot = !(temp > 0.f);
  const bool keep = a.probs != nullptr && !onehot;     // the values stay in shared memory for the probabilities
  float* out = a.out_logits ? a.out_logits + (int64_t)r * a.out_ld : nullptr;
  const int entries = R.nd + R.nb;
  const bool special = entries > 0;

  // the thread's largest value: of a step's group bg (-1: none yet), or of a single token si
  float best = -INFINITY, sbest = -INFINITY;
  int bg = -1;
  unsigned si = 0xffffffffu;
  auto single = [&](int c, float x) {                  // a token computed on its own
    const unsigned t = (unsigned)(start + c);
    if (keep) xs[c] = x;
    if (out) out[t] = x;
    // NaN above everything, then the larger value, then the lower position
    const bool above = x != x ? !(sbest != sbest) || t < si : x > sbest || (x == sbest && t < si);
    if (above) {
      sbest = x;
      si = t;
    }
  };
  auto token = [&](int j) -> int64_t { return j < R.nd ? R.draft[j] : (int64_t)R.bt[j - R.nd]; };
  if (special) {
    for (int j = tid; j < entries; j += THREADS) {
      const int64_t t = token(j), c = t - start;
      if ((t < 0 || t >= a.V) && rank == 0) flag_status(a.dev_status, MTPSD_STATUS_INDEX_RANGE);
      if (c >= 0 && c < len && (atomicOr(&bits[c >> 5], 1u << (c & 31)) >> (c & 31) & 1)) s_dup = 1;
    }
    __syncthreads();
  }

  // ---- the chunk
  const void* const rx = R.x;
  const uint16_t* const rw = R.word;
  const uint8_t* const rm = R.mask;
  constexpr int U = G > 1 ? 2 : 4;                     // groups of a thread in flight
  static_assert(32 * G * U <= STEP, "the queue has room for a step");
  const int groups = len / G;
  // what a group needs, as loaded: 16 bytes of logits (or one value), its table words, its mask bits
  struct Group {
    uint32_t v[G == 1 ? 1 : 4];
    uint32_t w[G == 1 ? 1 : G / 2];
    uint32_t mk;
  };
  constexpr uint32_t ALL = (1u << G) - 1;
  auto load = [&](int g, Group& q) {
    const int64_t t = start + (int64_t)g * G;
    if constexpr (G == 1) {
      q.v[0] = __float_as_uint(raw_logit<BF16>(rx, t));
      q.w[0] = rw ? rw[t] : 0u;
    } else {
      const uint4 v = *(const uint4*)((const char*)rx + t * (BF16 ? 2 : 4));
      q.v[0] = v.x; q.v[1] = v.y; q.v[2] = v.z; q.v[3] = v.w;
      if constexpr (BF16) {
        const uint4 k = rw ? *(const uint4*)(rw + t) : make_uint4(0, 0, 0, 0);
        q.w[0] = k.x; q.w[1] = k.y; q.w[2] = k.z; q.w[3] = k.w;
      } else {
        const uint2 k = rw ? *(const uint2*)(rw + t) : make_uint2(0, 0);
        q.w[0] = k.x; q.w[1] = k.y;
      }
    }
    q.mk = rm ? rm[t >> 3] >> (t & 7) & ALL : ALL;
  };
  int queued = 0;                                      // of this warp (the same in every lane)
  auto flush = [&]() {
    __syncwarp();                                      // the positions and the steps' values are written
    for (int i = lane; i < queued; i += 32) {
      const int c = queue[i];
      const int64_t t = start + c;
      const float x = penalise(&R, raw_logit<BF16>(rx, t), rw[t], 0);
      single(c, !rm || (rm[t >> 3] >> (t & 7) & 1) ? x : -INFINITY);
    }
    __syncwarp();
    queued = 0;
  };
  // called by whole warps (the queue's places come from ballots); valid: this lane has a group
  auto handle = [&](int g, bool valid, const Group& q) {
    const int c = g * G;
    float x[G];
#pragma unroll
    for (int e = 0; e < G; ++e)
      x[e] = __uint_as_float(!BF16 || G == 1 ? q.v[e] : (e & 1) ? q.v[e / 2] & 0xffff0000u : q.v[e / 2] << 16);
    if (q.mk != ALL)
#pragma unroll
      for (int e = 0; e < G; ++e)
        if (!(q.mk >> e & 1)) x[e] = -INFINITY;
    // sp: not the stream's to handle: marked tokens, and tokens with a table word
    uint32_t sp = special && valid ? ((const uint8_t*)bits)[c >> 3] >> (c & 7) & ALL : 0;
    uint32_t any = 0;
#pragma unroll
    for (int e = 0; e < (G + 1) / 2; ++e) any |= q.w[e];
    if (__any_sync(0xffffffffu, valid && any)) {
      uint32_t nz = 0;
#pragma unroll
      for (int e = 0; e < (G + 1) / 2; ++e) {
        // bit 15 of each half where its 16 bits are not all zero
        const uint32_t h = ((q.w[e] & 0x7fff7fffu) + 0x7fff7fffu) | q.w[e];
        nz |= (h >> 15 & 1u | h >> 30 & 2u) << 2 * e;
      }
      nz = valid ? nz & ~sp : 0;
      sp |= nz;
      while (const uint32_t who = __ballot_sync(0xffffffffu, nz != 0)) {
        if (nz) queue[queued + __popc(who & ((1u << lane) - 1))] = (uint16_t)(c + __ffs(nz) - 1);
        nz &= nz - 1;
        queued += __popc(who);
      }
    }
    if (!valid) return;
    if (out) {
      if (G > 1 && p.vec_out && !sp) {
#pragma unroll
        for (int e = 0; e < G; e += 4) *(float4*)(out + start + c + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
      } else {
#pragma unroll
        for (int e = 0; e < G; ++e)
          if (!(sp >> e & 1)) out[start + c + e] = x[e];
      }
    }
    if (sp)
#pragma unroll
      for (int e = 0; e < G; ++e)
        if (sp >> e & 1) x[e] = -INFINITY;             // in shared memory too, until its own value comes
    float gm = x[0];
#pragma unroll
    for (int e = 1; e < G; ++e) gm = max_nan(gm, x[e]);
    if (!(gm <= best) && best == best) {               // the first group with the largest value; a NaN stays
      best = gm;
      bg = g;
    }
    if (keep) {
      if constexpr (G == 1) xs[c] = x[0];
      else
#pragma unroll
        for (int e = 0; e < G; e += 4) *(float4*)(xs + c + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
    }
  };
  for (int g0 = tid; g0 - lane < groups; g0 += U * THREADS) {
    if (queued > QUEUE - STEP) flush();
    Group q[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (g0 + u * THREADS < groups) load(g0 + u * THREADS, q[u]);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (g0 + u * THREADS - lane < groups) handle(g0 + u * THREADS, g0 + u * THREADS < groups, q[u]);
  }
  flush();
  // the tokens behind the last whole group, one per thread
  if (G > 1 && tid < len - groups * G) {
    const int c = groups * G + tid;
    if (!(special && bits[c >> 5] >> (c & 31) & 1)) {
      const int64_t t = start + c;
      const float x = penalise(&R, raw_logit<BF16>(rx, t), rw ? rw[t] : 0u, 0);
      single(c, !rm || (rm[t >> 3] >> (t & 7) & 1) ? x : -INFINITY);
    }
  }
  if (special) {
    __syncthreads();                                   // the stream's values are written
    const bool scan = s_dup != 0;                      // some token has several entries: the first one takes it
    for (int j = tid; j < entries; j += THREADS) {
      const int64_t t = token(j), c = t - start;
      if (c < 0 || c >= len) continue;
      bool again = false;
      if (scan)
        for (int k = 0; k < j; ++k) again = again || token(k) == t;
      if (!again) single((int)c, token_value<BF16>(&R, t, j - R.nd, scan));
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
      for (int e = 0; e < G; ++e) {                    // the group's first token with that value
        const int c = bg * G + e;
        const int64_t t = start + c;
        if (special && bits[c >> 5] >> (c & 31) & 1) continue;
        const bool open = !rm || (rm[t >> 3] >> (t & 7) & 1);
        if (rw && rw[t] && open) continue;             // these were taken one by one
        const float x = keep ? xs[c] : out ? out[t] : open ? raw_logit<BF16>(rx, t) : -INFINITY;
        if (nan ? x != x : x == m) {
          idx = min(idx, (unsigned)t);
          break;
        }
      }
    }
    if (idx != 0xffffffffu) atomicMin(&s_idx, idx);
  }
  // ---- the chunk's sum of exponentials, kept in place of the values
  // log2(e) / T, finite so that equal values give 2^0 and positive so that a masked one gives 0
  const float c2 = onehot ? 0.f : fminf(fmaxf(__fdiv_rn(1.44269504f, temp), 1e-38f), 3.4e38f);
  auto expo = [&](float x, float top) { return exp2_fast((x - top) * c2); };
  float sum = 0.f;
  if (keep) {
    __syncthreads();                                   // the values above are read; s_red too
    const int n4 = len / 4;
    if (m != INFINITY) {
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
    } else {                                           // +inf entries share the mass
      for (int i = tid; i < len; i += THREADS) {
        const float v = xs[i] == INFINITY ? 1.f : 0.f;
        xs[i] = v;
        sum += v;
      }
    }
    if (m == -INFINITY) sum = 0.f;                     // nothing allowed in the chunk
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_red[warp] = sum;
  }
  __syncthreads();
  if (keep) {
    sum = s_red[0];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) sum += s_red[w];
  }
  // ---- the row: one exchange within the cluster
  float top = m, total = sum;
  unsigned arg = s_idx;
  if (p.cluster > 1) {
    __syncwarp();
    cluster_wait();
    if (warp == 0) {             // one warp exchanges and waits; the others sleep at the block's barrier
      if (lane < p.cluster)
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                         map_rank(&s_peer[rank], lane)),
                     "r"(__float_as_uint(m)), "r"(__float_as_uint(sum)), "r"(arg), "r"(0u), "r"(map_rank(&s_bar, lane))
                     : "memory");
      __syncwarp();
      mbar::wait<true>(&s_bar, 0, &s_abort, a.dev_status, mbar::DEFAULT_LIMIT_NS);
      __syncwarp();
      float cm = -INFINITY, cs = 0.f;
      unsigned ci = 0xffffffffu;
      if (lane < p.cluster) {
        const float4 v = s_peer[lane];
        cm = v.x;
        cs = v.y;
        ci = __float_as_uint(v.z);
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
    }
    __syncthreads();
    top = s_row.x;
    total = s_row.y;
    arg = __float_as_uint(s_row.z);
  }
  const bool empty = top == -INFINITY;
  if (first) {
    if (a.argmax) a.argmax[r] = empty ? -1 : (int64_t)arg;
    if (empty) flag_status(a.dev_status, MTPSD_STATUS_EMPTY_ROW);
  }
  // ---- the chunk's probabilities
  if (a.probs) {
    float* o = a.probs + (int64_t)r * a.probs_ld + start;
    const bool stored = keep && !empty;                // else zeros, and one at the greedy token
    // a NaN maximum makes every probability NaN
    const float f = !stored ? 0.f : (m == top ? 1.f : m == -INFINITY ? 0.f : expo(m, top));
    const float scale = stored ? __fdiv_rn(f, total) : 0.f;
    const bool bad = stored && top != top;
    auto prob = [&](int c) -> float {
      if (bad) return NAN;
      if (stored) return m == -INFINITY ? 0.f : xs[c] * scale;
      return onehot && !empty && (unsigned)(start + c) == arg ? 1.f : 0.f;
    };
    if (p.vec_probs) {
      const int n4 = len / 4;
      for (int i = tid; i < n4; i += THREADS) {
        float4 v;
        if (stored && !bad && m != -INFINITY) {
          v = ((float4*)xs)[i];
          v.x *= scale; v.y *= scale; v.z *= scale; v.w *= scale;
        } else {
          v = make_float4(prob(4 * i), prob(4 * i + 1), prob(4 * i + 2), prob(4 * i + 3));
        }
        ((float4*)o)[i] = v;
      }
      if (tid < len - 4 * n4) o[4 * n4 + tid] = prob(4 * n4 + tid);
    } else {
      for (int c = tid; c < len; c += THREADS) o[c] = prob(c);
    }
  }
}

using Kernel = void (*)(const Params);

}  // namespace lgt

int launch_process_logits(const mtpsd_logits_args& a, cudaStream_t st) {
  using namespace lgt;
  Params p;
  p.a = a;
  // CTAs per row: chunks that leave room for two CTAs per SM, and enough CTAs for every SM twice, but no chunk below
  // 4096 tokens (its share of the launch and the exchange would exceed its reads)
  p.cluster = 1;
  while (p.cluster < MAX_CLUSTER) {
    const int64_t chunk = ceil_div(a.V, p.cluster);
    if (chunk <= (a.probs ? 24576 : MAX_CHUNK) && ((int64_t)a.R * p.cluster >= 2 * num_sms() || chunk <= 4096)) break;
    p.cluster *= 2;
  }
  p.chunk = (int)(ceil_div(ceil_div(a.V, p.cluster), 128) * 128);
  const bool bf16 = a.dtype == MTPSD_BF16;
  const bool vec_in = (uintptr_t)a.logits % 16 == 0 && a.ld * (bf16 ? 2 : 4) % 16 == 0;
  p.vec_out = (uintptr_t)a.out_logits % 16 == 0 && a.out_ld % 4 == 0;
  p.vec_probs = (uintptr_t)a.probs % 16 == 0 && a.probs_ld % 4 == 0;
  const int smem = QUEUE_BYTES + p.chunk / 8 + (a.probs ? p.chunk * 4 : 0);
  static std::atomic<uint64_t> attr[4];
  const int which = (bf16 ? 2 : 0) + (vec_in ? 1 : 0);
  Kernel kern = bf16 ? (vec_in ? process_logits_kernel<true, 8> : process_logits_kernel<true, 1>)
                     : (vec_in ? process_logits_kernel<false, 4> : process_logits_kernel<false, 1>);
  if (!set_smem_limit_once(kern, QUEUE_BYTES + MAX_CHUNK / 8 + MAX_CHUNK * 4, attr[which])) {
    set_error("process_logits: cudaFuncSetAttribute failed");
    return MTPSD_ECUDA;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.R * p.cluster);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = p.cluster;
  attrs[1].val.clusterDim.y = 1;
  attrs[1].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = p.cluster > 1 ? 2 : 1;
  cudaLaunchKernelEx(&cfg, kern, p);
  return check_launch("process_logits");
}

}  // namespace mtpsd
