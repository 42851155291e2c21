// Penalties, biases and the grammar mask on the verify rows' logits, the greedy
// token and the target distribution ([P1] "阶段 3:拒绝采样与 Bitmask").
//
// Memory bound: every logit is read once and every probability written once.  A
// cluster of 1, 2, 4 or 8 CTAs takes a row, each a chunk of the vocabulary.
// 1. Tokens that need more than the table and the mask (the row's drafts, the
//    request's biases) are marked in a bitmap and computed one per thread.
// 2. The chunk streams through: x = logit, penalties where the table word is not
//    zero, -inf where the mask bit is; the other tokens' values go to shared
//    memory when probabilities are wanted, and every thread keeps its largest
//    group of values.
// 3. The chunk's largest value m_c (and its lowest position) and, over shared
//    memory, s_c = sum exp((x - m_c) / T) are exchanged within the cluster once:
//    the row's maximum is m = max m_c and its sum s = sum_c s_c exp((m_c - m) / T).
// 4. The chunk's probabilities exp((x - m_c) / T) * exp((m_c - m) / T) / s are written.
// All values, the maximum and the sums are float32; the sums add at most chunk /
// 512 values per thread before the tree, in an order fixed by the sizes.
#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"

namespace mtpsd {
namespace lgt {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int MAX_CHUNK = 49152;              // 192 KB of values
constexpr int MAX_CLUSTER = 8;
static_assert((int64_t)MAX_CHUNK * MAX_CLUSTER == 393216, "the vocabulary that the call allows");

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
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t ld_cluster_u32(const void* p, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// What one row of the call reads (request b, local row i).
struct Row {
  const void* x;
  const uint16_t* word;     // table row or NULL
  const uint8_t* mask;      // mask row (bytes) or NULL
  const int64_t* draft;
  int nd;                   // drafts that the row follows
  const int32_t* bt;
  const float* bv;
  int nb;                   // biases
  float rep, freq, pres;
};

template <bool BF16>
__device__ __forceinline__ float raw_logit(const Row& r, int64_t t) {
  return BF16 ? __bfloat162float(((const __nv_bfloat16*)r.x)[t]) : ((const float*)r.x)[t];
}

// The penalties of a token with table word w and `extra` more outputs (each step rounded to float32, as documented).
__device__ __forceinline__ float penalise(const Row& r, float x, uint32_t w, int extra) {
  const int n = (int)(w & 32767u) + extra;
  if ((w & 32768u) || n > 0) x = x > 0.f ? __fdiv_rn(x, r.rep) : __fmul_rn(x, r.rep);
  if (n > 0) x = __fsub_rn(__fsub_rn(x, __fmul_rn(r.freq, (float)n)), r.pres);
  return x;
}

__device__ __forceinline__ bool allowed(const Row& r, int64_t t) { return !r.mask || ((r.mask[t >> 3] >> (t & 7)) & 1); }

// x of a token of the drafts or the biases.  bias: its one bias, or, when the chunk has tokens with more than one
// (scan), every one of the list in order.
template <bool BF16>
__device__ float special_value(const Row& r, int64_t t, bool has_bias, float bias, bool scan) {
  int extra = 0;
  for (int j = 0; j < r.nd; ++j) extra += r.draft[j] == t;
  float x = penalise(r, raw_logit<BF16>(r, t), r.word ? r.word[t] : 0u, extra);
  if (scan) {
    for (int j = 0; j < r.nb; ++j)
      if (r.bt[j] == t) x = __fadd_rn(x, r.bv[j]);
  } else if (has_bias) {
    x = __fadd_rn(x, bias);
  }
  return allowed(r, t) ? x : -INFINITY;
}

// G: tokens per thread and step: 16 bytes of logits, or 1 when the rows are not 16-byte aligned.
template <bool BF16, int G>
__global__ void __launch_bounds__(THREADS, 2) process_logits_kernel(const __grid_constant__ Params p) {
  const mtpsd_logits_args& a = p.a;
  extern __shared__ float smem[];
  __shared__ float s_red[WARPS];
  __shared__ unsigned s_idx;
  __shared__ int s_dup;
  __shared__ float s_pub[2];             // the chunk's maximum and sum
  __shared__ unsigned s_pub_idx;         // the lowest position of the maximum
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = p.cluster > 1 ? cluster_rank() : 0;
  const uint32_t r = blockIdx.x / p.cluster;
  griddep_wait();                // the previous kernel's writes are visible from here on
  griddep_launch_dependents();
  if (r < a.row_offsets[0] || r >= a.row_offsets[a.B]) return;   // a padded batch (the whole cluster leaves)
  const int b = request_of_row_warp(a.row_offsets, a.B, r);
  const int64_t start = (int64_t)rank * p.chunk;
  const int len = (int)max((int64_t)0, min((int64_t)p.chunk, a.V - start));
  const bool first = rank == 0 && tid == 0;

  Row R;
  R.x = (const char*)a.logits + (int64_t)r * a.ld * (BF16 ? 2 : 4);
  R.word = nullptr;
  if (a.counts) {
    const int64_t row = a.count_rows ? a.count_rows[b] : b;
    if (row >= 0 && row < a.counts_rows) R.word = (const uint16_t*)a.counts + row * a.counts_ld;
    else if (row != -1 && first) flag_status(a.dev_status, MTPSD_STATUS_ROW_RANGE);
  }
  R.mask = nullptr;
  if (a.bitmask) {
    const int64_t m = a.mask_rows ? (int64_t)a.mask_rows[r] : (int64_t)r;
    if (m >= 0 && m < a.n_masks) R.mask = (const uint8_t*)(a.bitmask + m * ((a.V + 31) / 32));
    else if (m != -1 && first) flag_status(a.dev_status, MTPSD_STATUS_ROW_RANGE);
  }
  R.draft = a.draft ? a.draft + (int64_t)b * a.K : nullptr;
  R.nd = a.draft ? (int)min((int64_t)r - a.row_offsets[b], (int64_t)a.K) : 0;
  R.bt = nullptr;
  R.bv = nullptr;
  R.nb = 0;
  if (a.bias_offsets) {
    const uint32_t lo = a.bias_offsets[b], hi = a.bias_offsets[b + 1], end = (uint32_t)a.n_bias;
    if (hi > end && first) flag_status(a.dev_status, MTPSD_STATUS_INDEX_RANGE);
    R.bt = a.bias_tokens + lo;
    R.bv = a.bias_values + lo;
    R.nb = min(hi, end) > lo ? (int)(min(hi, end) - lo) : 0;
  }
  R.rep = a.repetition ? a.repetition[b] : 1.f;
  R.freq = a.frequency ? a.frequency[b] : 0.f;
  R.pres = a.presence ? a.presence[b] : 0.f;
  const float temp = a.temperature ? a.temperature[b] : 1.f;
  const bool onehot = !(temp > 0.f);
  const bool keep = a.probs != nullptr && !onehot;     // the values stay in shared memory for the probabilities
  float* out = a.out_logits ? a.out_logits + (int64_t)r * a.out_ld : nullptr;
  uint32_t* bits = (uint32_t*)smem;                    // [chunk / 32]: tokens of the drafts and the biases
  float* xs = smem + p.chunk / 32;                     // [chunk]
  const bool special = R.nd + R.nb > 0;

  // the thread's largest value: of a step's group bg (-1: none yet), or the special token bi
  float best = -INFINITY, sbest = -INFINITY;
  int bg = -1;
  unsigned si = 0xffffffffu;
  if (tid == 0) {
    s_idx = 0xffffffffu;
    s_dup = 0;
  }
  if (special) {
    for (int i = tid; i < p.chunk / 32; i += THREADS) bits[i] = 0;
    __syncthreads();
    for (int j = tid; j < R.nb; j += THREADS) {
      const int64_t t = R.bt[j], c = t - start;
      if ((t < 0 || t >= a.V) && rank == 0) flag_status(a.dev_status, MTPSD_STATUS_INDEX_RANGE);
      if (c >= 0 && c < len && (atomicOr(&bits[c >> 5], 1u << (c & 31)) >> (c & 31) & 1)) s_dup = 1;
    }
    __syncthreads();
    const bool scan = s_dup != 0;
    auto take = [&](int64_t t, bool has_bias, float bias) {
      const float x = special_value<BF16>(R, t, has_bias, bias, scan);
      if (keep) xs[t - start] = x;
      if (out) out[t] = x;
      // NaN above everything, then the larger value, then the lower position
      const bool above = x != x ? !(sbest != sbest) || (unsigned)t < si
                                : x > sbest || (x == sbest && (unsigned)t < si);
      if (above) {
        sbest = x;
        si = (unsigned)t;
      }
    };
    for (int j = tid; j < R.nb; j += THREADS) {
      const int64_t t = R.bt[j], c = t - start;
      if (c < 0 || c >= len) continue;
      bool again = false;                              // a token with several biases is its first entry's
      if (scan)
        for (int k = 0; k < j; ++k) again = again || R.bt[k] == t;
      if (!again) take(t, true, R.bv[j]);
    }
    for (int j = tid; j < R.nd; j += THREADS) {
      const int64_t t = R.draft[j], c = t - start;
      if ((t < 0 || t >= a.V) && rank == 0) flag_status(a.dev_status, MTPSD_STATUS_INDEX_RANGE);
      // a draft that is a bias's token, or another draft's, is taken by that entry
      if (c >= 0 && c < len && !(atomicOr(&bits[c >> 5], 1u << (c & 31)) >> (c & 31) & 1)) take(t, false, 0.f);
    }
  }
  __syncthreads();

  // ---- the chunk
  constexpr int U = G > 1 ? 4 : 8;                     // groups of a thread in flight
  const int groups = len / G;
  // what a group needs, as loaded: 16 bytes of logits (or one value), its table words, its mask bits
  struct Group {
    uint32_t v[G == 1 ? 1 : 4];
    uint32_t w[G == 1 ? 1 : G / 2];
    uint32_t mk;
  };
  auto load = [&](int g, Group& q) {
    const int64_t t = start + (int64_t)g * G;
    if constexpr (G == 1) {
      q.v[0] = __float_as_uint(raw_logit<BF16>(R, t));
      q.w[0] = R.word ? R.word[t] : 0u;
    } else {
      const uint4 v = *(const uint4*)((const char*)R.x + t * (BF16 ? 2 : 4));
      q.v[0] = v.x; q.v[1] = v.y; q.v[2] = v.z; q.v[3] = v.w;
      if constexpr (BF16) {
        const uint4 k = R.word ? *(const uint4*)(R.word + t) : make_uint4(0, 0, 0, 0);
        q.w[0] = k.x; q.w[1] = k.y; q.w[2] = k.z; q.w[3] = k.w;
      } else {
        const uint2 k = R.word ? *(const uint2*)(R.word + t) : make_uint2(0, 0);
        q.w[0] = k.x; q.w[1] = k.y;
      }
    }
    q.mk = R.mask ? R.mask[t >> 3] >> (t & 7) & ((1u << G) - 1) : (1u << G) - 1;
  };
  auto handle = [&](int g, const Group& q) {
    float x[G];
    uint32_t any = 0;
#pragma unroll
    for (int e = 0; e < G; ++e)
      x[e] = __uint_as_float(!BF16 || G == 1 ? q.v[e] : (e & 1) ? q.v[e / 2] & 0xffff0000u : q.v[e / 2] << 16);
#pragma unroll
    for (int e = 0; e < (G + 1) / 2; ++e) any |= q.w[e];
    if (any)
#pragma unroll
      for (int e = 0; e < G; ++e) {
        const uint32_t w = (e & 1) ? q.w[e / 2] >> 16 : q.w[e / 2] & 0xffffu;
        if (w) x[e] = penalise(R, x[e], w, 0);
      }
    if (q.mk != (1u << G) - 1)
#pragma unroll
      for (int e = 0; e < G; ++e)
        if (!(q.mk >> e & 1)) x[e] = -INFINITY;
    const int c = g * G;
    const uint32_t sp = special ? bits[c >> 5] >> (c & 31) & ((1u << G) - 1) : 0;
    float gm = -INFINITY;
#pragma unroll
    for (int e = 0; e < G; ++e)
      if (!(sp >> e & 1)) gm = max_nan(gm, x[e]);
    if (!(gm <= best) && best == best) {               // the first group with the largest value; a NaN stays
      best = gm;
      bg = g;
    }
    if (sp) {
#pragma unroll
      for (int e = 0; e < G; ++e)
        if (!(sp >> e & 1)) {
          if (keep) xs[c + e] = x[e];
          if (out) out[start + c + e] = x[e];
        }
      return;
    }
    if (keep) {
      if constexpr (G == 1) xs[c] = x[0];
      else
#pragma unroll
        for (int e = 0; e < G; e += 4) *(float4*)(xs + c + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
    }
    if (out) {
      if (G > 1 && p.vec_out) {
#pragma unroll
        for (int e = 0; e < G; e += 4) *(float4*)(out + start + c + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
      } else {
#pragma unroll
        for (int e = 0; e < G; ++e) out[start + c + e] = x[e];
      }
    }
  };
  for (int g0 = tid; g0 < groups; g0 += U * THREADS) {
    Group q[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (g0 + u * THREADS < groups) load(g0 + u * THREADS, q[u]);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (g0 + u * THREADS < groups) handle(g0 + u * THREADS, q[u]);
  }
  // the tokens behind the last whole group, one per thread
  if (G > 1 && tid < len - groups * G) {
    const int c = groups * G + tid;
    const int64_t t = start + c;
    if (!(special && bits[c >> 5] >> (c & 31) & 1)) {
      float x = penalise(R, raw_logit<BF16>(R, t), R.word ? R.word[t] : 0u, 0);
      if (!allowed(R, t)) x = -INFINITY;
      if (keep) xs[c] = x;
      if (out) out[t] = x;
      const bool above = x != x ? !(sbest != sbest) || (unsigned)t < si : x > sbest || (x == sbest && (unsigned)t < si);
      if (above) {
        sbest = x;
        si = (unsigned)t;
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
      for (int e = 0; e < G; ++e) {                    // the group's first token with that value
        const int c = bg * G + e;
        const int64_t t = start + c;
        if (special && bits[c >> 5] >> (c & 31) & 1) continue;
        float x;
        if (keep) x = xs[c];
        else if (out) x = out[t];
        else {
          x = penalise(R, raw_logit<BF16>(R, t), R.word ? R.word[t] : 0u, 0);
          if (!allowed(R, t)) x = -INFINITY;
        }
        if (nan ? x != x : x == m) {
          idx = min(idx, (unsigned)t);
          break;
        }
      }
    }
    if (idx != 0xffffffffu) atomicMin(&s_idx, idx);
  }
  // ---- the chunk's sum of exponentials, kept in place of the values
  // an infinite temperature: every allowed token alike (the masked ones' -inf times 0 would be a NaN)
  const float inv_t = onehot ? 0.f : temp == INFINITY ? 1e-38f : __fdiv_rn(1.f, temp);
  float sum = 0.f;
  if (keep) {
    __syncthreads();                                   // the values above are read; s_red too
    auto expo = [&](float x) { return x == m ? 1.f : expf((x - m) * inv_t); };
    const int n4 = len / 4;
    for (int i = tid; i < n4; i += THREADS) {
      float4 v = ((float4*)xs)[i];
      v.x = expo(v.x); v.y = expo(v.y); v.z = expo(v.z); v.w = expo(v.w);
      ((float4*)xs)[i] = v;
      sum += (v.x + v.y) + (v.z + v.w);
    }
    if (tid < len - 4 * n4) {
      const float v = expo(xs[4 * n4 + tid]);
      xs[4 * n4 + tid] = v;
      sum += v;
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
    if (tid == 0) {
      s_pub[0] = m;
      s_pub[1] = sum;
      s_pub_idx = s_idx;
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    float cm = -INFINITY, cs = 0.f;
    unsigned ci = 0xffffffffu;
    if (lane < p.cluster) {
      cm = __uint_as_float(ld_cluster_u32(&s_pub[0], lane));
      cs = __uint_as_float(ld_cluster_u32(&s_pub[1], lane));
      ci = ld_cluster_u32(&s_pub_idx, lane);
    }
    __syncwarp();
    cluster_arrive();            // nobody's values are read any more; waited for at the end
    top = cm;
#pragma unroll
    for (int o = 4; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    top = __shfl_sync(0xffffffffu, top, 0);
    if (!(top != top ? cm != cm : cm == top)) ci = 0xffffffffu;
    total = cs == 0.f ? 0.f : cs * (cm == top ? 1.f : expf((cm - top) * inv_t));
#pragma unroll
    for (int o = 4; o; o >>= 1) {
      ci = min(ci, __shfl_xor_sync(0xffffffffu, ci, o));
      total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    arg = __shfl_sync(0xffffffffu, ci, 0);
    total = __shfl_sync(0xffffffffu, total, 0);
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
    const float f = !stored ? 0.f : (m == top ? 1.f : m == -INFINITY ? 0.f : expf((m - top) * inv_t));
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
  __syncwarp();
  if (p.cluster > 1) cluster_wait();
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
  const int smem = p.chunk / 8 + (a.probs ? p.chunk * 4 : 0);
  static std::atomic<uint64_t> attr[4];
  const int which = (bf16 ? 2 : 0) + (vec_in ? 1 : 0);
  Kernel kern = bf16 ? (vec_in ? process_logits_kernel<true, 8> : process_logits_kernel<true, 1>)
                     : (vec_in ? process_logits_kernel<false, 4> : process_logits_kernel<false, 1>);
  if (!set_smem_limit_once(kern, MAX_CHUNK / 8 + MAX_CHUNK * 4, attr[which])) {
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
