// Penalties, biases and the grammar mask on the verify rows' logits, the greedy
// token and the target distribution.
//
// One CTA per row, three passes over the row: the largest value with its lowest
// position, the sum of exponentials, the probabilities.
#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"

namespace mtpsd {

struct LogitsRow {
  const mtpsd_logits_args* a;
  const void* x;
  const int16_t* word;
  const int32_t* mask;
  const int64_t* draft;
  int nd;
  const int32_t* bt;
  const float* bv;
  int nb;
  float rep, freq, pres;
};

// x of token t after the penalties, the biases and the mask
__device__ float processed(const LogitsRow& r, int64_t t) {
  const mtpsd_logits_args& a = *r.a;
  float x = a.dtype == MTPSD_F32 ? ((const float*)r.x)[t] : __bfloat162float(((const __nv_bfloat16*)r.x)[t]);
  const int w = r.word ? r.word[t] : 0;
  int n = w & 32767;
  for (int j = 0; j < r.nd; ++j) n += r.draft[j] == t;
  if (w < 0 || n > 0) x = x > 0.f ? __fdiv_rn(x, r.rep) : __fmul_rn(x, r.rep);
  if (n > 0) x = __fsub_rn(__fsub_rn(x, __fmul_rn(r.freq, (float)n)), r.pres);
  for (int j = 0; j < r.nb; ++j)
    if (r.bt[j] == t) x = __fadd_rn(x, r.bv[j]);
  if (r.mask && !((r.mask[t >> 5] >> (t & 31)) & 1)) x = -INFINITY;
  return x;
}

__global__ void __launch_bounds__(512) process_logits_kernel(const __grid_constant__ mtpsd_logits_args a) {
  griddep_wait();                // the previous kernel's writes are visible from here on
  griddep_launch_dependents();
  const uint32_t r = blockIdx.x;
  if (r < a.row_offsets[0] || r >= a.row_offsets[a.B]) return;
  __shared__ unsigned long long s_best;
  __shared__ float s_sum[16];
  const int b = request_of_row(a.row_offsets, a.B, r);
  const int i = (int)(r - a.row_offsets[b]);
  const bool first = threadIdx.x == 0;
  LogitsRow R;
  R.a = &a;
  R.x = (const char*)a.logits + (int64_t)r * a.ld * (a.dtype == MTPSD_F32 ? 4 : 2);
  R.word = nullptr;
  if (a.counts) {
    const int64_t row = a.count_rows ? a.count_rows[b] : b;
    if (row >= 0 && row < a.counts_rows) R.word = a.counts + row * a.counts_ld;
    else if (row != -1 && first) flag_status(a.dev_status, MTPSD_STATUS_ROW_RANGE);
  }
  R.mask = nullptr;
  if (a.bitmask) {
    const int64_t m = a.mask_rows ? (int64_t)a.mask_rows[r] : (int64_t)r;
    if (m >= 0 && m < a.n_masks) R.mask = a.bitmask + m * ((a.V + 31) / 32);
    else if (m != -1 && first) flag_status(a.dev_status, MTPSD_STATUS_ROW_RANGE);
  }
  R.draft = a.draft ? a.draft + (int64_t)b * a.K : nullptr;
  R.nd = a.draft ? min(i, a.K) : 0;
  R.nb = 0;
  if (a.bias_offsets) {
    const uint32_t lo = a.bias_offsets[b], hi = min(a.bias_offsets[b + 1], (uint32_t)a.n_bias);
    if (a.bias_offsets[b + 1] > (uint32_t)a.n_bias && first) flag_status(a.dev_status, MTPSD_STATUS_INDEX_RANGE);
    R.bt = a.bias_tokens + lo;
    R.bv = a.bias_values + lo;
    R.nb = hi > lo ? (int)(hi - lo) : 0;
  }
  for (int j = threadIdx.x; j < R.nb; j += blockDim.x)
    if (R.bt[j] < 0 || R.bt[j] >= a.V) flag_status(a.dev_status, MTPSD_STATUS_INDEX_RANGE);
  for (int j = threadIdx.x; j < R.nd; j += blockDim.x)
    if (R.draft[j] < 0 || R.draft[j] >= a.V) flag_status(a.dev_status, MTPSD_STATUS_INDEX_RANGE);
  R.rep = a.repetition ? a.repetition[b] : 1.f;
  R.freq = a.frequency ? a.frequency[b] : 0.f;
  R.pres = a.presence ? a.presence[b] : 0.f;
  const float temp = a.temperature ? a.temperature[b] : 1.f;
  if (first) s_best = 0;
  __syncthreads();
  // (order-preserving key, inverted position): NaN above +inf, and the lowest position of equal values
  unsigned long long best = 0;
  for (int64_t t = threadIdx.x; t < a.V; t += blockDim.x) {
    const float x = processed(R, t);
    const uint32_t k = x != x ? 0xffffffffu : float_key(x);
    const unsigned long long v = ((unsigned long long)k << 32) | (uint32_t)~(uint32_t)t;
    best = v > best ? v : best;
  }
  atomicMax(&s_best, best);
  __syncthreads();
  const uint32_t top_key = (uint32_t)(s_best >> 32);
  const float top = top_key == 0xffffffffu ? NAN : key_float(top_key);
  const int64_t arg = top == -INFINITY ? -1 : (int64_t)(uint32_t)~(uint32_t)s_best;
  if (first) {
    if (a.argmax) a.argmax[r] = arg;
    if (arg < 0) flag_status(a.dev_status, MTPSD_STATUS_EMPTY_ROW);
  }
  const bool onehot = !(temp > 0.f);
  auto expo = [&](float x) { return x == top ? 1.f : expf(__fdiv_rn(x - top, temp)); };
  float total = 1.f;
  if (a.probs && !onehot && arg >= 0) {
    float sum = 0.f;
    for (int64_t t = threadIdx.x; t < a.V; t += blockDim.x) sum += expo(processed(R, t));
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = sum;
    __syncthreads();
    total = 0.f;
    for (int k = 0; k < 16; ++k) total += s_sum[k];
  }
  for (int64_t t = threadIdx.x; t < a.V; t += blockDim.x) {
    const float x = processed(R, t);
    if (a.probs)
      a.probs[(int64_t)r * a.probs_ld + t] = arg < 0 ? 0.f : onehot ? (t == arg ? 1.f : 0.f) : __fdiv_rn(expo(x), total);
    if (a.out_logits) a.out_logits[(int64_t)r * a.out_ld + t] = x;
  }
}

int launch_process_logits(const mtpsd_logits_args& a, cudaStream_t st) {
  launch_k(process_logits_kernel, a.R, 512, 0, st, a);
  return check_launch("process_logits");
}

}  // namespace mtpsd
