// The token table of the repetition, frequency and presence penalties: one
// int16 word per (request, token), sign bit = in the prompt, low 15 bits = the
// number of occurrences in the output, held at 32767.
//
// Build: one CTA per request clears its row and adds its tokens one by one.
// Accept: one thread per token that the step has put out.
#include "common.cuh"
#include "internal.h"

namespace mtpsd {

// Adds one occurrence (or sets the prompt bit) in the 16-bit word t of a row.  The words are updated
// through the aligned 32-bit word that holds two of them, by compare and swap, so that a count at its
// limit never carries into its neighbour; adding with a limit is order-independent.
__device__ __forceinline__ void add_word(int16_t* row, int64_t t, bool prompt) {
  uint32_t* w = (uint32_t*)(row + (t & ~(int64_t)1));
  const int sh = (t & 1) ? 16 : 0;
  uint32_t old = *(volatile uint32_t*)w;
  for (;;) {
    const uint32_t v = (old >> sh) & 0xffffu;
    const uint32_t n = prompt ? (v | 0x8000u) : ((v & 0x7fffu) < 0x7fffu ? v + 1 : v);
    if (n == v) return;
    const uint32_t got = atomicCAS(w, old, (old & ~(0xffffu << sh)) | (n << sh));
    if (got == old) return;
    old = got;
  }
}

// The table row of request b, or -1: none, outside the table, or (distinct) already the row of an earlier request.
__device__ __forceinline__ int64_t table_row(const int32_t* rows, int b, int n_rows, bool distinct, int32_t* status) {
  const int64_t row = rows ? rows[b] : b;
  if (row < -1 || row >= n_rows) {
    flag_status(status, MTPSD_STATUS_ROW_RANGE);
    return -1;
  }
  if (distinct && rows && row >= 0)
    for (int i = 0; i < b; ++i)
      if (rows[i] == row) {
        flag_status(status, MTPSD_STATUS_INDEX_RANGE);
        return -1;
      }
  return row;
}

__global__ void __launch_bounds__(512) token_counts_build_kernel(const int64_t* __restrict__ tokens, int64_t S,
                                                                 const uint32_t* __restrict__ offsets,
                                                                 const int64_t* __restrict__ n_prompt, int64_t V,
                                                                 int16_t* __restrict__ counts, int64_t ld, int n_rows,
                                                                 const int32_t* __restrict__ rows, int32_t* status) {
  griddep_wait();                // the previous kernel's writes are visible from here on
  griddep_launch_dependents();
  const int b = blockIdx.x;
  __shared__ int64_t s_row;
  if (threadIdx.x == 0) s_row = table_row(rows, b, n_rows, true, status);
  __syncthreads();
  if (s_row < 0) return;
  int16_t* row = counts + s_row * ld;
  for (int64_t t = threadIdx.x; t < ld / 8; t += blockDim.x) ((int4*)row)[t] = make_int4(0, 0, 0, 0);
  __syncthreads();
  const int64_t a = offsets[b], e = offsets[b + 1];
  if (e > S && threadIdx.x == 0) flag_status(status, MTPSD_STATUS_ROW_RANGE);
  const int64_t end = e < S ? e : S;
  const int64_t cut = n_prompt ? n_prompt[b] : end - a;
  for (int64_t j = a + threadIdx.x; j < end; j += blockDim.x) {
    const int64_t t = tokens[j];
    if (t < 0 || t >= V) flag_status(status, MTPSD_STATUS_INDEX_RANGE);
    else add_word(row, t, j - a < cut);
  }
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
  const int64_t row = table_row(rows, b, n_rows, false, status);
  if (row < 0) return;
  const int64_t t = j < K ? draft[(int64_t)b * K + j] : next[b];
  if (t < 0 || t >= V) flag_status(status, MTPSD_STATUS_INDEX_RANGE);
  else add_word(counts + row * ld, t, false);
}

int launch_token_counts_build(const int64_t* tokens, int64_t S, const uint32_t* offsets, const int64_t* n_prompt, int B,
                              int64_t V, int16_t* counts, int64_t ld, int n_rows, const int32_t* rows, int32_t* status,
                              cudaStream_t st) {
  launch_k(token_counts_build_kernel, B, 512, 0, st, tokens, S, offsets, n_prompt, V, counts, ld, n_rows, rows, status);
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
