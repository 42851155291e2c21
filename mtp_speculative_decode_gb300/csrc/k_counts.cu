// The token table of the repetition, frequency and presence penalties: one
// int16 word per (request, token), sign bit = in the prompt, low 15 bits = the
// number of occurrences in the output, held at 32767.
//
// Build: one launch clears the rows; a second counts, a CTA per 4096 tokens of a
// request.  Text repeats its tokens, so the CTA first gathers them in a hash table in
// shared memory and adds each distinct token once (one global update per token took
// 1162 us for 128 requests of 1024 .. 131072 tokens: the updates of a frequent token
// queue up).  The updates are additions with a limit and bit sets: any order gives the
// same table.  Bounded by writing and clearing the table and by the updates in L2.
// Accept: one thread per token that the step has put out.
#include "common.cuh"
#include "internal.h"

namespace mtpsd {

constexpr int SLICE = 4096;                   // tokens of a CTA
constexpr int SLOTS = 2 * SLICE;              // of its hash table
constexpr uint32_t EMPTY = 0xffffffffu;       // no key: tokens are below 2^31 - 1
constexpr int BUILD_THREADS = 512;
constexpr int BUILD_SMEM = SLOTS * 8;
constexpr int CLEAR_THREADS = 256;
constexpr int CLEAR_VECS = 8;                 // 16-byte stores per thread

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

__global__ void __launch_bounds__(CLEAR_THREADS) token_counts_clear_kernel(int16_t* __restrict__ counts, int64_t ld,
                                                                           int n_rows, const int32_t* __restrict__ rows,
                                                                           int32_t* status) {
  griddep_wait();                // the previous kernel's writes are visible from here on
  griddep_launch_dependents();
  const int64_t row = own_table_row(rows, blockIdx.y, n_rows, blockIdx.x == 0 ? status : nullptr);
  if (row < 0) return;
  int4* at = (int4*)(counts + row * ld);
  const int64_t v0 = (int64_t)blockIdx.x * CLEAR_THREADS * CLEAR_VECS + threadIdx.x;
#pragma unroll
  for (int i = 0; i < CLEAR_VECS; ++i)
    if (v0 + i * CLEAR_THREADS < ld / 8) at[v0 + i * CLEAR_THREADS] = make_int4(0, 0, 0, 0);
}

__global__ void __launch_bounds__(BUILD_THREADS) token_counts_build_kernel(
    const int64_t* __restrict__ tokens, int64_t S, const uint32_t* __restrict__ offsets,
    const int64_t* __restrict__ n_prompt, int B, int64_t V, int16_t* __restrict__ counts, int64_t ld, int n_rows,
    const int32_t* __restrict__ rows, int32_t* status) {
  extern __shared__ __align__(16) uint32_t smem[];
  uint32_t* keys = smem;                      // token | prompt << 31
  uint32_t* times = smem + SLOTS;
  __shared__ int s_b;
  __shared__ int64_t s_slice;
  const int tid = threadIdx.x, lane = tid & 31;
  for (int i = tid; i < SLOTS / 4; i += BUILD_THREADS) {
    ((uint4*)keys)[i] = make_uint4(EMPTY, EMPTY, EMPTY, EMPTY);
    ((uint4*)times)[i] = make_uint4(0, 0, 0, 0);
  }
  griddep_wait();                // the previous kernel's writes are visible from here on
  griddep_launch_dependents();
  // this CTA's slice: the blockIdx.x-th of all the requests' slices
  if (tid < 32) {
    int64_t before = 0;
    int found = -1;
    for (int b0 = 0; b0 < B && found < 0; b0 += 32) {
      const int b = b0 + lane;
      int64_t n = 0;
      if (b < B) n = ceil_div(max((int64_t)0, min((int64_t)offsets[b + 1], S) - (int64_t)offsets[b]), SLICE);
      int64_t upto = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      const unsigned who = __ballot_sync(0xffffffffu, before + upto > (int64_t)blockIdx.x);
      if (who) {
        found = b0 + __ffs(who) - 1;
        before += __shfl_sync(0xffffffffu, upto - n, __ffs(who) - 1);
      } else {
        before += __shfl_sync(0xffffffffu, upto, 31);
      }
    }
    if (lane == 0) {
      s_b = found;
      s_slice = (int64_t)blockIdx.x - before;
    }
    // the requests that end past the tokens, once
    if (blockIdx.x == 0)
      for (int b = lane; b < B; b += 32)
        if ((int64_t)offsets[b + 1] > S) flag_status(status, MTPSD_STATUS_ROW_RANGE);
  }
  __syncthreads();
  const int b = s_b;
  if (b < 0) return;             // the launch has a CTA per request to spare
  const int64_t row = own_table_row(rows, b, n_rows, nullptr);      // flagged when the rows were cleared
  if (row < 0) return;
  const int64_t first = offsets[b], end = min((int64_t)offsets[b + 1], S);
  const int64_t j0 = first + s_slice * SLICE, j1 = min(j0 + SLICE, end);
  const int64_t cut = n_prompt ? first + n_prompt[b] : end;
  constexpr int U = SLICE / BUILD_THREADS;
  int64_t t[U];
#pragma unroll
  for (int u = 0; u < U; ++u) t[u] = j0 + tid + u * BUILD_THREADS < j1 ? tokens[j0 + tid + u * BUILD_THREADS] : -1;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t j = j0 + tid + u * BUILD_THREADS;
    if (j >= j1) break;
    if (t[u] < 0 || t[u] >= V) {
      flag_status(status, MTPSD_STATUS_INDEX_RANGE);
      continue;
    }
    const bool prompt = j < cut;
    const uint32_t key = (uint32_t)t[u] | (prompt ? 0x80000000u : 0u);
    uint32_t slot = key * 2654435761u >> 19;  // 13 bits
    for (;;) {                   // at most half the slots are taken: an empty one or the key's is found
      uint32_t k = ((volatile uint32_t*)keys)[slot];
      if (k == EMPTY) k = atomicCAS(&keys[slot], EMPTY, key);
      if (k == EMPTY || k == key) break;
      slot = (slot + 1) & (SLOTS - 1);
    }
    if (!prompt) atomicAdd(&times[slot], 1u);
  }
  __syncthreads();
  int16_t* at = counts + row * ld;
  const bool below = end - first <= 0x7fff;   // no count of this request can pass the limit
  for (int i = tid; i < SLOTS; i += BUILD_THREADS) {
    const uint32_t key = keys[i];
    if (key == EMPTY) continue;
    const int64_t tok = key & 0x7fffffffu;
    uint32_t* w = (uint32_t*)(at + (tok & ~(int64_t)1));
    const int sh = (tok & 1) ? 16 : 0;
    if (key >> 31) atomicOr(w, 0x8000u << sh);
    else if (below) atomicAdd(w, times[i] << sh);
    else add_word(at, tok, times[i]);
  }
}
static_assert(SLOTS == 1 << 13, "the hash gives a slot");

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
  if (!set_smem_limit_once(token_counts_build_kernel, BUILD_SMEM, attr)) {
    set_error("token_counts_build: cudaFuncSetAttribute failed");
    return MTPSD_ECUDA;
  }
  const int per_row = (int)ceil_div(ld / 8, CLEAR_THREADS * CLEAR_VECS);
  launch_k(token_counts_clear_kernel, dim3(per_row, B), CLEAR_THREADS, 0, st, counts, ld, n_rows, rows, status);
  if (int rc = check_launch("token_counts_build")) return rc;
  // a slice per 4096 tokens and one for what is left of each request
  const int64_t slices = S / SLICE + B;
  launch_k(token_counts_build_kernel, (unsigned)slices, BUILD_THREADS, BUILD_SMEM, st, tokens, S, offsets, n_prompt, B, V,
           counts, ld, n_rows, rows, status);
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
