// Launchers of the head's kernels: the FP8 product, the token table and the logits' processing (internal header).
#pragma once

#include "../../include/mtpsd.h"
#include "internal.h"

namespace mtpsd {

// FP8 product with block-128 scales
struct GemmFp8Plan {
  const uint8_t* a; const float* a_scale;
  const uint8_t* w; const float* w_scale; int w_scale_rows;
  int64_t M, N, K;
  bool out_f32; void* out; int64_t ld_out;
  int32_t* status;
};
int launch_gemm_fp8(const GemmFp8Plan& p, cudaStream_t st);
int launch_gemm_fp8_pair(const GemmFp8Plan& p, cudaStream_t st);   // many rows: pairs of CTAs (K > 0)

// logits of the verify rows and the token table of their penalties
int launch_process_logits(const mtpsd_logits_args& a, cudaStream_t st);
int launch_token_counts_build(const int64_t* tokens, int64_t S, const uint32_t* offsets, const int64_t* n_prompt, int B,
                              int64_t V, int16_t* counts, int64_t ld, int n_rows, const int32_t* rows, int32_t* status,
                              cudaStream_t st);
int launch_token_counts_accept(const int64_t* draft, const int32_t* n_acc, const int64_t* next, int B, int K, int64_t V,
                               int16_t* counts, int64_t ld, int n_rows, const int32_t* rows, int32_t* status,
                               cudaStream_t st);

}  // namespace mtpsd
