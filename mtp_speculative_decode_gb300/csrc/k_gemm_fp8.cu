// Matrix product of FP8 E4M3 codes with a float32 scale for each block of 128:
//   out[m,n] = sum_kb sa[m,kb] sw[n',kb] sum_{k in kb} a[m,k] w[n,k]
// One CTA per 32 x 32 outputs: the block's codes are decoded into shared
// memory, each thread sums 2 x 2 products of the block in float32 and adds the
// scaled block sum to its accumulators.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace mtpsd {

__device__ __forceinline__ float e4m3_float(uint32_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)c, __NV_E4M3)));
}

__global__ void __launch_bounds__(256) gemm_fp8_kernel(GemmFp8Plan p) {
  griddep_wait();                // the previous kernel's writes are visible from here on
  griddep_launch_dependents();
  __shared__ float sa[32][132], sw[32][132];
  const int64_t m0 = (int64_t)blockIdx.y * 32, n0 = (int64_t)blockIdx.x * 32;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t kbs = p.K / 128;
  float acc[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
  for (int64_t kb = 0; kb < kbs; ++kb) {
    for (int i = threadIdx.x; i < 32 * 32; i += 256) {
      const int r = i >> 5, c = (i & 31) * 4;
      const uint32_t va = m0 + r < p.M ? *(const uint32_t*)(p.a + (m0 + r) * p.K + kb * 128 + c) : 0u;
      const uint32_t vw = n0 + r < p.N ? *(const uint32_t*)(p.w + (n0 + r) * p.K + kb * 128 + c) : 0u;
      for (int e = 0; e < 4; ++e) {
        sa[r][c + e] = e4m3_float((va >> (8 * e)) & 255u);
        sw[r][c + e] = e4m3_float((vw >> (8 * e)) & 255u);
      }
    }
    __syncthreads();
    float part[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
    for (int k = 0; k < 128; ++k)
      for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j) part[i][j] = fmaf(sa[ty + 16 * i][k], sw[tx + 16 * j][k], part[i][j]);
    for (int i = 0; i < 2; ++i)
      for (int j = 0; j < 2; ++j) {
        const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
        if (m < p.M && n < p.N)
          acc[i][j] = fmaf(part[i][j], p.a_scale[m * kbs + kb] * p.w_scale[(n / p.w_scale_rows) * kbs + kb], acc[i][j]);
      }
    __syncthreads();
  }
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j) {
      const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= p.M || n >= p.N) continue;
      if (p.out_f32) ((float*)p.out)[m * p.ld_out + n] = acc[i][j];
      else ((__nv_bfloat16*)p.out)[m * p.ld_out + n] = __float2bfloat16_rn(acc[i][j]);
    }
}

int launch_gemm_fp8(const GemmFp8Plan& p, cudaStream_t st) {
  launch_k(gemm_fp8_kernel, dim3((unsigned)ceil_div(p.N, 32), (unsigned)ceil_div(p.M, 32)), 256, 0, st, p);
  return check_launch("gemm_fp8_block128");
}

}  // namespace mtpsd
