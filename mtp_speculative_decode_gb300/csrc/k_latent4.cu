// 4-bit latent cache rows from bf16 or float32 rows.  One warp per token: lane l holds values 8 l .. 8 l + 7 and 256 + 8 l ..;
// two neighbouring lanes share a block of 16, so its largest magnitude takes one exchange, and a lane's eight codes are one
// 32-bit word of the row.  Reads 1152 (2304) bytes and writes 416 per token: bound by memory, and next to it by the 16 IEEE
// divisions that the code's definition asks of each lane.
#include "cache.h"
#include "common.cuh"
#include "latent4.cuh"

namespace mtpsd {

// Eight values as floats
template <bool F32IN>
__device__ __forceinline__ void load8(const void* base, int64_t at, float* v) {
  if constexpr (F32IN) {
    const float4* p = (const float4*)((const float*)base + at);
    const float4 a = p[0], b = p[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 u = *(const uint4*)((const __nv_bfloat16*)base + at);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

template <bool F32IN>
__global__ void __launch_bounds__(256) pack_latent_fp4_kernel(const void* __restrict__ latent, int64_t T, uint8_t* __restrict__ out,
                                                              const int64_t* __restrict__ slots, int64_t pool, int32_t* status) {
  griddep_wait();                // the previous kernel's writes are visible from here on
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t warp = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  for (int64_t t = warp; t < T; t += nwarps) {
    float v[2][8], r[8];
    load8<F32IN>(latent, t * 576 + 8 * lane, v[0]);
    load8<F32IN>(latent, t * 576 + 256 + 8 * lane, v[1]);
    if (lane < 8) load8<F32IN>(latent, t * 576 + 512 + 8 * lane, r);
    const int64_t row = slots ? slots[t] : t;
    if (row < 0 || row >= pool) {
      if (lane == 0) flag_status(status, MTPSD_STATUS_WRITE_RANGE);
      continue;
    }
    uint8_t* o = out + row * lat4::ROW;
    lat4::store_values(v, o, lane);
    if (lane < 8) lat4::store_rope(r, o, lane);
  }
}

int launch_pack_latent_fp4(const void* latent, bool f32_in, int64_t T, uint8_t* out, const int64_t* slots, int64_t pool,
                           int32_t* status, cudaStream_t st) {
  int64_t blocks = (T + 7) / 8;
  if (blocks > 16 * num_sms()) blocks = 16 * num_sms();
  if (f32_in) launch_k(pack_latent_fp4_kernel<true>, (int)blocks, 256, 0, st, latent, T, out, slots, pool, status);
  else launch_k(pack_latent_fp4_kernel<false>, (int)blocks, 256, 0, st, latent, T, out, slots, pool, status);
  return check_launch("pack_latent_fp4");
}

}  // namespace mtpsd
