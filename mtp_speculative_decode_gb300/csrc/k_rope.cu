// Norms of queries and keys for each head and their position rotation in one pass over the data, the results stored in the type
// and at the place where the next kernel reads them (plain rows, FP8 codes with scales, cache rows by slot).
//
// What it has to move bounds it (each value read and written once); a head's sums never leave its lanes' registers.  A head
// takes L lanes (4 .. 32), each holding 16-byte vectors of 8 values.  The vectors are dealt out so that the two partners of a
// half-split rotation lie in the same lane: pair slots hold vector i of the first half and vector i of the second, rest slots what is
// not turned.  A lane group takes several heads of one token in turn and keeps the token's cosines and sines in registers
// meanwhile (the weights come from L1 for each head); the next head's values are loaded before the present one is computed.
// Shapes that are no multiples of 8 values or of 16 bytes take the element kernel (a warp per head, the head in shared memory).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "cache.h"
#include "common.cuh"
#include "latent4.cuh"

namespace mtpsd {
namespace {

constexpr int MAX_D = 1024;

struct Side {
  const void* x;
  int64_t xt, xh;             // strides, elements
  void* out;
  int64_t ot, oh;             // strides, elements of the output (bytes for codes and cache rows)
  float* scale;
  const float* w;
  const float* b;
  const int64_t* slots;       // null: row t
  int64_t pool;
  int heads, D, norm, norm_dim, rot_start, out_type;
  bool in_f32, skip;          // skip: dims that are neither normed nor turned are where they belong already (in place)
  int lanes, groups;          // lanes per head; lane groups per token (each takes every groups-th head)
  int nr;                     // pair vectors: the first is rot_start / 8, its partner nr further
  int64_t items;              // T * groups
  int blocks;
};

struct Args {
  Side q, k;
  int64_t T;
  const int64_t* positions;
  const float* cs;            // [n_pos, rot_dim]: cosines, sines
  int64_t n_pos;
  int rot_dim, inter;
  float eps;
  int32_t* status;
};

template <bool F32>
struct Raw { uint4 a; };
template <>
struct Raw<true> { uint4 a, b; };

template <bool F32>
__device__ __forceinline__ void load_raw(const void* base, int64_t at, Raw<F32>& r) {
  if constexpr (F32) {
    const uint4* p = (const uint4*)((const float*)base + at);
    r.a = p[0];
    r.b = p[1];
  } else {
    r.a = *(const uint4*)((const __nv_bfloat16*)base + at);
  }
}
template <bool F32>
__device__ __forceinline__ void to_floats(const Raw<F32>& r, float* v) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
  if constexpr (F32) {
    const uint32_t u[4] = {r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(w[i]);
      v[4 + i] = __uint_as_float(u[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ void load8f(const float* p, float* v) {
  const float4 a = *(const float4*)p, b = *(const float4*)(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *(const uint32_t*)&p;
}
__device__ __forceinline__ uint4 bf16x8(const float* v) {
  return make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
}
__device__ __forceinline__ uint2 codes8(const float* v, float scale) {
  uint32_t c[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    c[i >> 2] |= (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(v[i], scale), __NV_SATFINITE, __NV_E4M3) << (8 * (i & 3));
  return make_uint2(c[0], c[1]);
}
__device__ __forceinline__ void turn(float& x, float& y, float c, float n) {
  const float p = x, q = y;
  x = p * c - q * n;
  y = p * n + q * c;
}
// x r w with one rounding (and 2^-48): the first product's error goes into the second.  The error of an infinite first product would
// be infinity less infinity; ANY_R takes it for a number (it is far smaller than 1 otherwise), so that infinity remains.  Only eps 0 and a
// head whose squares have no float32 value make r infinite: such calls take a form of the kernel with ANY_R, the others' form of few
// registers goes without it (8192 tokens x 40 heads of 128: 39.6 us, 40.7 with).
template <bool ANY_R>
__device__ __forceinline__ float mul3(float x, float r, float w) {
  const float p = x * r, e = fmaf(x, r, -p);
  return fmaf(p, w, (ANY_R ? fmaxf(e, -1.0f) : e) * w);
}
// Largest over `lanes` neighbouring lanes (all lanes of the warp take part)
__device__ __forceinline__ float group_max(float m, int lanes) {
  for (int o = lanes >> 1; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
__device__ __forceinline__ float group_sum(float s, int lanes) {
  for (int o = lanes >> 1; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}
__device__ __forceinline__ float amax8(const float* v, float m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}

// A token's output row and whether it is there; flagged by the caller's lane 0.
__device__ __forceinline__ bool token_ok(const Args& a, const Side& s, int64_t t, int64_t* row, int64_t* pos, int32_t* bits) {
  *pos = 0;
  *row = t;
  if (a.rot_dim) {
    *pos = a.positions[t];
    if (*pos < 0 || *pos >= a.n_pos) {
      *bits |= MTPSD_STATUS_ROW_RANGE;
      return false;
    }
  }
  if (s.slots) {
    *row = s.slots[t];
    if (*row < 0 || *row >= s.pool) {
      *bits |= MTPSD_STATUS_WRITE_RANGE;
      return false;
    }
  }
  return true;
}

// PS pair slots (two vectors each) and RS rest slots per lane.
template <bool F32, int PS, int RS>
__device__ __forceinline__ void run_side(const Args& a, const Side& s, int block) {
  constexpr int NV = 2 * PS + RS;
  const int L = s.lanes;
  const int lane = threadIdx.x & 31, l = lane & (L - 1);
  const int64_t item = (int64_t)block * (blockDim.x / L) + threadIdx.x / L;
  // no lane leaves early: the shuffles are the whole warp's
  const bool have = item < s.items;
  const int64_t t = have ? item / s.groups : 0;
  const int g = have ? (int)(item % s.groups) : 0;
  int32_t bits = 0;
  int64_t row = 0, pos = 0;
  const bool ok = have && token_ok(a, s, t, &row, &pos, &bits);
  if (bits && l == 0 && g == 0) flag_status(a.status, bits);

  const int nv = s.D >> 3, rs = s.rot_start >> 3, nr = s.nr;
  int vec[NV];      // the lane's vectors, or -1
#pragma unroll
  for (int j = 0; j < PS; ++j) {
    const int i = l + L * j;
    vec[2 * j] = i < nr ? rs + i : -1;
    vec[2 * j + 1] = i < nr ? rs + nr + i : -1;
  }
#pragma unroll
  for (int j = 0; j < RS; ++j) {
    const int i = l + L * j, v = i < rs ? i : i + 2 * nr;
    vec[2 * PS + j] = v < nv ? v : -1;
  }
  // cosines and sines of the lane's pair slots: half-split, of pairs 8 i .. 8 i + 7; interleaved, of the first vector's four pairs,
  // then the second's
  float cs[PS > 0 ? PS : 1][2][8];
  if (ok && a.rot_dim) {
#pragma unroll
    for (int j = 0; j < PS; ++j)
      if (vec[2 * j] >= 0) {
        const int i = l + L * j;
        const float* c = a.cs + pos * a.rot_dim + (a.inter ? 4 : 8) * i;
        const int second = a.inter ? 4 * nr : 4;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const float4 p = *(const float4*)(c + m * (a.rot_dim >> 1)), q = *(const float4*)(c + m * (a.rot_dim >> 1) + second);
          float* d = cs[j][m];
          d[0] = p.x; d[1] = p.y; d[2] = p.z; d[3] = p.w; d[4] = q.x; d[5] = q.y; d[6] = q.z; d[7] = q.w;
        }
      }
  }
  const int nnorm = s.norm ? s.norm_dim >> 3 : 0;   // vectors that the norm covers
  const float inv_n = s.norm ? 1.0f / (float)s.norm_dim : 0.f;
  Raw<F32> raw[NV];
  auto load = [&](int h) {
    const int64_t base = t * s.xt + h * s.xh;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (vec[i] >= 0) load_raw<F32>(s.x, base + vec[i] * 8, raw[i]);
  };
  const int steps = (s.heads + s.groups - 1) / s.groups;    // the same for all lanes
  if (ok && g < s.heads) load(g);
  for (int k = 0; k < steps; ++k) {
    const int h = g + k * s.groups;
    const bool on = ok && h < s.heads;
    float v[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (on && vec[i] >= 0) {
        to_floats<F32>(raw[i], v[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
      }
    }
    if (ok && h + s.groups < s.heads) load(h + s.groups);
    if (s.norm) {
      float mean = 0.f;
      if (s.norm == MTPSD_NORM_LAYER) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if ((unsigned)vec[i] < (unsigned)nnorm) {
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += v[i][e];
          }
        mean = group_sum(sum, L) * inv_n;
      }
      float sq = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if ((unsigned)vec[i] < (unsigned)nnorm) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[i][e] -= mean;
            sq = fmaf(v[i][e], v[i][e], sq);
          }
        }
      const float r = __frsqrt_rn(fmaf(group_sum(sq, L), inv_n, a.eps));
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if ((unsigned)vec[i] < (unsigned)nnorm) {
          float wt[8];
          if (s.w) {
            load8f(s.w + vec[i] * 8, wt);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = mul3<(RS > 0)>(v[i][e], r, wt[e]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] *= r;
          }
          if (s.b) {
            load8f(s.b + vec[i] * 8, wt);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] += wt[e];
          }
        }
    }
    if (a.rot_dim) {
#pragma unroll
      for (int j = 0; j < PS; ++j) {
        if (vec[2 * j] < 0) continue;
        float* x = v[2 * j];
        float* y = v[2 * j + 1];
        if (!a.inter) {
#pragma unroll
          for (int e = 0; e < 8; ++e) turn(x[e], y[e], cs[j][0][e], cs[j][1][e]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            turn(x[2 * e], x[2 * e + 1], cs[j][0][e], cs[j][1][e]);
            turn(y[2 * e], y[2 * e + 1], cs[j][0][4 + e], cs[j][1][4 + e]);
          }
        }
      }
    }
    if (s.out_type == MTPSD_FP8_E4M3) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) m = amax8(v[i], m);
      const float scale = fp8_block_scale(group_max(m, L));
      if (on) {
        uint8_t* o = (uint8_t*)s.out + row * s.ot + h * s.oh;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (vec[i] >= 0) *(uint2*)(o + vec[i] * 8) = codes8(v[i], scale);
        if (l == 0) s.scale[row * s.heads + h] = scale;
      }
      continue;
    }
    if constexpr (PS == 1 && RS == 2) {   // cache rows: 32 lanes, rest slots = values 8 l .. and 256 + 8 l .., pair slots = rope
      if (s.out_type == MTPSD_FP8_DS_MLA || s.out_type == MTPSD_FP4_MLA) {
        uint8_t* o = (uint8_t*)s.out + row * s.ot;
        const bool eight = s.out_type == MTPSD_FP8_DS_MLA;
        if (eight) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float scale = fp8_block_scale(group_max(amax8(v[2 + j], 0.f), 16));   // a block of 128: 16 lanes
            if (on) {
              *(uint2*)(o + 256 * j + 8 * lane) = codes8(v[2 + j], scale);
              if ((lane & 15) == 0) *(float*)(o + 512 + 4 * (2 * j + (lane >> 4))) = scale;
            }
          }
        } else if (__any_sync(0xffffffffu, on)) {     // one token per warp: all lanes or none
          lat4::store_values(v + 2, o, lane);
        }
        if (on && vec[0] >= 0) {
          uint4* rope = (uint4*)(o + (eight ? 528 : lat4::OFF_ROPE));
          rope[vec[0] - 64] = bf16x8(v[0]);
          rope[vec[1] - 64] = bf16x8(v[1]);
        }
        continue;
      }
    }
    if (!on) continue;
    const int64_t base = row * s.ot + h * s.oh;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (vec[i] < 0) continue;
      if (s.skip && i >= 2 * PS && vec[i] >= nnorm) continue;
      if (s.out_type == MTPSD_F32) {
        float4* o = (float4*)((float*)s.out + base + vec[i] * 8);
        o[0] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
        o[1] = make_float4(v[i][4], v[i][5], v[i][6], v[i][7]);
      } else {
        *(uint4*)((__nv_bfloat16*)s.out + base + vec[i] * 8) = bf16x8(v[i]);
      }
    }
  }
}

// CTAs of 256 threads per SM that the registers have to allow: the loads in flight carry the bandwidth.  Measured on 16384 x 128
// heads of 64 rope values (bf16): four CTAs (64 registers, 40 bytes of spills) take 126 us, three 133, five 155 (256 bytes).  The form
// of the latent rows and the indexer's heads spills 192 bytes at three CTAs (80 registers).
constexpr int min_ctas(bool f32, int slots) { return slots >= 8 ? 1 : (slots >= 4 ? (f32 ? 2 : 3) : (f32 ? 3 : 4)); }
template <bool F32, int QP, int QR, int KP, int KR>
__global__ void __launch_bounds__(256, min_ctas(F32, 2 * (QP > KP ? QP : KP) + (QR > KR ? QR : KR))) norm_rope_kernel(const __grid_constant__ Args a) {
  griddep_wait();                // the previous kernel's writes are visible from here on
  griddep_launch_dependents();
  if ((int)blockIdx.x < a.q.blocks) run_side<F32, QP, QR>(a, a.q, blockIdx.x);
  else run_side<F32, KP, KR>(a, a.k, blockIdx.x - a.q.blocks);
}

// Any shape and alignment: a warp per head, its values in shared memory between the norm and the rotation.
template <bool F32>
__global__ void __launch_bounds__(256) norm_rope_elements_kernel(const __grid_constant__ Args a) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float buf[8][MAX_D];
  const Side& s = a.k;
  const int lane = threadIdx.x & 31;
  float* v = buf[threadIdx.x >> 5];
  const int64_t items = a.T * s.heads, warps = (int64_t)gridDim.x * 8;
  for (int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); item < items; item += warps) {
    const int64_t t = item / s.heads;
    const int h = (int)(item % s.heads);
    int32_t bits = 0;
    int64_t row, pos;
    if (!token_ok(a, s, t, &row, &pos, &bits)) {
      if (lane == 0 && h == 0) flag_status(a.status, bits);
      continue;
    }
    const int64_t at = t * s.xt + h * s.xh;
    float sum = 0.f;
    for (int i = lane; i < s.D; i += 32) {
      float x;
      if constexpr (F32) x = ((const float*)s.x)[at + i];
      else x = __bfloat162float(((const __nv_bfloat16*)s.x)[at + i]);
      v[i] = x;
      if (i < s.norm_dim) sum += x;
    }
    if (s.norm) {
      const float n = (float)s.norm_dim;
      const float mean = s.norm == MTPSD_NORM_LAYER ? group_sum(sum, 32) / n : 0.f;
      float sq = 0.f;
      for (int i = lane; i < s.norm_dim; i += 32) {
        const float d = v[i] - mean;
        sq = fmaf(d, d, sq);
      }
      const float r = __frsqrt_rn(group_sum(sq, 32) / n + a.eps);
      for (int i = lane; i < s.norm_dim; i += 32) {
        float y = s.w ? mul3<true>(v[i] - mean, r, s.w[i]) : (v[i] - mean) * r;
        if (s.b) y += s.b[i];
        v[i] = y;
      }
    }
    __syncwarp();
    const int half = a.rot_dim >> 1;
    for (int i = lane; i < half; i += 32) {
      const float c = a.cs[pos * a.rot_dim + i], n = a.cs[pos * a.rot_dim + half + i];
      float* p = v + s.rot_start + (a.inter ? 2 * i : i);
      turn(p[0], p[a.inter ? 1 : half], c, n);
    }
    __syncwarp();
    const int64_t base = row * s.ot + h * s.oh;
    if (s.out_type == MTPSD_FP8_E4M3) {
      float m = 0.f;
      for (int i = lane; i < s.D; i += 32) m = fmaxf(m, fabsf(v[i]));
      const float scale = fp8_block_scale(group_max(m, 32));
      for (int i = lane; i < s.D; i += 32)
        ((uint8_t*)s.out)[base + i] = (uint8_t)__nv_cvt_float_to_fp8(__fdiv_rn(v[i], scale), __NV_SATFINITE, __NV_E4M3);
      if (lane == 0) s.scale[row * s.heads + h] = scale;
    } else {
      for (int i = lane; i < s.D; i += 32) {
        if (s.out_type == MTPSD_F32) ((float*)s.out)[base + i] = v[i];
        else ((__nv_bfloat16*)s.out)[base + i] = __float2bfloat16_rn(v[i]);
      }
    }
    __syncwarp();                // the next head overwrites the buffer
  }
}

bool fits16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// Lanes and slots for the vector kernel: 0 (one pair slot), 1 (one and two rest slots), 2 (two and four); -1: the element kernel.
int plan_side(const mtpsd_head_side& c, const NormRopePlan& p, bool key, Side* s) {
  // (the head stride of a single head says nothing)
  s->x = c.x; s->xt = c.x_token_stride; s->xh = c.heads > 1 ? c.x_head_stride : 0;
  s->out = c.out; s->ot = c.out_token_stride; s->oh = c.heads > 1 ? c.out_head_stride : 0; s->scale = c.scale;
  s->w = c.weight; s->b = c.bias;
  s->slots = key ? p.slots : nullptr;
  s->pool = p.pool;
  s->heads = c.heads; s->D = c.D; s->norm = c.norm; s->norm_dim = c.norm ? c.norm_dim : 0; s->rot_start = c.rot_start;
  s->out_type = c.out_dtype;
  s->in_f32 = c.dtype == MTPSD_F32;
  s->skip = c.out == c.x;
  const bool rows = c.out_dtype == MTPSD_FP8_DS_MLA || c.out_dtype == MTPSD_FP4_MLA;
  const int in_vec = s->in_f32 ? 4 : 8;                                              // elements of 16 bytes
  const int out_vec = c.out_dtype == MTPSD_F32 ? 4 : (c.out_dtype == MTPSD_BF16 ? 8 : (rows ? 16 : 8));
  const bool ok = c.D % 8 == 0 && p.rot_dim % 16 == 0 && (!p.rot_dim || c.rot_start % 8 == 0) && (!c.norm || c.norm_dim % 8 == 0) &&
                  fits16(c.x) && c.x_token_stride % in_vec == 0 && s->xh % in_vec == 0 &&
                  ((uintptr_t)c.out % (c.out_dtype == MTPSD_FP8_E4M3 ? 8 : 16)) == 0 && c.out_token_stride % out_vec == 0 &&
                  (rows || s->oh % out_vec == 0) && fits16(c.weight) && fits16(c.bias) && fits16(p.cos_sin);
  if (!ok) return -1;
  s->nr = rows ? 4 : p.rot_dim / 16;
  if (rows) s->rot_start = 512;
  else if (!p.rot_dim) s->rot_start = 0;
  const int rest = c.D / 8 - 2 * s->nr;
  int inst = 2;
  s->lanes = 32;
  for (int L = 4; L <= 32; L *= 2) {
    if (s->nr <= L && rest <= 2 * L && (!rows || L == 32)) {
      s->lanes = L;
      inst = rest == 0 && !(c.norm && p.eps == 0.f) ? 0 : 1;     // (infinite reciprocal roots: mul3)
      break;
    }
  }
  // A lane group takes several heads of a token (up to 8) while that leaves every SM 32 warps: the token's angles are loaded once.
  const int64_t warps = p.T * c.heads * s->lanes / 32;
  int64_t each = warps / (32 * (int64_t)num_sms());
  each = each < 1 ? 1 : (each > 8 ? 8 : each);
  s->groups = (int)ceil_div(c.heads, each);
  s->items = p.T * s->groups;
  s->blocks = (int)ceil_div(s->items, 256 / s->lanes);
  return inst;
}

template <bool F32, int QP, int QR>
void launch_k_side(const Args& a, int ki, cudaStream_t st) {
  const unsigned n = (unsigned)(a.q.blocks + a.k.blocks);
  if (ki == 0) launch_k(norm_rope_kernel<F32, QP, QR, 1, 0>, n, 256, 0, st, a);
  else if (ki == 1) launch_k(norm_rope_kernel<F32, QP, QR, 1, 2>, n, 256, 0, st, a);
  else launch_k(norm_rope_kernel<F32, QP, QR, 2, 4>, n, 256, 0, st, a);
}
template <bool F32>
void launch_sides(const Args& a, int qi, int ki, cudaStream_t st) {
  if (qi == 0) launch_k_side<F32, 1, 0>(a, ki, st);
  else if (qi == 1) launch_k_side<F32, 1, 2>(a, ki, st);
  else launch_k_side<F32, 2, 4>(a, ki, st);
}

}  // namespace

int launch_norm_rope(const NormRopePlan& p, cudaStream_t st) {
  Args a{};
  a.T = p.T; a.positions = p.positions; a.cs = p.cos_sin; a.n_pos = p.n_pos; a.rot_dim = p.rot_dim; a.inter = p.interleaved;
  a.eps = p.eps; a.status = p.status;
  Side side[2] = {};
  int inst[2] = {-2, -2};      // absent
  const mtpsd_head_side* c[2] = {p.q, p.k};
  for (int i = 0; i < 2; ++i)
    if (c[i]) inst[i] = plan_side(*c[i], p, i == 1, &side[i]);
  // Both sides in one launch where both take the vector kernel on one type; but a large call whose sides take different forms of it
  // goes in two, each with as many CTAs per SM as its own registers allow.
  const bool large = inst[0] != inst[1] && side[0].blocks + side[1].blocks > 8 * num_sms();
  if (inst[0] >= 0 && inst[1] >= 0 && side[0].in_f32 == side[1].in_f32 && !large) {
    a.q = side[0];
    a.k = side[1];
    if (a.q.in_f32) launch_sides<true>(a, inst[0], inst[1], st);
    else launch_sides<false>(a, inst[0], inst[1], st);
    return check_launch("norm_rope");
  }
  for (int i = 0; i < 2; ++i) {
    if (inst[i] == -2) continue;
    a.q = Side{};              // blocks 0
    a.k = side[i];
    if (inst[i] >= 0) {
      if (a.k.in_f32) launch_sides<true>(a, inst[i], inst[i], st);
      else launch_sides<false>(a, inst[i], inst[i], st);
    } else if (side[i].out_type == MTPSD_FP8_DS_MLA || side[i].out_type == MTPSD_FP4_MLA) {
      set_error("norm_rope: cache rows need 16-byte aligned rows");   // (refused before: the vector kernel alone writes them)
      return MTPSD_EUNSUPPORTED;
    } else {
      const int64_t want = ceil_div(p.T * side[i].heads, 8), most = 8 * (int64_t)num_sms();
      const unsigned n = (unsigned)(want < most ? want : most);
      if (a.k.in_f32) launch_k(norm_rope_elements_kernel<true>, n, 256, 0, st, a);
      else launch_k(norm_rope_elements_kernel<false>, n, 256, 0, st, a);
    }
    if (int rc = check_launch("norm_rope")) return rc;
  }
  return MTPSD_OK;
}

}  // namespace mtpsd
