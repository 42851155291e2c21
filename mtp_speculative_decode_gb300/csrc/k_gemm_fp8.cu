// Matrix product of FP8 E4M3 codes with a float32 scale for each block of 128:
//   out[m,n] = sum_kb sa[m,kb] sw[n',kb] sum_{k in kb} a[m,k] w[n,k]
// on the tensor cores (tcgen05.mma kind::f8f6f4, TMEM accumulators, TMA-staged
// operands).
//
// The scales change with every block of 128 values of K, so the tensor cores
// sum one block at a time: four MMAs of K = 32 into a fresh TMEM buffer, which
// the epilogue warps read, scale and add to float32 accumulators in registers
// while the next blocks' MMAs run into the other buffers.
//
// One MMA has M = 128 weight rows (operand A) and N = up to 256 rows of a
// (operand B), so the rarely-many rows of a cost only as much as there are of
// them and the weight streams through once: a tile is 128 outputs x `cols` rows
// (cols: the rows cut into equal tiles of at most 256, rounded up to 16).  TMEM
// lane = output, column = row of a: an epilogue thread's outputs share their
// weight row, the row scales of a are broadcast reads of shared memory, and a
// warp stores 32 consecutive outputs.
//
// Roles (352 threads, one CTA per SM):
//   warps 0-7   epilogue: warp w reads the TMEM lanes 32 (w % 4) .. +31 and the columns of half w / 4.
//   warp 8      TMA producer: a ring of stages of one block (128 x 128 bytes of w, cols x 128 of a).
//   warp 9      TMEM allocation and MMA issue.
//   warp 10     scales: a ring of slots of four blocks' scales; with 128 x 128 weight blocks it
//               multiplies the one weight scale of the tile's block in, else the slot holds the 128
//               rows' scales too and the epilogue multiplies by its own.
// With few tiles the blocks of K of a tile are split over a cluster of up to 8 CTAs (consecutive
// runs of blocks), which add their accumulators through distributed shared memory in rank order.
// The order of every sum is fixed by the sizes and the device.  Every mbarrier wait is bounded
// (2 s): on expiry the kernel flags MTPSD_STATUS_WAIT_TIMEOUT, drains its copies, frees TMEM and returns.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <string.h>

#include "common.cuh"
#include "internal.h"
#include "mbar.cuh"

namespace mtpsd {
namespace gtc {

constexpr int TILE_N = 128;               // outputs (weight rows) per tile
constexpr int KB = 128;                   // bytes of a block
constexpr int EPI_WARPS = 8;
constexpr int PRODUCER_WARP = 8, MMA_WARP = 9, SCALE_WARP = 10;
constexpr int THREADS = 32 * 11;
constexpr int SG = 4;                     // blocks per scale slot
constexpr int NSLOT = 4;                  // scale slots in flight
constexpr int TMEM_COLS = 512;
constexpr int MAX_SPLIT = 8;
constexpr int W_BYTES = TILE_N * KB;

// NC: accumulator registers per epilogue thread / 32; a tile has at most 64 NC columns
template <int NC>
struct Shape {
  static constexpr int COLS = 64 * NC;
  static constexpr int STAGE = W_BYTES + COLS * KB;
  static constexpr int NSTAGE = 200 * 1024 / STAGE;                     // 8, 6, 5, 4
  static constexpr int BUF_COLS = NC == 3 ? 256 : COLS;                 // TMEM columns of one buffer
  static constexpr int NBUF = TMEM_COLS / BUF_COLS;                     // 8, 4, 2, 2
  static constexpr int SLOT_FLOATS = SG * (COLS + TILE_N);
  static constexpr int OFF_SCALE = NSTAGE * STAGE;
  static constexpr int OFF_BAR = OFF_SCALE + NSLOT * SLOT_FLOATS * 4;
  static constexpr int N_BARS = 2 * NSTAGE + 2 * NBUF + 2 * NSLOT + 1;
  static constexpr int OFF_MISC = OFF_BAR + N_BARS * 8;
  static constexpr int BYTES = OFF_MISC + 16 + 1024;                    // + alignment slack
  static_assert(BYTES <= 232448, "shared memory per CTA");
  static_assert(COLS * TILE_N * 4 <= NSTAGE * STAGE, "the partial tile fits the stage ring");
  static_assert(OFF_BAR % 16 == 0, "barriers are aligned");
};

struct Params {
  const float* sa;
  const float* sw;
  void* out;
  int64_t ld_out;
  int M, N, kbs;          // rows of a, outputs, blocks of K
  int cols;               // columns of a tile (a multiple of 16)
  int n_mt, tiles;        // tiles along M, tiles
  int split;              // CTAs per cluster
  int out_f32;
  int vec_scales;         // a block row's scales can be read four at a time
  int32_t* status;
};

__device__ __forceinline__ uint32_t saddr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(bar)), "r"(count));
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(bar)) : "memory");
}
// Warp-uniform bounded wait (all 32 lanes): false when it gave up.
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
  return __all_sync(0xffffffffu, mbar::wait<false>(bar, parity, abort_flag, status, mbar::DEFAULT_LIMIT_NS));
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      ::"r"(dst), "l"((uint64_t)map), "r"(x), "r"(y), "r"(saddr(bar))
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t pred = 0;
  asm volatile("{\n .reg .b32 rx;\n .reg .pred px;\n elect.sync rx|px, 0xffffffff;\n selp.b32 %0, 1, 0, px;\n}\n"
               : "=r"(pred));
  return pred != 0;
}
// Shared-memory matrix descriptor: K-major, 128-byte swizzle, 8-row atoms of 1024 bytes, version 1.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t smem_byte_addr) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_byte_addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)1 << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
// Instruction descriptor: kind::f8f6f4, E4M3 x E4M3 -> F32, both K-major, M = 128, N = n (a multiple of 16).
__device__ __forceinline__ uint32_t idesc_n(int n) { return (1u << 4) | ((uint32_t)n >> 3 << 17) | ((128u >> 4) << 24); }
__device__ __forceinline__ void mma_fp8(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(tmem_d),
      "l"(a), "l"(b), "r"(id), "r"(accumulate));
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(saddr(bar))
               : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t cta_addr, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(cta_addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
// Pairs of floats in one 64-bit register: the FMA pipe does both in one instruction.
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
  return v;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  uint32_t lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
  return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ void store_out(const Params& p, int64_t off, float v) {
  if (p.out_f32) ((float*)p.out)[off] = v;
  else ((__nv_bfloat16*)p.out)[off] = __float2bfloat16_rn(v);
}

// ROWS1: the weight's scales are per row and block (else per 128 x 128 block).
template <int NC, bool ROWS1>
__global__ void __launch_bounds__(THREADS, 1) gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmap_w,
                                                              const __grid_constant__ CUtensorMap tmap_a,
                                                              const __grid_constant__ Params p) {
  using S = Shape<NC>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t* full = (uint64_t*)(sm + S::OFF_BAR);
  uint64_t* empty = full + S::NSTAGE;
  uint64_t* t_full = empty + S::NSTAGE;
  uint64_t* t_empty = t_full + S::NBUF;
  uint64_t* s_full = t_empty + S::NBUF;
  uint64_t* s_empty = s_full + NSLOT;
  uint64_t* drain = s_empty + NSLOT;
  uint32_t* tmem_slot = (uint32_t*)(sm + S::OFF_MISC);
  volatile int* abort_flag = (volatile int*)(sm + S::OFF_MISC + 4);
  float* scales = (float*)(sm + S::OFF_SCALE);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::NSTAGE; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < S::NBUF; ++i) {
      mbar_init(&t_full[i], 1);
      mbar_init(&t_empty[i], EPI_WARPS);
    }
    for (int i = 0; i < NSLOT; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], EPI_WARPS);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_slot)),
                 "r"(TMEM_COLS));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (warp == PRODUCER_WARP && p.kbs > 0 && elect_one()) {
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&tmap_w) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&tmap_a) : "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();                // the previous kernel's writes are visible from here on
  griddep_launch_dependents();

  const int rank = p.split > 1 ? (int)cluster_rank() : 0;
  const int first = (int)blockIdx.x / p.split, step = (int)gridDim.x / p.split;   // this cluster's tiles
  const int kb0 = (int)((int64_t)rank * p.kbs / p.split), kb1 = (int)((int64_t)(rank + 1) * p.kbs / p.split);
  uint64_t acc[16 * NC];
  constexpr int CH = NC == 4 ? 16 : 32;   // columns per TMEM read: with 128 accumulators there is no room for 32 more

  if (warp == PRODUCER_WARP) {
    int n = 0;
    bool ok = true;
    const uint32_t bytes = (uint32_t)(W_BYTES + p.cols * KB);
    for (int tile = first; tile < p.tiles && ok; tile += step) {
      const int n0 = tile / p.n_mt * TILE_N, m0 = tile % p.n_mt * p.cols;
      for (int kb = kb0; kb < kb1; ++kb, ++n) {
        const int stage = n % S::NSTAGE, round = n / S::NSTAGE;
        if (round > 0) ok = wait_all(&empty[stage], (round - 1) & 1, abort_flag, p.status);
        if (!ok) break;
        if (elect_one()) {
          const uint32_t dst = saddr(sm + stage * S::STAGE);
          mbar_expect_tx(&full[stage], bytes);
          tma_load_2d(dst, &tmap_w, kb * KB, n0, &full[stage]);
          tma_load_2d(dst + W_BYTES, &tmap_a, kb * KB, m0, &full[stage]);
        }
        __syncwarp();
      }
    }
    if (*abort_flag && lane == 0) {   // drain this CTA's copies still in flight (bounded)
      volatile int dummy = 0;
      for (int s = 0; s < S::NSTAGE; ++s) {
        const int issued = n / S::NSTAGE + (s < n % S::NSTAGE ? 1 : 0);   // loads of stage s
        if (issued > 0) mbar::wait<false>(&full[s], (issued - 1) & 1, &dummy, p.status, mbar::DEFAULT_LIMIT_NS);
      }
    }
  } else if (warp == MMA_WARP) {
    int n = 0;
    bool ok = true;
    const uint32_t id = idesc_n(p.cols);
    for (int tile = first; tile < p.tiles && ok; tile += step) {
      for (int kb = kb0; kb < kb1; ++kb, ++n) {
        const int stage = n % S::NSTAGE, buf = n % S::NBUF, round = n / S::NBUF;
        ok = wait_all(&full[stage], (n / S::NSTAGE) & 1, abort_flag, p.status);
        if (ok && round > 0) ok = wait_all(&t_empty[buf], (round - 1) & 1, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t w_base = saddr(sm + stage * S::STAGE), a_base = w_base + W_BYTES;
          const uint32_t d = tmem_base + (uint32_t)(buf * S::BUF_COLS);
#pragma unroll
          for (int kk = 0; kk < KB / 32; ++kk)
            mma_fp8(d, sw128_desc(w_base + kk * 32), sw128_desc(a_base + kk * 32), id, kk > 0 ? 1u : 0u);
          mma_commit(&t_full[buf]);
          mma_commit(&empty[stage]);
        }
        __syncwarp();
      }
    }
    if (elect_one()) mma_commit(drain);   // every MMA has completed before TMEM is released
    __syncwarp();
    volatile int dummy = 0;
    mbar::wait<false>(drain, 0, &dummy, p.status, mbar::DEFAULT_LIMIT_NS);
  } else if (warp == SCALE_WARP) {
    // slot: [SG][COLS] scales of the tile's rows of a, then (ROWS1) [SG][128] scales of its weight rows
    int n = 0;
    bool ok = true;
    // the scales of blocks kb .. kb + 3 of one row (blocks past kb1 and rows past the last: 0)
    auto load4 = [&](const float* base, int64_t row, int64_t rows, int kb, float* v) {
      v[0] = v[1] = v[2] = v[3] = 0.f;
      if (row >= rows) return;
      const float* s = base + row * p.kbs + kb;
      if (p.vec_scales && (kb & 3) == 0 && kb + 3 < p.kbs) {
        const float4 f = __ldg((const float4*)s);
        v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
      } else {
#pragma unroll
        for (int j = 0; j < SG; ++j)
          if (kb + j < kb1) v[j] = __ldg(s + j);
      }
    };
    for (int tile = first; tile < p.tiles && ok; tile += step) {
      const int nt = tile / p.n_mt, m0 = tile % p.n_mt * p.cols;
      for (int kb = kb0; kb < kb1; kb += SG, ++n) {
        float v[2 * NC][SG], w[4][SG], b[SG] = {1.f, 1.f, 1.f, 1.f};
        // all of the slot's loads in flight before the wait for its release
#pragma unroll
        for (int i = 0; i < 2 * NC; ++i)
          if (32 * i < p.cols) load4(p.sa, m0 + 32 * i + lane, p.M, kb, v[i]);
        if (ROWS1) {
#pragma unroll
          for (int i = 0; i < 4; ++i) load4(p.sw, (int64_t)nt * TILE_N + 32 * i + lane, p.N, kb, w[i]);
        } else {
          load4(p.sw, nt, nt + 1, kb, b);
        }
        const int slot = n % NSLOT, round = n / NSLOT;
        if (round > 0) ok = wait_all(&s_empty[slot], (round - 1) & 1, abort_flag, p.status);
        if (!ok) break;
        float* dst = scales + slot * S::SLOT_FLOATS;
#pragma unroll
        for (int i = 0; i < 2 * NC; ++i)
          if (32 * i < p.cols)
#pragma unroll
            for (int j = 0; j < SG; ++j) dst[j * S::COLS + 32 * i + lane] = ROWS1 ? v[i][j] : v[i][j] * b[j];
        if (ROWS1)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < SG; ++j) dst[SG * S::COLS + j * TILE_N + 32 * i + lane] = w[i][j];
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_full[slot]);
      }
    }
  } else {
    const int quarter = warp & 3, c0 = (warp >> 2) * 32 * NC;      // this warp's TMEM lanes and first column
    int n = 0, ns = 0;
    bool ok = true;
    for (int tile = first; tile < p.tiles && ok; tile += step) {
#pragma unroll
      for (int i = 0; i < 16 * NC; ++i) acc[i] = 0ull;
      for (int kb = kb0; kb < kb1; ++kb, ++n) {
        const int slot = ns % NSLOT, j = (kb - kb0) % SG;
        if (j == 0) ok = wait_all(&s_full[slot], (ns / NSLOT) & 1, abort_flag, p.status);
        const int buf = n % S::NBUF;
        if (ok) ok = wait_all(&t_full[buf], (n / S::NBUF) & 1, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
        const float* sc = scales + slot * S::SLOT_FLOATS + j * S::COLS + c0;
        uint64_t rw = 0;
        if (ROWS1) {
          const uint32_t r = __float_as_uint(scales[slot * S::SLOT_FLOATS + SG * S::COLS + j * TILE_N + quarter * 32 + lane]);
          rw = pack2(r, r);
        }
        const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(buf * S::BUF_COLS + c0);
        const int mine = min(32 * NC, p.cols - c0) + CH - 1;          // chunks with columns of the tile
#pragma unroll
        for (int c = 0; c < 32 * NC / CH; ++c) {
          if ((c + 1) * CH > mine) break;
          uint32_t t[CH];
          if constexpr (CH == 32) tmem_ld32(taddr + CH * c, t);
          else tmem_ld16(taddr + CH * c, t);
          tmem_ld_wait();
          if ((c + 2) * CH > mine || c == 32 * NC / CH - 1) {      // the warp's last read of the buffer
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&t_empty[buf]);
          }
#pragma unroll
          for (int i = 0; i < CH / 4; ++i) {
            const ulonglong2 s = *(const ulonglong2*)(sc + CH * c + 4 * i);
            const uint64_t s0 = ROWS1 ? mul2(s.x, rw) : s.x, s1 = ROWS1 ? mul2(s.y, rw) : s.y;
            uint64_t* q = acc + CH / 2 * c + 2 * i;
            q[0] = fma2(pack2(t[4 * i], t[4 * i + 1]), s0, q[0]);
            q[1] = fma2(pack2(t[4 * i + 2], t[4 * i + 3]), s1, q[1]);
          }
        }
        if (mine < CH) {            // no columns: release the buffer at once
          __syncwarp();
          if (lane == 0) mbar_arrive(&t_empty[buf]);
        }
        if (j == SG - 1 || kb == kb1 - 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[slot]);
          ++ns;
        }
      }
      if (!ok || p.split > 1) break;
      const int64_t n_out = (int64_t)(tile / p.n_mt) * TILE_N + quarter * 32 + lane;
      const int m0 = tile % p.n_mt * p.cols + c0, m_end = min(p.M, tile % p.n_mt * p.cols + p.cols);
      if (n_out < p.N) {
        int64_t off = (int64_t)m0 * p.ld_out + n_out;
#pragma unroll
        for (int i = 0; i < 16 * NC; ++i) {
          const float2 v = unpack2(acc[i]);
          if (m0 + 2 * i < m_end) store_out(p, off, v.x);
          if (m0 + 2 * i + 1 < m_end) store_out(p, off + p.ld_out, v.y);
          off += 2 * p.ld_out;
        }
      }
    }
  }

  __syncwarp();
  if (p.split > 1) {
    // The cluster's one tile: every rank's accumulators into its own stage ring (its copies and MMAs are
    // done: the epilogue has seen the last block), then each rank sums a part of the columns over the ranks.
    float* part = (float*)sm;                               // [cols][128 outputs]
    __syncthreads();
    if (warp < EPI_WARPS) {
      const int quarter = warp & 3, c0 = (warp >> 2) * 32 * NC;
#pragma unroll
      for (int i = 0; i < 16 * NC; ++i) {
        const float2 v = unpack2(acc[i]);
        part[(c0 + 2 * i) * TILE_N + quarter * 32 + lane] = v.x;
        part[(c0 + 2 * i + 1) * TILE_N + quarter * 32 + lane] = v.y;
      }
    }
    cluster_sync();
    if (warp < EPI_WARPS) {
      const int tile = first;
      const int m0 = tile % p.n_mt * p.cols, m_cols = min(p.cols, p.M - m0);
      const int r0 = (int)((int64_t)rank * m_cols / p.split), r1 = (int)((int64_t)(rank + 1) * m_cols / p.split);
      const int o = threadIdx.x & (TILE_N - 1);
      const int64_t n_out = (int64_t)(tile / p.n_mt) * TILE_N + o;
      for (int c = r0 + (threadIdx.x >> 7); c < r1; c += 2) {
        const uint32_t at = saddr(part + c * TILE_N + o);
        float v[MAX_SPLIT];
#pragma unroll
        for (int r = 0; r < MAX_SPLIT; ++r) v[r] = r < p.split ? ld_cluster(at, r) : 0.f;
        float sum = v[0];
#pragma unroll
        for (int r = 1; r < MAX_SPLIT; ++r)
          if (r < p.split) sum += v[r];
        if (n_out < p.N) store_out(p, (int64_t)(m0 + c) * p.ld_out + n_out, sum);
      }
    }
    cluster_sync();                // no CTA leaves while another reads its shared memory
  }
  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS));
  }
}

using Kernel = void (*)(const CUtensorMap, const CUtensorMap, const Params);

template <bool ROWS1>
Kernel pick(int nc) {
  switch (nc) {
    case 1: return gemm_fp8_kernel<1, ROWS1>;
    case 2: return gemm_fp8_kernel<2, ROWS1>;
    case 3: return gemm_fp8_kernel<3, ROWS1>;
    default: return gemm_fp8_kernel<4, ROWS1>;
  }
}

int smem_bytes(int nc) {
  return nc == 1 ? Shape<1>::BYTES : nc == 2 ? Shape<2>::BYTES : nc == 3 ? Shape<3>::BYTES : Shape<4>::BYTES;
}

cudaLaunchConfig_t config(unsigned grid, int split, int nc, cudaStream_t st, cudaLaunchAttribute* attrs) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem_bytes(nc);
  cfg.stream = st;
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = split;
  attrs[1].val.clusterDim.y = 1;
  attrs[1].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = split > 1 ? 2 : 1;
  return cfg;
}

// Clusters of `split` CTAs that run at once (one CTA per SM); cached per device.
int resident_clusters(int split) {
  if (split == 1) return num_sms();
  static std::atomic<int> cache[kMaxCachedDevices][MAX_SPLIT + 1];
  const int dev = current_device();
  const bool cacheable = dev >= 0 && dev < kMaxCachedDevices;
  if (cacheable) {
    const int v = cache[dev][split].load(std::memory_order_relaxed);
    if (v) return v > 0 ? v : 0;
  }
  int n = 0;
  cudaLaunchAttribute attrs[2];
  cudaLaunchConfig_t cfg = config((unsigned)split, split, 4, 0, attrs);
  if (cudaOccupancyMaxActiveClusters(&n, (void*)gemm_fp8_kernel<4, false>, &cfg) != cudaSuccess) {
    cudaGetLastError();            // not a fault of the call: such clusters are not used
    n = 0;
  }
  if (cacheable) cache[dev][split].store(n > 0 ? n : -1, std::memory_order_relaxed);
  return n;
}

// CTAs per tile: the split of K with the shortest modelled time, in blocks: waves of tiles, each of
// (its share of the blocks + the cost of starting, summing and storing a tile).
int choose_split(int64_t tiles, int kbs) {
  const double fixed = 6, join = 3;
  int best = 1;
  double best_t = 0;
  for (int s = 1; s <= MAX_SPLIT && s <= std::max(kbs, 1); ++s) {
    const int64_t at_once = resident_clusters(s);
    if (at_once < 1) continue;
    const double t = (double)ceil_div(tiles, at_once) * ((double)ceil_div(kbs, s) + fixed + (s > 1 ? join : 0));
    if (s == 1 || t < best_t) {
      best = s;
      best_t = t;
    }
  }
  return best;
}

}  // namespace gtc

int launch_gemm_fp8(const GemmFp8Plan& g, cudaStream_t st) {
  using namespace gtc;
  if (cc_major() != 10 || !tma_available()) {
    set_error("gemm_fp8_block128: needs a GPU of compute capability 10.x");
    return MTPSD_EUNSUPPORTED;
  }
  Params p;
  p.sa = g.a_scale; p.sw = g.w_scale; p.out = g.out; p.ld_out = g.ld_out;
  p.M = (int)g.M; p.N = (int)g.N; p.kbs = (int)(g.K / KB);
  p.n_mt = (int)ceil_div(g.M, 256);
  p.cols = (int)(ceil_div(ceil_div(g.M, p.n_mt), 16) * 16);
  const int64_t tiles = ceil_div(g.N, TILE_N) * p.n_mt;
  if (tiles > 0x3fffffffLL / MAX_SPLIT) {
    set_error("gemm_fp8_block128: too many output tiles");
    return MTPSD_EUNSUPPORTED;
  }
  p.tiles = (int)tiles;
  p.out_f32 = g.out_f32;
  p.vec_scales = p.kbs % 4 == 0 && (uintptr_t)g.a_scale % 16 == 0 && (uintptr_t)g.w_scale % 16 == 0;
  p.status = g.status;
  const int nc = (p.cols + 63) / 64;
  CUtensorMap mw, ma;
  memset(&mw, 0, sizeof(mw));
  memset(&ma, 0, sizeof(ma));
  if (p.kbs > 0 && (!make_tma_2d(&mw, 0, g.w, (uint64_t)g.K, (uint64_t)g.N, (uint64_t)g.K, KB, TILE_N, true) ||
                    !make_tma_2d(&ma, 0, g.a, (uint64_t)g.K, (uint64_t)g.M, (uint64_t)g.K, KB, (uint32_t)p.cols, true))) {
    set_error("gemm_fp8_block128: cuTensorMapEncodeTiled failed");
    return MTPSD_ECUDA;
  }
  const bool rows1 = g.w_scale_rows == 1;
  Kernel kern = rows1 ? pick<true>(nc) : pick<false>(nc);
  static std::atomic<uint64_t> attr[8], attr4;
  if (!set_smem_limit_once(kern, smem_bytes(nc), attr[(rows1 ? 4 : 0) + nc - 1]) ||
      !set_smem_limit_once(gemm_fp8_kernel<4, false>, smem_bytes(4), attr4)) {
    set_error("gemm_fp8_block128: cudaFuncSetAttribute failed");
    return MTPSD_ECUDA;
  }
  p.split = choose_split(p.tiles, p.kbs);
  const unsigned grid = p.split > 1 ? (unsigned)(p.tiles * p.split) : (unsigned)std::min<int64_t>(p.tiles, num_sms());
  cudaLaunchAttribute attrs[2];
  cudaLaunchConfig_t cfg = config(grid, p.split, nc, st, attrs);
  cudaLaunchKernelEx(&cfg, kern, mw, ma, p);
  return check_launch("gemm_fp8_block128");
}

}  // namespace mtpsd
