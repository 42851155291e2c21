// FP8 product with block-128 scales for many rows: the arithmetic of
// k_gemm_fp8.cu on pairs of CTAs (tcgen05.mma cta_group::2).
//
// A tile is 256 rows of a (operand A, M = 256, 128 per CTA) x 256 outputs
// (operand B, N = 256): each CTA of the pair stages its 128 rows of a and 128
// of the 256 weight rows, and the two tensor cores share both halves of B.  Per
// block a CTA moves 32 KB through shared memory for 4.2 M products, against 48
// KB for a 128 x 256 tile of its own: at the full MMA rate (512 cycles a block)
// the TMA writes and the operand reads then take 256 cycles each of the
// shared-memory port, so that it is no longer the limit.
// The rows of a lie on the TMEM lanes here, so with 128 x 128 weight blocks a
// thread multiplies by one scale per lane and block, without a read per column.
//
// Roles (384 threads, one CTA per SM), as k_gemm_fp8.cu but:
//   warps 0-7   epilogue: lanes 32 (w % 4) .. +31, columns 128 (w / 4) .. +127; 128 accumulators a thread
//               (setmaxnreg moves the other warps' registers here: 208 against 88).
//   warp 8      TMA producer of this CTA's operands; both CTAs' copies complete on the leader's barrier.
//   warp 9      TMEM allocation; in the leader (even) CTA the MMA issue for the pair.
//   warp 10     scales of this CTA's rows of a;  warp 11  scales of the tile's weight rows.
// With few tiles the blocks of K are split over up to 4 pairs of one cluster.
#include <algorithm>
#include <string.h>

#include "gemm_fp8.cuh"

namespace mtpsd {
namespace gtp {
using namespace gtc;

constexpr int ROWS = 128;                 // rows of a per CTA, weight rows per CTA
constexpr int COLS = 256;                 // outputs of a tile
constexpr int EPI_WARPS = 8;
constexpr int PRODUCER_WARP = 8, MMA_WARP = 9, SCALE_WARP = 10;
constexpr int THREADS = 32 * 12;
constexpr int MAX_SPLIT = 4;
constexpr int HALF_BYTES = ROWS * KB;     // one operand's share of a stage
constexpr int STAGE = 2 * HALF_BYTES;
constexpr int NSTAGE = 6;
constexpr int NBUF = TMEM_COLS / COLS;
constexpr int SLOT_FLOATS = SG * (ROWS + COLS);
constexpr int TR_LD = 40;                 // row stride (floats) of 8 rows x 32 columns: fragment rows miss each other's banks
constexpr int TR_LD_BF16 = 36;            // the same in words of two bf16, 8 rows x 64 columns
constexpr int TR_LD_ROWS = 17;            // the same for 32 rows x 16 columns of the one-row-per-thread layout
constexpr int TR_FLOATS = 640;            // per epilogue warp
constexpr int PART_LD = COLS + 8;         // row stride of a partial tile
constexpr int OFF_SCALE = NSTAGE * STAGE;
constexpr int OFF_TR = OFF_SCALE + NSLOT * SLOT_FLOATS * 4;
constexpr int OFF_BAR = OFF_TR + EPI_WARPS * TR_FLOATS * 4;
constexpr int N_BARS = 2 * NSTAGE + 2 * NBUF + 2 * NSLOT + 1;
constexpr int OFF_MISC = OFF_BAR + N_BARS * 8;
constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;         // + alignment slack
constexpr int EPI_REGS = 208, ROLE_REGS = 88;
static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
static_assert(ROWS * PART_LD * 4 <= NSTAGE * STAGE, "the partial tile fits the stage ring");
static_assert(8 * TR_LD <= TR_FLOATS && 8 * TR_LD_BF16 <= TR_FLOATS && 32 * TR_LD_ROWS <= TR_FLOATS, "the transposes fit");
// setmaxnreg shares out what the launch allots: 65536 / 384 threads, rounded down to 8
static_assert(256 * EPI_REGS + 128 * ROLE_REGS <= THREADS * 168, "register split");

struct Params {
  const float* sa;
  const float* sw;
  void* out;
  int64_t ld_out;
  int M, N, kbs;          // rows of a, outputs, blocks of K
  int n_mt, tiles;        // tiles along M, tiles
  int split;              // pairs per cluster
  int out_f32;
  int vec_out;            // bf16 outputs can be stored in pairs
  int vec_rows;           // a row's outputs can be stored 32 bytes at a time
  int vec_scales;         // a block row's scales can be read four at a time
  int32_t* status;
};

__device__ __forceinline__ uint32_t map_rank(uint32_t cta_addr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(cta_addr), "r"(rank));
  return a;
}
// The copy's destination is this CTA's; its bytes complete on the barrier at a cluster address.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(dst), "l"((uint64_t)map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mma_fp8_pair(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(tmem_d),
      "l"(a), "l"(b), "r"(id), "r"(accumulate));
}
// Arrives on the barrier at this offset in both CTAs of the pair when the pair's MMAs so far are done.
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar, uint32_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(saddr(bar)),
      "h"((uint16_t)mask)
      : "memory");
}
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void store_32b(void* at, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ uint32_t bf16_pair(float2 v) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
  return *(const uint32_t*)&b;
}
__device__ __forceinline__ bool wait_all_cluster(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
  return __all_sync(0xffffffffu, mbar::wait<true>(bar, parity, abort_flag, status, mbar::DEFAULT_LIMIT_NS));
}

// ROWS1: the weight's scales are per row and block (else per 128 x 128 block).
template <bool ROWS1>
__global__ void __launch_bounds__(THREADS, 1) gemm_fp8_pair_kernel(const __grid_constant__ CUtensorMap tmap_w,
                                                                   const __grid_constant__ CUtensorMap tmap_a,
                                                                   const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t* full = (uint64_t*)(sm + OFF_BAR);        // the leader's is used
  uint64_t* empty = full + NSTAGE;
  uint64_t* t_full = empty + NSTAGE;
  uint64_t* t_empty = t_full + NBUF;                 // the leader's is used
  uint64_t* s_full = t_empty + NBUF;
  uint64_t* s_empty = s_full + NSLOT;
  uint64_t* drain = s_empty + NSLOT;
  uint32_t* tmem_slot = (uint32_t*)(sm + OFF_MISC);
  volatile int* abort_flag = (volatile int*)(sm + OFF_MISC + 4);
  float* scales = (float*)(sm + OFF_SCALE);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_rank(), leader = crank & ~1u, side = crank & 1u;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NSTAGE; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < NBUF; ++i) {
      mbar_init(&t_full[i], 1);
      mbar_init(&t_empty[i], 2 * EPI_WARPS);
    }
    for (int i = 0; i < NSLOT; ++i) {
      mbar_init(&s_full[i], 2);
      mbar_init(&s_empty[i], EPI_WARPS);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_slot)),
                 "r"(TMEM_COLS));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  if (warp == PRODUCER_WARP && elect_one()) {
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&tmap_w) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&tmap_a) : "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                // both CTAs' barriers exist before any copy or arrival from the other
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();                // the previous kernel's writes are visible from here on
  griddep_launch_dependents();

  const int width = 2 * p.split, part_rank = (int)crank >> 1;
  const int first = (int)blockIdx.x / width, step = (int)gridDim.x / width;       // this cluster's tiles
  const int kb0 = (int)((int64_t)part_rank * p.kbs / p.split), kb1 = (int)((int64_t)(part_rank + 1) * p.kbs / p.split);

  if (warp >= EPI_WARPS) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(ROLE_REGS));
    if (warp == PRODUCER_WARP) {
      int stage = 0, n = 0;
      bool ok = true;
      for (int tile = first; tile < p.tiles && ok; tile += step) {
        const int n0 = tile / p.n_mt * COLS + (int)side * ROWS, m0 = (tile % p.n_mt * 2 + (int)side) * ROWS;
        for (int kb = kb0; kb < kb1; ++kb, ++n) {
          if (n >= NSTAGE) ok = wait_all(&empty[stage], (n / NSTAGE - 1) & 1, abort_flag, p.status);
          if (!ok) break;
          if (elect_one()) {
            const uint32_t dst = saddr(sm + stage * STAGE), bar = map_rank(saddr(&full[stage]), leader);
            if (side == 0) mbar_expect_tx(&full[stage], 2 * STAGE);    // both CTAs' copies
            tma_load_pair(dst, &tmap_a, kb * KB, m0, bar);
            tma_load_pair(dst + HALF_BYTES, &tmap_w, kb * KB, n0, bar);
          }
          __syncwarp();
          if (++stage == NSTAGE) stage = 0;
        }
      }
      if (*abort_flag && side == 0 && lane == 0) {   // drain the pair's copies still in flight (bounded)
        volatile int dummy = 0;
        for (int s = 0; s < NSTAGE; ++s) {
          const int issued = n / NSTAGE + (s < n % NSTAGE ? 1 : 0);   // loads of stage s
          if (issued > 0) mbar::wait<true>(&full[s], (issued - 1) & 1, &dummy, p.status, mbar::DEFAULT_LIMIT_NS);
        }
      }
    } else if (warp == MMA_WARP && side == 0) {
      int stage = 0, n = 0;
      bool ok = true;
      const uint32_t id = (1u << 4) | ((uint32_t)COLS >> 3 << 17) | ((256u >> 4) << 24);   // M = 256, N = 256
      const uint32_t mask = 3u << leader;
      for (int tile = first; tile < p.tiles && ok; tile += step) {
        for (int kb = kb0; kb < kb1; ++kb, ++n) {
          const int buf = n % NBUF, round = n / NBUF;
          ok = wait_all_cluster(&full[stage], (n / NSTAGE) & 1, abort_flag, p.status);
          if (ok && round > 0) ok = wait_all_cluster(&t_empty[buf], (round - 1) & 1, abort_flag, p.status);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t a_base = saddr(sm + stage * STAGE), b_base = a_base + HALF_BYTES;
            const uint32_t d = tmem_base + (uint32_t)(buf * COLS);
#pragma unroll
            for (int kk = 0; kk < KB / 32; ++kk)
              mma_fp8_pair(d, sw128_desc(a_base + kk * 32), sw128_desc(b_base + kk * 32), id, kk > 0 ? 1u : 0u);
            mma_commit_pair(&t_full[buf], mask);
            mma_commit_pair(&empty[stage], mask);
          }
          __syncwarp();
          if (++stage == NSTAGE) stage = 0;
        }
      }
      if (elect_one()) mma_commit_pair(drain, mask);   // every MMA has completed before TMEM is released
      __syncwarp();
      volatile int dummy = 0;
      mbar::wait<false>(drain, 0, &dummy, p.status, mbar::DEFAULT_LIMIT_NS);
    } else if (warp >= SCALE_WARP) {
      // slot: [SG][128] scales of this CTA's rows of a, then [SG][256] of the tile's weight rows (ROWS1) or
      // [SG][2] of its two blocks
      const bool rows = warp == SCALE_WARP;
      int n = 0;
      bool ok = true;
      for (int tile = first; tile < p.tiles && ok; tile += step) {
        const int nt = tile / p.n_mt;
        const float* base = rows ? p.sa : p.sw;
        const int64_t row0 = rows ? (int64_t)(tile % p.n_mt * 2 + (int)side) * ROWS
                                  : ROWS1 ? (int64_t)nt * COLS : (int64_t)nt * (COLS / 128);
        const int64_t end = rows ? p.M : ROWS1 ? p.N : ((int64_t)p.N + 127) / 128;
        const int per = rows ? ROWS : ROWS1 ? COLS : 2;             // scales per block
        const int ld = rows ? ROWS : ROWS1 ? COLS : 2;
        for (int kb = kb0; kb < kb1; kb += SG, ++n) {
          const int slot = n % NSLOT;
          float* dst = scales + slot * SLOT_FLOATS + (rows ? 0 : SG * ROWS);
          bool waited = n < NSLOT;
          for (int i0 = 0; i0 < per; i0 += 128) {
            float v[4][SG];
#pragma unroll
            for (int i = 0; i < 4; ++i) {         // blocks past kb1 and rows past the last: 0
              const int at = i0 + 32 * i + lane;
              v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.f;
              if (at >= per || row0 + at >= end) continue;
              const float* s = base + (row0 + at) * p.kbs + kb;
              if (p.vec_scales && (kb & 3) == 0) {
                const float4 f = __ldg((const float4*)s);
                v[i][0] = f.x; v[i][1] = f.y; v[i][2] = f.z; v[i][3] = f.w;
              } else {
#pragma unroll
                for (int j = 0; j < SG; ++j)
                  if (kb + j < kb1) v[i][j] = __ldg(s + j);
              }
            }
            if (!waited) ok = wait_all(&s_empty[slot], (n / NSLOT - 1) & 1, abort_flag, p.status);
            waited = true;
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (i0 + 32 * i + lane < per)
#pragma unroll
                for (int j = 0; j < SG; ++j) dst[j * ld + i0 + 32 * i + lane] = v[i][j];
          }
          if (!ok) break;
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_full[slot]);
        }
      }
    }
    __syncwarp();
    if (p.split > 1) cluster_sync();   // (1) the partial tiles are written
    cluster_sync();                    // (2) nobody reads another CTA's shared memory or TMEM any more
    if (warp == MMA_WARP) {
      tc_fence_after();
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS));
    }
    return;
  }

  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_REGS));
  const int quarter = warp & 3, c0 = (warp >> 2) * 128;            // this warp's TMEM lanes and first column
  const int fr = lane >> 2, fc = 2 * (lane & 3);                   // fragment row and column of this lane
  // ROWS1: acc[4 g + i]: columns c0 + 8 g + fc, +1, row 32 quarter + 8 i + fr (the 16x256b read of k_gemm_fp8.cu);
  // else acc[i]: columns c0 + 2 i, +1, row 32 quarter + lane (the 32x32b read, twice as fast: 128 x 256 values
  // take 306 cycles, against 612 which the additions then cannot hide)
  float2 acc[64];
  {
    int buf = 0, t_phase = 0, slot = 0, s_phase = 0;
    bool ok = true;
    const uint32_t te0 = map_rank(saddr(&t_empty[0]), leader);
    const uint32_t taddr0 = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)c0;
    for (int tile = first; tile < p.tiles && ok; tile += step) {
      const int m_own = (tile % p.n_mt * 2 + (int)side) * ROWS + quarter * 32;    // the warp's first row of a
      const bool live = m_own < p.M;
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = make_float2(0.f, 0.f);
      for (int kb = kb0, j = 0; kb < kb1; ++kb) {
        if (j == 0) ok = wait_all(&s_full[slot], s_phase, abort_flag, p.status);
        if (!ok) break;
        const float* sc = scales + slot * SLOT_FLOATS;
        float rs[4];                                               // the scales of the thread's rows
        if (ROWS1) {
#pragma unroll
          for (int i = 0; i < 4; ++i) rs[i] = sc[j * ROWS + quarter * 32 + 8 * i + fr];
        } else {
          rs[0] = sc[j * ROWS + quarter * 32 + lane] * sc[SG * ROWS + 2 * j + (c0 >> 7)];
        }
        const float* scw = sc + SG * ROWS + j * COLS + c0 + fc;
        ok = wait_all(&t_full[buf], t_phase, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t taddr = taddr0 + (uint32_t)(buf * COLS);
        if (live) {
          // 32 columns x 32 lanes at a time; the next read is in flight while one is added
          uint32_t t[2][32];
          auto read = [&](int c) {
            if constexpr (ROWS1) {
              tmem_ld_x4(taddr + 32 * c, t[c & 1]);
              tmem_ld_x4(taddr + (16u << 16) + 32 * c, t[c & 1] + 16);
            } else {
              tmem_ld_rows32(taddr + 32 * c, t[c & 1]);
            }
          };
          read(0);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tmem_ld_wait();
            if (c < 3) {
              read(c + 1);
            } else {               // the warp's last read of the buffer
              tc_fence_before();
              __syncwarp();
              if (lane == 0) arrive_at(te0 + 8 * buf);
            }
            if constexpr (ROWS1) {
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                const float2 s = *(const float2*)(scw + 32 * c + 8 * g);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  float2& q = acc[4 * (4 * c + g) + i];
                  const uint32_t* v = t[c & 1] + 16 * (i >> 1) + 4 * g + 2 * (i & 1);
                  q.x = fmaf(__uint_as_float(v[0]), rs[i] * s.x, q.x);
                  q.y = fmaf(__uint_as_float(v[1]), rs[i] * s.y, q.y);
                }
              }
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float2& q = acc[16 * c + i];
                q.x = fmaf(__uint_as_float(t[c & 1][2 * i]), rs[0], q.x);
                q.y = fmaf(__uint_as_float(t[c & 1][2 * i + 1]), rs[0], q.y);
              }
            }
          }
        } else {
          __syncwarp();
          if (lane == 0) arrive_at(te0 + 8 * buf);
        }
        if (++buf == NBUF) {
          buf = 0;
          t_phase ^= 1;
        }
        if (++j == SG || kb == kb1 - 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[slot]);
          j = 0;
          if (++slot == NSLOT) {
            slot = 0;
            s_phase ^= 1;
          }
        }
      }
      if (!ok || p.split > 1) break;
      if (!live) continue;
      const int n_first = tile / p.n_mt * COLS + c0;
      float* tr = (float*)(sm + OFF_TR) + warp * TR_FLOATS;
      if constexpr (!ROWS1) {
        const int es = p.out_f32 ? 4 : 2, row = m_own + lane;
        uint8_t* o = (uint8_t*)p.out + ((int64_t)row * p.ld_out + n_first) * es;
        if (p.vec_rows && n_first + 128 <= p.N) {           // 32 bytes of its own row per thread
          if (row < p.M) {
            if (p.out_f32) {
#pragma unroll
              for (int i = 0; i < 64; i += 4) store_32b(o + 8 * i, (const uint32_t*)&acc[i]);
            } else {
#pragma unroll
              for (int i = 0; i < 64; i += 8) {
                uint32_t v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = bf16_pair(acc[i + e]);
                store_32b(o + 4 * i, v);
              }
            }
          }
        } else {                   // through the warp's own shared memory, so that a store covers 16 consecutive outputs
#pragma unroll
          for (int c = 0; c < 128; c += 16) {
            if (n_first + c >= p.N) break;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              tr[lane * TR_LD_ROWS + 2 * i] = acc[c / 2 + i].x;
              tr[lane * TR_LD_ROWS + 2 * i + 1] = acc[c / 2 + i].y;
            }
            __syncwarp();
            const int col = n_first + c + (lane & 15);
            for (int r = lane >> 4; r < 32; r += 2) {
              if (m_own + r >= p.M) break;
              const float v = tr[r * TR_LD_ROWS + (lane & 15)];
              const int64_t off = (int64_t)(m_own + r) * p.ld_out + col;
              if (col >= p.N) continue;
              if (p.out_f32) ((float*)p.out)[off] = v;
              else ((__nv_bfloat16*)p.out)[off] = __float2bfloat16_rn(v);
            }
            __syncwarp();
          }
        }
        continue;
      }
      // eight rows at a time through the warp's own shared memory, so that a store covers consecutive outputs
      if (p.out_f32) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < 128; c += 32) {
#pragma unroll
            for (int g = 0; g < 4; ++g) *(float2*)(tr + fr * TR_LD + 8 * g + fc) = acc[4 * (c / 8 + g) + i];
            __syncwarp();
            const int col = n_first + c + lane;
            float* o = (float*)p.out + (int64_t)(m_own + 8 * i) * p.ld_out + col;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (m_own + 8 * i + e < p.M && col < p.N) o[e * p.ld_out] = tr[e * TR_LD + lane];
            __syncwarp();
          }
      } else {
        uint32_t* tw = (uint32_t*)tr;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < 128; c += 64) {
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              tw[fr * TR_LD_BF16 + 4 * g + (lane & 3)] = bf16_pair(acc[4 * (c / 8 + g) + i]);
            }
            __syncwarp();
            const int col = n_first + c + 2 * lane;
            __nv_bfloat16* o = (__nv_bfloat16*)p.out + (int64_t)(m_own + 8 * i) * p.ld_out + col;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if (m_own + 8 * i + e >= p.M) break;
              const uint32_t w = tw[e * TR_LD_BF16 + lane];
              if (p.vec_out && col + 1 < p.N) {
                *(uint32_t*)(o + e * p.ld_out) = w;
              } else {
                if (col < p.N) ((uint16_t*)(o + e * p.ld_out))[0] = (uint16_t)w;
                if (col + 1 < p.N) ((uint16_t*)(o + e * p.ld_out))[1] = (uint16_t)(w >> 16);
              }
            }
            __syncwarp();
          }
      }
    }
  }
  __syncwarp();
  if (p.split > 1) {
    // The cluster's one tile: every CTA's accumulators into its own stage ring (the last block's MMAs are
    // done, so no copy or MMA uses it), then each pair sums a part of the rows over the pairs, in order.
    float* part = (float*)sm;                               // [128][PART_LD]
    if constexpr (ROWS1) {
#pragma unroll
      for (int g = 0; g < 16; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *(float2*)(part + (quarter * 32 + 8 * i + fr) * PART_LD + c0 + 8 * g + fc) = acc[4 * g + i];
    } else {
#pragma unroll
      for (int i = 0; i < 64; i += 2)
        *(float4*)(part + (quarter * 32 + lane) * PART_LD + c0 + 2 * i) = make_float4(acc[i].x, acc[i].y, acc[i + 1].x, acc[i + 1].y);
    }
    cluster_sync();                // (1)
    const int m_first = (first % p.n_mt * 2 + (int)side) * ROWS, n_first = first / p.n_mt * COLS;
    const int rows = min(ROWS, p.M - m_first);              // <= 0: this CTA's rows are past the last
    const int r0 = rows > 0 ? part_rank * rows / p.split : 0, r1 = rows > 0 ? (part_rank + 1) * rows / p.split : 0;
    for (int r = r0 + warp; r < r1; r += EPI_WARPS) {
      // a row's 256 outputs: columns 4 lane .. +3 and 128 + 4 lane .. +3, every remote read in flight at once
      float4 v[MAX_SPLIT][2];
#pragma unroll
      for (int q = 0; q < MAX_SPLIT; ++q)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          v[q][h] = q < p.split ? ld_cluster4(saddr(part + r * PART_LD + 128 * h + 4 * lane), 2 * q + side)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float4 sum = v[0][h];
#pragma unroll
        for (int q = 1; q < MAX_SPLIT; ++q)
          if (q < p.split) {
            sum.x += v[q][h].x; sum.y += v[q][h].y; sum.z += v[q][h].z; sum.w += v[q][h].w;
          }
        const int col = n_first + 128 * h + 4 * lane;
        const int64_t off = (int64_t)(m_first + r) * p.ld_out + col;
        const float e[4] = {sum.x, sum.y, sum.z, sum.w};
        if (p.out_f32) {
          if (p.vec_rows && col + 3 < p.N) {
            *(float4*)((float*)p.out + off) = sum;
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (col + i < p.N) ((float*)p.out)[off + i] = e[i];
          }
        } else {
          if (p.vec_rows && col + 3 < p.N) {
            *(uint2*)((__nv_bfloat16*)p.out + off) =
                make_uint2(bf16_pair(make_float2(sum.x, sum.y)), bf16_pair(make_float2(sum.z, sum.w)));
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (col + i < p.N) ((__nv_bfloat16*)p.out)[off + i] = __float2bfloat16_rn(e[i]);
          }
        }
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  cluster_sync();                  // (2)
}

cudaLaunchConfig_t config(unsigned grid, int split, cudaStream_t st, cudaLaunchAttribute* attrs) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = st;
  attrs[0].id = cudaLaunchAttributeClusterDimension;
  attrs[0].val.clusterDim.x = 2 * split;
  attrs[0].val.clusterDim.y = 1;
  attrs[0].val.clusterDim.z = 1;
  attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = 2;
  return cfg;
}

// Clusters of `split` pairs that run at once; cached per device.
int resident_clusters(int split) {
  static std::atomic<int> cache[kMaxCachedDevices][MAX_SPLIT + 1];
  const int dev = current_device();
  const bool cacheable = dev >= 0 && dev < kMaxCachedDevices;
  if (cacheable) {
    const int v = cache[dev][split].load(std::memory_order_relaxed);
    if (v) return v > 0 ? v : 0;
  }
  int n = 0;
  cudaLaunchAttribute attrs[2];
  cudaLaunchConfig_t cfg = config(2u * split, split, 0, attrs);
  if (cudaOccupancyMaxActiveClusters(&n, (void*)gemm_fp8_pair_kernel<false>, &cfg) != cudaSuccess) {
    cudaGetLastError();            // not a fault of the call: such clusters are not used
    n = 0;
  }
  if (cacheable) cache[dev][split].store(n > 0 ? n : -1, std::memory_order_relaxed);
  return n;
}

// Pairs per tile: the split of K with the shortest modelled time, in blocks (as k_gemm_fp8.cu).
int choose_split(int64_t tiles, int kbs) {
  const double fixed = 6, join = 3;
  int best = 0;
  double best_t = 0;
  for (int s = 1; s <= MAX_SPLIT && s <= std::max(kbs, 1); ++s) {
    const int64_t at_once = resident_clusters(s);
    if (at_once < 1) continue;
    const double t = (double)ceil_div(tiles, at_once) * ((double)ceil_div(kbs, s) + fixed + (s > 1 ? join : 0));
    if (best == 0 || t < best_t) {
      best = s;
      best_t = t;
    }
  }
  return best;
}

}  // namespace gtp

int launch_gemm_fp8_pair(const GemmFp8Plan& g, cudaStream_t st) {
  using namespace gtp;
  Params p;
  p.sa = g.a_scale; p.sw = g.w_scale; p.out = g.out; p.ld_out = g.ld_out;
  p.M = (int)g.M; p.N = (int)g.N; p.kbs = (int)(g.K / KB);
  p.n_mt = (int)ceil_div(g.M, 2 * ROWS);
  const int64_t tiles = ceil_div(g.N, COLS) * p.n_mt;
  if (tiles > 0x3fffffffLL / (2 * MAX_SPLIT)) {
    set_error("gemm_fp8_block128: too many output tiles");
    return MTPSD_EUNSUPPORTED;
  }
  p.tiles = (int)tiles;
  p.out_f32 = g.out_f32;
  p.vec_out = !g.out_f32 && g.ld_out % 2 == 0 && (uintptr_t)g.out % 4 == 0;
  p.vec_rows = g.ld_out * (g.out_f32 ? 4 : 2) % 32 == 0 && (uintptr_t)g.out % 32 == 0;
  p.vec_scales = p.kbs % 4 == 0 && (uintptr_t)g.a_scale % 16 == 0 && (uintptr_t)g.w_scale % 16 == 0;
  p.status = g.status;
  CUtensorMap mw, ma;
  if (!make_tma_2d(&mw, 0, g.w, (uint64_t)g.K, (uint64_t)g.N, (uint64_t)g.K, KB, ROWS, true) ||
      !make_tma_2d(&ma, 0, g.a, (uint64_t)g.K, (uint64_t)g.M, (uint64_t)g.K, KB, ROWS, true)) {
    set_error("gemm_fp8_block128: cuTensorMapEncodeTiled failed");
    return MTPSD_ECUDA;
  }
  static std::atomic<uint64_t> attr[2];
  if (!set_smem_limit_once(gemm_fp8_pair_kernel<false>, SMEM_BYTES, attr[0]) ||
      !set_smem_limit_once(gemm_fp8_pair_kernel<true>, SMEM_BYTES, attr[1])) {
    set_error("gemm_fp8_block128: cudaFuncSetAttribute failed");
    return MTPSD_ECUDA;
  }
  p.split = choose_split(p.tiles, p.kbs);
  if (p.split < 1) {
    set_error("gemm_fp8_block128: no pair of CTAs fits the device");
    return MTPSD_EUNSUPPORTED;
  }
  const int64_t clusters = p.split > 1 ? p.tiles : std::min<int64_t>(p.tiles, resident_clusters(1));
  cudaLaunchAttribute attrs[2];
  cudaLaunchConfig_t cfg = config((unsigned)(clusters * 2 * p.split), p.split, st, attrs);
  if (g.w_scale_rows == 1) cudaLaunchKernelEx(&cfg, gemm_fp8_pair_kernel<true>, mw, ma, p);
  else cudaLaunchKernelEx(&cfg, gemm_fp8_pair_kernel<false>, mw, ma, p);
  return check_launch("gemm_fp8_block128");
}

}  // namespace mtpsd
