// FP8 product with block-128 scales for many rows: the arithmetic of
// k_gemm_fp8.cu on pairs of CTAs (tcgen05.mma cta_group::2).
//
// A tile is 256 rows of a (operand A, M = 256, 128 per CTA) x 64 NP outputs
// (operand B, N = 128, 192 or 256, chosen so that the tiles fill the last wave):
// each CTA of the pair stages its 128 rows of a and half of the weight rows, and
// the two tensor cores share both halves of B.  With N = 256, per
// block a CTA moves 32 KB through shared memory for 4.2 M products, against 48
// KB for a 128 x 256 tile of its own: at the full MMA rate (512 cycles a block)
// the TMA writes and the operand reads then take 256 cycles each of the
// shared-memory port, so that it is no longer the limit.
// The rows of a lie on the TMEM lanes here, so with 128 x 128 weight blocks a
// thread multiplies by one scale per lane and block, without a read per column.
//
// Roles (384 threads, one CTA per SM), as k_gemm_fp8.cu but:
//   warps 0-7   epilogue: lanes 32 (w % 4) .. +31, of every 64 columns the 32 of half w / 4; 32 NP
//               accumulators a thread (setmaxnreg moves the other warps' registers here: 208 against 88).
//               Sixteen warps of half as many were slower (697 against 601 us at 768 x 154880 x 6144): a warp's waits and
//               hand-offs cost the same whatever it adds.  That was before the scales and probes were fetched a block
//               ahead, and has not been measured since.
//   warp 8      TMA producer of this CTA's operands; both CTAs' copies complete on the leader's barrier.
//   warp 9      TMEM allocation; in the leader (even) CTA the MMA issue for the pair.
//   warp 10     scales of this CTA's rows of a;  warp 11  scales of the tile's weight rows.
// What bounds it: 768 x 154880 x 6144 with quantised normal values takes 585 us as one call between kernels that draw
// little (2070 MHz, 2.5 PFLOP/s) and 625 to 637 back to back, where the GPU is at its power limit (1389 of 1400 W, down to
// 1702 MHz); 192 rows 205 and 223.  The tensor cores are busy half of the time, and an epilogue warp's 910 cycles a block
// set the pace (the reads of TMEM and the additions 400, the fetch of the next scales and barrier 180, the hand-over of the
// buffer and the first read's latency most of the rest).  On codes of one sign, 564 us as it is: reads of 16 columns at a
// time 583; the buffer handed over in two halves, so that four are in flight, 727 (twice the hand-overs); the next block's
// first read in front of this block's last additions 667 (spills).  Zeros for codes draw 755 W.
// ROWS1: 192 x 154880 x 6144 takes 315 us, 768 rows 923, 256 x 6144 x 6144 24.0 (19.8 with 128 x 128 blocks): it reads TMEM
// in the 16x256b shape, and a scale for every column.
// With few tiles the blocks of K are split over up to 4 pairs of one cluster.
#include <algorithm>

#include "gemm_fp8.cuh"

namespace mtpsd {
namespace gtp {
using namespace gtc;

constexpr int ROWS = 128;                 // rows of a per CTA, weight rows per CTA
constexpr int COLS = 256;                 // most outputs of a tile
constexpr int RUNS = COLS / 64;           // runs of 64 outputs: each lies in one 128 x 128 weight block
constexpr int PW = 2;                     // 16-column pieces of a run of 64 per epilogue warp
constexpr int EPI_WARPS = 8;
constexpr int PRODUCER_WARP = 8, MMA_WARP = 9, SCALE_WARP = 10;
constexpr int THREADS = 32 * 12;
constexpr int MAX_SPLIT = 4;
constexpr int HALF_BYTES = ROWS * KB;     // one operand's share of a stage
constexpr int STAGE = 2 * HALF_BYTES;
constexpr int NSTAGE = 6;
constexpr int NBUF = TMEM_COLS / COLS;
constexpr int SLOT_FLOATS = SG * (ROWS + COLS);
constexpr int TR_LD = 9;                  // row stride (floats) of the transposed store of 32 rows x 8 columns
constexpr int TR_FLOATS = 32 * TR_LD;     // per epilogue warp
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
__device__ __forceinline__ void st_cluster1(uint32_t cta_addr, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_rank(cta_addr, rank)), "r"(v) : "memory");
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

// NP: a tile has 64 NP outputs.  ROWS1: the weight's scales are per row and block (else per 128 x 128 block).
template <int NP, bool ROWS1>
__global__ void __launch_bounds__(THREADS, 1) gemm_fp8_pair_kernel(const __grid_constant__ CUtensorMap tmap_w,
                                                                   const __grid_constant__ CUtensorMap tmap_a,
                                                                   const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + (-saddr(smem_raw) & 1023u);     // no cast: loads stay loads of shared memory
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

  constexpr int BN = 64 * NP;
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
        const int n0 = tile / p.n_mt * BN + (int)side * (BN / 2), m0 = (tile % p.n_mt * 2 + (int)side) * ROWS;
        for (int kb = kb0; kb < kb1; ++kb, ++n) {
          if (n >= NSTAGE) ok = wait_all(&empty[stage], (n / NSTAGE - 1) & 1, abort_flag, p.status);
          if (!ok) break;
          if (elect_one()) {
            const uint32_t dst = saddr(sm + stage * STAGE), bar = map_rank(saddr(&full[stage]), leader);
            if (side == 0) mbar_expect_tx(&full[stage], 2u * HALF_BYTES + (uint32_t)(BN * KB));    // both CTAs' copies
            tma_load_pair(dst, &tmap_a, kb * KB, m0, bar);
            tma_load_pair(dst + HALF_BYTES, &tmap_w, kb * KB, n0, bar);
          }
          __syncwarp();
          if (++stage == NSTAGE) stage = 0;
        }
      }
      // The leader's commits arrive in both CTAs: every one is awaited, so that none is still on its way to the shared
      // memory of a CTA that has left.
      for (int s = 0; s < NSTAGE && ok; ++s) {
        const int issued = n / NSTAGE + (s < n % NSTAGE ? 1 : 0);     // loads of stage s
        if (issued > 0) ok = wait_all(&empty[s], (issued - 1) & 1, abort_flag, p.status);
      }
      // The pair's copies land before its CTAs leave, whoever waits for them: after an expired wait nobody else may.  Copies of
      // the odd CTA that the leader has not announced have had the limit of that CTA's own waits to land.
      if (side == 0 && lane == 0) {
        for (int s = 0; s < NSTAGE; ++s) {
          const int issued = n / NSTAGE + (s < n % NSTAGE ? 1 : 0);   // loads of stage s
          if (issued > 0) mbar::drain<true>(&full[s], (issued - 1) & 1, p.status);
        }
      }
    } else if (warp == MMA_WARP) {
      if (side == 0 && elect_one()) {      // one thread of the pair waits and issues
        int stage = 0, n = 0;
        bool ok = true;
        const uint32_t id = (1u << 4) | ((uint32_t)BN >> 3 << 17) | ((256u >> 4) << 24);   // M = 256, N = BN
        const uint32_t mask = 3u << leader;
        for (int tile = first; tile < p.tiles && ok; tile += step) {
          for (int kb = kb0; kb < kb1; ++kb, ++n) {
            const int buf = n % NBUF, round = n / NBUF;
            ok = mbar::wait<true>(&full[stage], (n / NSTAGE) & 1, abort_flag, p.status, mbar::DEFAULT_LIMIT_NS);
            if (ok && round > 0)
              ok = mbar::wait<true>(&t_empty[buf], (round - 1) & 1, abort_flag, p.status, mbar::DEFAULT_LIMIT_NS);
            if (!ok) break;
            tc_fence_after();
            const uint64_t a = sw128_desc(saddr(sm + stage * STAGE));
            const uint32_t d = tmem_base + (uint32_t)(buf * COLS);
#pragma unroll
            for (int kk = 0; kk < KB / 32; ++kk)         // descriptors count 16 bytes
              mma_fp8_pair(d, a + 2 * kk, a + (HALF_BYTES >> 4) + 2 * kk, id, kk > 0 ? 1u : 0u);
            mma_commit_pair(&t_full[buf], mask);
            mma_commit_pair(&empty[stage], mask);
            if (++stage == NSTAGE) stage = 0;
          }
        }
        mma_commit_pair(drain, mask);                    // every MMA has completed before TMEM is released
      }
      __syncwarp();
      mbar::drain<true>(drain, 0, p.status);        // in both CTAs: the last commit arrives in both
    } else if (warp >= SCALE_WARP) {
      // slot: [SG][128] scales of this CTA's rows of a, then [SG][256] of the tile's weight rows (ROWS1) or
      // [SG][4] of the blocks of its runs of 64
      const bool rows = warp == SCALE_WARP;
      int n = 0;
      bool ok = true;
      for (int tile = first; tile < p.tiles && ok; tile += step) {
        const int nt = tile / p.n_mt;
        const float* base = rows ? p.sa : p.sw;
        const int64_t row0 = rows ? (int64_t)(tile % p.n_mt * 2 + (int)side) * ROWS : (int64_t)nt * BN;
        const int64_t end = rows ? p.M : p.N;
        const int per = rows ? ROWS : ROWS1 ? BN : NP;      // scales per block
        const int ld = rows ? ROWS : ROWS1 ? COLS : RUNS;
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
              int64_t row = row0 + (rows || ROWS1 ? at : 64 * at);
              if (at >= per || row >= end) continue;
              if (!rows && !ROWS1) row >>= 7;
              const float* s = base + row * p.kbs + kb;
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
  const int quarter = warp & 3, c0 = 16 * PW * (warp >> 2);        // this warp's TMEM lanes and columns 64 r + c0 .. +31
  const int fr = lane >> 2, fc = 2 * (lane & 3);                   // fragment row and column of this lane
  // Piece c holds the columns at(c) = 64 (c / PW) + 16 (c % PW) + c0 .. +15.  ROWS1: acc[8 c + 4 g + i]: columns
  // at(c) + 8 g + fc, +1, row 32 quarter + 8 i + fr (the 16x256b read of k_gemm_fp8.cu); else acc[8 c + i]: columns
  // at(c) + 2 i, +1, row 32 quarter + lane (the 32x32b read, twice as fast: 768 x 154880 x 6144 took 855 us with the other)
  uint64_t acc[8 * NP * PW];
  // A wait that gave up makes the warp walk on without waiting, to the end, and store nothing: the blocks' loop then has
  // no exit to test for.
  bool gave_up = false;
  auto finish = [&](uint64_t* bar, uint32_t parity) {               // of a wait whose first probe failed
    if (!gave_up) gave_up = !mbar::wait<false>(bar, parity, abort_flag, p.status, mbar::DEFAULT_LIMIT_NS);
  };
  {
    int n = 0, slot = 0, s_phase = 0;             // blocks so far, scale slot
    const uint32_t te0 = map_rank(saddr(&t_empty[0]), leader);
    const uint32_t taddr0 = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)c0;
    for (int tile = first; tile < p.tiles; tile += step) {
      const int m_own = (tile % p.n_mt * 2 + (int)side) * ROWS + quarter * 32;    // the warp's first row of a
      const bool live = m_own < p.M;
#pragma unroll
      for (int i = 0; i < 8 * NP * PW; ++i) acc[i] = 0ull;
      // The scales of a block and the probe for its products are fetched while the block before is still being
      // added: the chain of a block (waits, scales, reads of TMEM) is what bounds this loop.
      float rs[4];
      float4 w4;
      const float* scw;
      bool ready;
      auto fetch = [&](int j, int block) {
        const float* sc = scales + slot * SLOT_FLOATS + j * ROWS + quarter * 32;
        scw = scales + slot * SLOT_FLOATS + SG * ROWS + j * (ROWS1 ? COLS : RUNS);
        if constexpr (ROWS1) {
#pragma unroll
          for (int i = 0; i < 4; ++i) rs[i] = sc[8 * i + fr];
        } else {
          w4 = *(const float4*)scw;
          rs[0] = sc[lane];
        }
        ready = mbar::try_wait<false>(&t_full[block % NBUF], block / NBUF & 1);
      };
      auto next_slot = [&]() {
        if (!mbar::try_wait<false>(&s_full[slot], s_phase)) finish(&s_full[slot], s_phase);
        __syncwarp();
      };
      auto leave_slot = [&]() {                   // every lane has read its scales
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[slot]);
        if (++slot == NSLOT) {
          slot = 0;
          s_phase ^= 1;
        }
      };
      next_slot();
      fetch(0, n);
      for (int kb = kb0, j = 0; kb < kb1; ++kb, ++n) {
        const int buf = n % NBUF;
        const bool last = kb == kb1 - 1;
        auto fetch_next = [&]() {
          if (++j == SG || last) {
            leave_slot();
            j = 0;
            if (last) return;
            next_slot();
          }
          fetch(j, n + 1);
        };
        uint64_t ws[NP];
        if constexpr (!ROWS1) {
          const float w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
          for (int i = 0; i < NP; ++i) ws[i] = pack2(make_float2(rs[0] * w[i], rs[0] * w[i]));
        }
        if (!ready) finish(&t_full[buf], n / NBUF & 1);
        __syncwarp();
        tc_fence_after();
        const uint32_t taddr = taddr0 + (uint32_t)(buf * COLS);
        if (live) {
          // the 32 columns of a run x 32 lanes at a time; the next run's read is in flight while one is added
          uint32_t t[2][32];
          auto read = [&](int r) {
            if constexpr (ROWS1) {
              tmem_ld_x2(taddr + 64 * r, t[r & 1]);
              tmem_ld_x2(taddr + (16u << 16) + 64 * r, t[r & 1] + 8);
              tmem_ld_x2(taddr + 64 * r + 16, t[r & 1] + 16);
              tmem_ld_x2(taddr + (16u << 16) + 64 * r + 16, t[r & 1] + 24);
            } else {
              tmem_ld_rows16(taddr + 64 * r, t[r & 1]);
              tmem_ld_rows16(taddr + 64 * r + 16, t[r & 1] + 16);
            }
          };
          read(0);
#pragma unroll
          for (int r = 0; r < NP; ++r) {
            tmem_ld_wait();
            if (r + 1 < NP) {
              read(r + 1);
            } else {               // the warp's last read of the buffer
              tc_fence_before();
              __syncwarp();
              if (lane == 0) arrive_at(te0 + 8 * buf);
              if constexpr (!ROWS1) fetch_next();
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int c = 2 * r + h;
              const uint32_t* tt = t[r & 1] + 16 * h;
              if constexpr (ROWS1) {
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                  const uint64_t s = *(const uint64_t*)(scw + 64 * r + 16 * h + c0 + 8 * g + fc);
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    uint64_t& q = acc[8 * c + 4 * g + i];
                    const uint32_t* v = tt + 8 * (i >> 1) + 4 * g + 2 * (i & 1);
                    q = fma2(pack2(v[0], v[1]), mul2(s, pack2(make_float2(rs[i], rs[i]))), q);
                  }
                }
              } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[8 * c + i] = fma2(pack2(tt[2 * i], tt[2 * i + 1]), ws[r], acc[8 * c + i]);
              }
            }
          }
          if constexpr (ROWS1) fetch_next();
        } else {
          if (lane == 0) arrive_at(te0 + 8 * buf);
          fetch_next();
        }
      }
      if (__any_sync(0xffffffffu, gave_up)) break;
      if (p.split > 1) break;
      if (!live) continue;
      const int n_first = tile / p.n_mt * BN + c0;
      if constexpr (!ROWS1) {
        if (p.vec_rows && tile / p.n_mt * BN + BN <= p.N) {          // 32 bytes of its own row per thread
          const int es = p.out_f32 ? 4 : 2, row = m_own + lane;
          uint8_t* o = (uint8_t*)p.out + ((int64_t)row * p.ld_out + n_first) * es;
          if (row < p.M) {
#pragma unroll
            for (int c = 0; c < NP * PW; ++c) {
              const int at = 64 * (c / PW) + 16 * (c % PW);
              if (p.out_f32) {
                store_32b(o + 4 * at, (const uint32_t*)&acc[8 * c]);
                store_32b(o + 4 * at + 32, (const uint32_t*)&acc[8 * c + 4]);
              } else {
                uint32_t v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = bf16_pair(unpack2(acc[8 * c + e]));
                store_32b(o + 2 * at, v);
              }
            }
          }
          continue;
        }
      }
      // eight columns at a time through the warp's own shared memory, so that a store covers consecutive outputs
      float* tr = (float*)(sm + OFF_TR) + warp * TR_FLOATS;
#pragma unroll
      for (int c = 0; c < NP * PW; ++c)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int col0 = n_first + 64 * (c / PW) + 16 * (c % PW) + 8 * g;
          if (col0 >= p.N) break;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 v = unpack2(acc[8 * c + 4 * g + i]);
            float* at = ROWS1 ? tr + (8 * i + fr) * TR_LD + fc : tr + lane * TR_LD + 2 * i;
            at[0] = v.x;
            at[1] = v.y;
          }
          __syncwarp();
          const int col = col0 + (lane & 7);
#pragma unroll
          for (int r0 = 0; r0 < 32; r0 += 4) {
            const int r = r0 + (lane >> 3);
            if (m_own + r >= p.M || col >= p.N) continue;
            const float v = tr[r * TR_LD + (lane & 7)];
            const int64_t off = (int64_t)(m_own + r) * p.ld_out + col;
            if (p.out_f32) ((float*)p.out)[off] = v;
            else ((__nv_bfloat16*)p.out)[off] = __float2bfloat16_rn(v);
          }
          __syncwarp();
        }
    }
  }
  __syncwarp();
  if (p.split > 1) {
    // The cluster's one tile: every CTA's accumulators into its own stage ring (the last block's MMAs are
    // done, so no copy or MMA uses it), then each pair sums a part of the rows over the pairs, in order.
    float* part = (float*)sm;                               // [128][PART_LD]
#pragma unroll
    for (int c = 0; c < NP * PW; ++c)
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = 64 * (c / PW) + 16 * (c % PW) + c0 + 8 * g;
          *(uint64_t*)(ROWS1 ? part + (quarter * 32 + 8 * i + fr) * PART_LD + at + fc
                             : part + (quarter * 32 + lane) * PART_LD + at + 2 * i) = acc[8 * c + 4 * g + i];
        }
    if (gave_up)                   // these sums are not all there (and copies may still come on top): no CTA is to store the tile
      for (int q = 0; q < 2 * p.split; ++q) st_cluster1(saddr((const void*)abort_flag), q, 1u);
    cluster_sync();                // (1)
    const int m_first = (first % p.n_mt * 2 + (int)side) * ROWS, n_first = first / p.n_mt * BN;
    const int n_end = min(p.N, n_first + BN);
    const int rows = *abort_flag ? 0 : min(ROWS, p.M - m_first);      // <= 0: this CTA's rows are past the last
    const int r0 = rows > 0 ? part_rank * rows / p.split : 0, r1 = rows > 0 ? (part_rank + 1) * rows / p.split : 0;
    for (int r = r0 + (warp >> 1); r < r1; r += EPI_WARPS / 2) {
      // half a row per warp, four columns per thread, every remote read in flight at once (columns past the
      // tile's are read too, inside the partial tile, and dropped)
      const int at = 128 * (warp & 1) + 4 * lane;
      float4 v[MAX_SPLIT];
#pragma unroll
      for (int q = 0; q < MAX_SPLIT; ++q)
        v[q] = q < p.split ? ld_cluster4(saddr(part + r * PART_LD + at), 2 * q + side) : make_float4(0.f, 0.f, 0.f, 0.f);
      float4 sum = v[0];
#pragma unroll
      for (int q = 1; q < MAX_SPLIT; ++q)
        if (q < p.split) {
          sum.x += v[q].x; sum.y += v[q].y; sum.z += v[q].z; sum.w += v[q].w;
        }
      const int col = n_first + at;
      const int64_t off = (int64_t)(m_first + r) * p.ld_out + col;
      if (p.vec_rows && col + 3 < n_end) {
        if (p.out_f32) *(float4*)((float*)p.out + off) = sum;
        else *(uint2*)((__nv_bfloat16*)p.out + off) =
            make_uint2(bf16_pair(make_float2(sum.x, sum.y)), bf16_pair(make_float2(sum.z, sum.w)));
      } else {
        const float e[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (col + i < n_end) {
            if (p.out_f32) ((float*)p.out)[off + i] = e[i];
            else ((__nv_bfloat16*)p.out)[off + i] = __float2bfloat16_rn(e[i]);
          }
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  cluster_sync();                  // (2)
}

using Kernel = void (*)(const CUtensorMap, const CUtensorMap, const Params);

template <bool ROWS1>
Kernel pick(int np) {
  return np == 2 ? gemm_fp8_pair_kernel<2, ROWS1> : np == 3 ? gemm_fp8_pair_kernel<3, ROWS1> : gemm_fp8_pair_kernel<4, ROWS1>;
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
  if (cudaOccupancyMaxActiveClusters(&n, (void*)gemm_fp8_pair_kernel<4, false>, &cfg) != cudaSuccess) {
    cudaGetLastError();            // not a fault of the call: such clusters are not used
    n = 0;
  }
  if (cacheable) cache[dev][split].store(n > 0 ? n : -1, std::memory_order_relaxed);
  return n;
}

// The tile width (64 np) and the pairs per tile (a split of K) with the shortest modelled time: waves of tiles, each of
// its blocks (940 cycles a block at 256 outputs, where 910 were measured; about 200 do not depend on the width) and a fixed cost
// (start of the pipeline, store; with a split the join through distributed shared memory).
void choose_tiles(int64_t N, int n_mt, int kbs, int* np, int* split) {
  const double fixed = 5000, join = 5000;
  *split = 0;
  double best = 0;
  for (int s = 1; s <= MAX_SPLIT && s <= std::max(kbs, 1); ++s) {
    const int64_t at_once = resident_clusters(s);
    if (at_once < 1) continue;
    for (int w = 4; w >= 2; --w) {
      const int64_t waves = ceil_div(ceil_div(N, 64 * w) * n_mt, at_once);
      const double t = (double)waves * ((double)ceil_div(kbs, s) * (200 + 185 * w) + fixed + (s > 1 ? join : 0));
      if (*split == 0 || t < best) {
        best = t;
        *split = s;
        *np = w;
      }
    }
  }
}

}  // namespace gtp

int launch_gemm_fp8_pair(const GemmFp8Plan& g, cudaStream_t st) {
  using namespace gtp;
  Params p;
  p.sa = g.a_scale; p.sw = g.w_scale; p.out = g.out; p.ld_out = g.ld_out;
  p.M = (int)g.M; p.N = (int)g.N; p.kbs = (int)(g.K / KB);
  p.n_mt = (int)ceil_div(g.M, 2 * ROWS);
  const bool rows1 = g.w_scale_rows == 1;
  static std::atomic<uint64_t> attr[2][5];
  if (!set_smem_limit_once(pick<false>(4), SMEM_BYTES, attr[0][4])) {     // before the occupancy is asked for
    set_error("gemm_fp8_block128: cudaFuncSetAttribute failed");
    return MTPSD_ECUDA;
  }
  int np = 4;
  choose_tiles(g.N, p.n_mt, p.kbs, &np, &p.split);
  if (p.split < 1) {
    set_error("gemm_fp8_block128: no pair of CTAs fits the device");
    return MTPSD_EUNSUPPORTED;
  }
  const int64_t tiles = ceil_div(g.N, 64 * np) * p.n_mt;
  if (tiles > 0x3fffffffLL / (2 * MAX_SPLIT)) {
    set_error("gemm_fp8_block128: too many output tiles");
    return MTPSD_EUNSUPPORTED;
  }
  p.tiles = (int)tiles;
  p.out_f32 = g.out_f32;
  p.vec_rows = g.ld_out * (g.out_f32 ? 4 : 2) % 32 == 0 && (uintptr_t)g.out % 32 == 0;
  p.vec_scales = p.kbs % 4 == 0 && (uintptr_t)g.a_scale % 16 == 0 && (uintptr_t)g.w_scale % 16 == 0;
  p.status = g.status;
  CUtensorMap mw, ma;
  if (!make_tma_2d(&mw, 0, g.w, (uint64_t)g.K, (uint64_t)g.N, (uint64_t)g.K, KB, (uint32_t)(32 * np), true) ||
      !make_tma_2d(&ma, 0, g.a, (uint64_t)g.K, (uint64_t)g.M, (uint64_t)g.K, KB, ROWS, true)) {
    set_error("gemm_fp8_block128: cuTensorMapEncodeTiled failed");
    return MTPSD_ECUDA;
  }
  Kernel kern = rows1 ? pick<true>(np) : pick<false>(np);
  if (!set_smem_limit_once(kern, SMEM_BYTES, attr[rows1][np])) {
    set_error("gemm_fp8_block128: cudaFuncSetAttribute failed");
    return MTPSD_ECUDA;
  }
  const int64_t clusters = p.split > 1 ? p.tiles : std::min<int64_t>(p.tiles, resident_clusters(1));
  cudaLaunchAttribute attrs[2];
  cudaLaunchConfig_t cfg = config((unsigned)(clusters * 2 * p.split), p.split, st, attrs);
  cudaLaunchKernelEx(&cfg, kern, mw, ma, p);
  return check_launch("gemm_fp8_block128");
}

}  // namespace mtpsd
