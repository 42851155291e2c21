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
// This kernel is for up to 64 rows of a (k_gemm_fp8_pair.cu takes more): one
// MMA has M = 128 weight rows (operand A) and N = the rows of a, rounded up to
// 16 (operand B), so the few rows of a cost only as much as there are of them
// and the weight streams through once.  A tile is `bn` <= 128 outputs: the weight
// read bounds these calls (16 x 154880 x 6144 runs at 98 % of the measured copy
// rate, 144 us; 64 rows at 96 %, 150 us), so bn is chosen such that the tiles load every SM alike; TMEM lanes
// past bn hold products of stale operands and are not stored.
//
// The epilogue reads TMEM (lane = output, column = row of a) in the 16x256b
// shape: a thread gets four lanes of every fourth column pair, so one 8-byte
// shared-memory read of two column scales serves eight values.  (With one lane
// per thread every scale is a broadcast read for one value: the reads took more
// shared-memory cycles than the MMAs' operands, 290 against 186 us without them
// at 192 x 154880 x 6144.)
//
// A warp's chain of waits and reads for a block takes about 1000 cycles, more than the block's bytes where a call has
// few tiles.  So the epilogue warps form 2 or 4 sets, of which set i takes the blocks with (block of K) % sets = i and adds
// for itself; at the end of a tile the sets' sums are added in order.  For the same reason one thread each issues the
// copies and the MMAs, instead of a warp that waits and votes.  64 x 6144 x 12288: 25.0 us with one set, 22.6 with two, 19.7
// with single threads; 16 x 6144 x 12288 22.8, 20.0 and 17.1; 64 x 154880 x 6144 158, 152 and 150.
//
// Roles (608 threads, one CTA per SM):
//   warps 0-15  epilogue: warp w takes the TMEM lanes 32 (w % 4) .. +31 and, of set (w / 4) % sets, 32 columns.
//   warp 16     TMA producer: a ring of stages of one block (128 x 128 bytes of w, cols x 128 of a).
//   warp 17     TMEM allocation and MMA issue.
//   warp 18     scales: a ring of slots of four blocks' scales of the rows of a and of the weight rows.
// With few tiles the blocks of K of a tile are split over a cluster of up to 8 CTAs (consecutive
// runs of blocks), which add their sums through distributed shared memory in rank order.
// The order of every sum is fixed by the sizes and the device.  Every mbarrier wait is bounded
// (2 s): on expiry the kernel flags MTPSD_STATUS_WAIT_TIMEOUT, stores nothing of the tiles it could not finish, waits for
// its copies in flight, frees TMEM and returns.
#include <algorithm>

#include "gemm_fp8.cuh"

namespace mtpsd {
namespace gtc {

constexpr int TILE_N = 128;               // most outputs (weight rows) of a tile
constexpr int EPI_WARPS = 16;
constexpr int PRODUCER_WARP = 16, MMA_WARP = 17, SCALE_WARP = 18;
constexpr int THREADS = 32 * 19;
constexpr int MAX_SPLIT = 8;
constexpr int W_BYTES = TILE_N * KB;
constexpr int PAD_N = TILE_N + 4;         // row stride (floats) of a partial tile: a fragment's four columns miss each other's banks

constexpr int COLS = 64;                  // most columns (rows of a) of a tile
constexpr int STAGE = W_BYTES + COLS * KB;
constexpr int NSTAGE = 6;
constexpr int NBUF = TMEM_COLS / COLS;
constexpr int SLOT_FLOATS = SG * (COLS + TILE_N);
constexpr int OFF_SCALE = NSTAGE * STAGE;
constexpr int OFF_PART = OFF_SCALE + NSLOT * SLOT_FLOATS * 4;     // the sets' accumulators: 2 x 64 or 4 x 32 columns
constexpr int OFF_BAR = OFF_PART + 2 * COLS * PAD_N * 4;
constexpr int N_BARS = 2 * NSTAGE + 2 * NBUF + 2 * NSLOT + 1;
constexpr int OFF_MISC = OFF_BAR + N_BARS * 8;
constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;         // + alignment slack
static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
static_assert(OFF_BAR % 16 == 0, "barriers are aligned");

struct Params {
  const float* sa;
  const float* sw;
  void* out;
  int64_t ld_out;
  int M, N, kbs;          // rows of a, outputs, blocks of K
  int cols;               // columns of a tile: M rounded up to 16
  int bn, tiles;          // outputs of a tile, tiles
  int w_rows;             // weight rows that share a scale: 1 or 128
  int split;              // CTAs per cluster
  int sets;               // sets of epilogue warps: 4 (up to 32 columns) or 2
  int out_f32;
  int vec_out;            // four consecutive outputs of a row can be stored at once
  int vec_scales;         // a block row's scales can be read four at a time
  int32_t* status;
};

// Outputs o .. o + 3 of a tile for row m of a.
__device__ __forceinline__ void store4(const Params& p, int m, int tile, int o, float4 v) {
  const int64_t n = (int64_t)tile * p.bn + o, off = (int64_t)m * p.ld_out + n;
  const int left = (int)min((int64_t)(p.bn - o), p.N - n);
  if (left >= 4 && p.vec_out) {
    if (p.out_f32) {
      *(float4*)((float*)p.out + off) = v;
    } else {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
      *(uint2*)((__nv_bfloat16*)p.out + off) = make_uint2(*(const uint32_t*)&lo, *(const uint32_t*)&hi);
    }
    return;
  }
  const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < left) {
      if (p.out_f32) ((float*)p.out)[off + i] = e[i];
      else ((__nv_bfloat16*)p.out)[off + i] = __float2bfloat16_rn(e[i]);
    }
}

__global__ void __launch_bounds__(THREADS, 1) gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmap_w,
                                                              const __grid_constant__ CUtensorMap tmap_a,
                                                              const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + (-saddr(smem_raw) & 1023u);     // no cast: loads stay loads of shared memory
  uint64_t* full = (uint64_t*)(sm + OFF_BAR);
  uint64_t* empty = full + NSTAGE;
  uint64_t* t_full = empty + NSTAGE;
  uint64_t* t_empty = t_full + NBUF;
  uint64_t* s_full = t_empty + NBUF;
  uint64_t* s_empty = s_full + NSLOT;
  uint64_t* drain = s_empty + NSLOT;
  uint32_t* tmem_slot = (uint32_t*)(sm + OFF_MISC);
  volatile int* abort_flag = (volatile int*)(sm + OFF_MISC + 4);
  float* scales = (float*)(sm + OFF_SCALE);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NSTAGE; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < NBUF; ++i) {
      mbar_init(&t_full[i], 1);
      mbar_init(&t_empty[i], EPI_WARPS / p.sets);
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
  if (warp == PRODUCER_WARP && elect_one()) {
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
  float* part = (float*)(sm + OFF_PART);     // [sets][128 / sets columns][PAD_N]: 128 outputs

  if (warp == PRODUCER_WARP) {
    if (elect_one()) {             // one thread waits and copies
      int n = 0, stage = 0;
      bool ok = true;
      const uint32_t bytes = (uint32_t)((p.bn + p.cols) * KB);
      for (int tile = first; tile < p.tiles && ok; tile += step) {
        const int n0 = tile * p.bn;
        for (int kb = kb0; kb < kb1; ++kb, ++n) {
          if (n >= NSTAGE)
            ok = mbar::wait_head<false>(&empty[stage], (n / NSTAGE - 1) & 1, abort_flag, p.status);
          if (!ok) break;
          const uint32_t dst = saddr(sm + stage * STAGE);
          mbar_expect_tx(&full[stage], bytes);
          tma_load_2d(dst, &tmap_w, kb * KB, n0, &full[stage]);
          tma_load_2d(dst + W_BYTES, &tmap_a, kb * KB, 0, &full[stage]);
          if (++stage == NSTAGE) stage = 0;
        }
      }
      // The copies land before the CTA leaves, whoever waits for them: after an expired wait nobody else may.
      for (int s = 0; s < NSTAGE; ++s) {
        const int issued = n / NSTAGE + (s < n % NSTAGE ? 1 : 0);     // loads of stage s
        if (issued > 0) mbar::drain<false>(&full[s], (issued - 1) & 1, p.status);
      }
    }
  } else if (warp == MMA_WARP) {
    if (elect_one()) {             // one thread waits and issues
      int n = 0, stage = 0;
      bool ok = true;
      const uint32_t id = idesc_n(p.cols);
      for (int tile = first; tile < p.tiles && ok; tile += step) {
        for (int kb = kb0; kb < kb1; ++kb, ++n) {
          const int buf = n % NBUF, round = n / NBUF;
          ok = mbar::wait_head<false>(&full[stage], (n / NSTAGE) & 1, abort_flag, p.status);
          if (ok && round > 0)
            ok = mbar::wait_head<false>(&t_empty[buf], (round - 1) & 1, abort_flag, p.status);
          if (!ok) break;
          tc_fence_after();
          const uint64_t w = sw128_desc(saddr(sm + stage * STAGE));    // descriptors count 16 bytes
          const uint32_t d = tmem_base + (uint32_t)(buf * COLS);
#pragma unroll
          for (int kk = 0; kk < KB / 32; ++kk) mma_fp8(d, w + 2 * kk, w + (W_BYTES >> 4) + 2 * kk, id, kk > 0 ? 1u : 0u);
          mma_commit(&t_full[buf]);
          mma_commit(&empty[stage]);
          if (++stage == NSTAGE) stage = 0;
        }
      }
      mma_commit(drain);           // every MMA has completed before TMEM is released
    }
    __syncwarp();
    mbar::drain<false>(drain, 0, p.status);
  } else if (warp == SCALE_WARP) {
    // slot: [SG][COLS] scales of the rows of a, then [SG][128] scales of the tile's weight rows
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
      for (int kb = kb0; kb < kb1; kb += SG, ++n) {
        float v[2][SG], w[4][SG];
        // all of the slot's loads in flight before the wait for its release
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (32 * i < p.cols) load4(p.sa, 32 * i + lane, p.M, kb, v[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t row = (int64_t)tile * p.bn + 32 * i + lane;
          load4(p.sw, p.w_rows == 1 ? row : row >> 7, p.w_rows == 1 ? p.N : ((int64_t)p.N + 127) >> 7, kb, w[i]);
        }
        const int slot = n % NSLOT, round = n / NSLOT;
        if (round > 0) ok = wait_all(&s_empty[slot], (round - 1) & 1, abort_flag, p.status);
        if (!ok) break;
        float* dst = scales + slot * SLOT_FLOATS;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (32 * i < p.cols)
#pragma unroll
            for (int j = 0; j < SG; ++j) dst[j * COLS + 32 * i + lane] = v[i][j];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < SG; ++j) dst[SG * COLS + j * TILE_N + 32 * i + lane] = w[i][j];
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_full[slot]);
      }
    }
  } else {
    const int quarter = warp & 3, set = (warp >> 2) % p.sets;      // this warp's TMEM lanes and set
    const int c0 = 32 * ((warp >> 2) / p.sets), cols_set = 2 * COLS / p.sets;      // first column, columns of a set's tile
    const int fr = lane >> 2, fc = 2 * (lane & 3);                 // fragment row and column of this lane
    const int nb = kb1 - kb0;
    int n = 0, slot = 0, s_phase = 0;                              // blocks of the tiles so far, scale slot
    // A wait that gave up makes the warp walk on without waiting, to the end: every warp comes to every barrier below.
    bool gave_up = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!mbar::try_wait<false>(bar, parity) && !gave_up)
        gave_up = !mbar::wait_head<false>(bar, parity, abort_flag, p.status);
      __syncwarp();
    };
    auto epilogue_barrier = [] { asm volatile("bar.sync 1, %0;" ::"n"(32 * EPI_WARPS) : "memory"); };
    for (int tile = first; tile < p.tiles; tile += step, n += nb) {
      // acc[8 q + 4 j + i]: columns 16 q + 8 j + fc, +1 of the warp's 32, output 8 i + fr of its 32
      uint64_t acc[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i] = 0ull;
      for (int b0 = 0; b0 < nb; b0 += SG) {
        wait(&s_full[slot], s_phase);
        for (int j = set; j < SG && b0 + j < nb; j += p.sets) {    // SG is a multiple of the sets
          const int block = n + b0 + j, buf = block % NBUF;
          const float* sc = scales + slot * SLOT_FLOATS + j * COLS + c0 + fc;
          const float* sr = scales + slot * SLOT_FLOATS + SG * COLS + j * TILE_N + quarter * 32 + fr;
          uint64_t rw[4];                                          // the weight scales of the thread's four outputs, twice each
#pragma unroll
          for (int i = 0; i < 4; ++i) rw[i] = pack2(make_float2(sr[8 * i], sr[8 * i]));
          wait(&t_full[buf], block / NBUF & 1);
          tc_fence_after();
          const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(buf * COLS + c0);
          uint32_t t[2][16];
#pragma unroll
          for (int q = 0; q < 2; ++q)
            if (c0 + 16 * q < p.cols) {
              tmem_ld_x2(taddr + 16 * q, t[q]);
              tmem_ld_x2(taddr + (16u << 16) + 16 * q, t[q] + 8);
            }
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&t_empty[buf]);
#pragma unroll
          for (int q = 0; q < 2; ++q)
            if (c0 + 16 * q < p.cols) {
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                const uint64_t s = *(const uint64_t*)(sc + 16 * q + 8 * g);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const uint32_t* v = t[q] + 8 * (i >> 1) + 4 * g + 2 * (i & 1);
                  acc[8 * q + 4 * g + i] = fma2(pack2(v[0], v[1]), mul2(s, rw[i]), acc[8 * q + 4 * g + i]);
                }
              }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[slot]);                // every lane has read the slot's scales
        if (++slot == NSLOT) {
          slot = 0;
          s_phase ^= 1;
        }
      }
      // ---- the sets' sums, in order, by all epilogue warps: a column at a time, four outputs per thread
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (c0 + 16 * q < p.cols) {
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 v = unpack2(acc[8 * q + 4 * g + i]);
              float* d = part + (set * cols_set + c0 + 16 * q + 8 * g + fc) * PAD_N + quarter * 32 + 8 * i + fr;
              d[0] = v.x;
              d[PAD_N] = v.y;
            }
        }
      epilogue_barrier();
      const bool whole = *abort_flag == 0;     // no warp of this CTA has given up before it wrote its sums
      for (int c = warp; c < p.M; c += EPI_WARPS) {
        float4 sum = *(const float4*)(part + c * PAD_N + 4 * lane);
        for (int k = 1; k < p.sets; ++k) {
          const float4 v = *(const float4*)(part + (k * cols_set + c) * PAD_N + 4 * lane);
          sum.x += v.x; sum.y += v.y; sum.z += v.z; sum.w += v.w;
        }
        if (p.split > 1) *(float4*)(part + c * PAD_N + 4 * lane) = sum;
        else if (whole) store4(p, c, tile, 4 * lane, sum);
      }
      if (p.split > 1) break;
      epilogue_barrier();            // the sums are read before the next tile's are written
    }
  }

  __syncwarp();
  if (p.split > 1) {
    // The cluster's one tile: each rank sums a part of the columns over the ranks, in order.
    cluster_sync();
    if (warp < EPI_WARPS) {
      const int r0 = rank * p.M / p.split, r1 = (rank + 1) * p.M / p.split;
      for (int c = r0 + warp; c < r1; c += EPI_WARPS) {
        float4 v[MAX_SPLIT];                               // every remote read in flight at once
#pragma unroll
        for (int r = 0; r < MAX_SPLIT; ++r)
          v[r] = r < p.split ? ld_cluster4(saddr(part + c * PAD_N + 4 * lane), r) : make_float4(0.f, 0.f, 0.f, 0.f);
        // whether a wait of some rank has expired: its sums are not all there, and nothing is stored (read behind the sums:
        // 1 x 576 x 6144 5.47 us in a graph, in front of them 5.61, without the flags 5.38)
        const uint32_t failed = ld_cluster1(saddr((const void*)abort_flag), (uint32_t)lane % (uint32_t)p.split);
        float4 sum = v[0];
#pragma unroll
        for (int r = 1; r < MAX_SPLIT; ++r)
          if (r < p.split) {
            sum.x += v[r].x; sum.y += v[r].y; sum.z += v[r].z; sum.w += v[r].w;
          }
        if (!__any_sync(0xffffffffu, failed)) store4(p, c, first, 4 * lane, sum);
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

cudaLaunchConfig_t config(unsigned grid, int split, cudaStream_t st, cudaLaunchAttribute* attrs) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
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
  cudaLaunchConfig_t cfg = config((unsigned)split, split, 0, attrs);
  if (cudaOccupancyMaxActiveClusters(&n, (void*)gemm_fp8_kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();            // not a fault of the call: such clusters are not used
    n = 0;
  }
  if (cacheable) cache[dev][split].store(n > 0 ? n : -1, std::memory_order_relaxed);
  return n;
}

// The outputs of a tile and the CTAs per tile (a split of K) with the shortest modelled time, in cycles: waves of
// tiles, each of its blocks (a block's four MMAs take 420; its operands arrive at the SM's share of the memory rate,
// 23 bytes a cycle with every SM loading, 50 at most) and a fixed cost (start of the pipeline, store; with a split the
// join through distributed shared memory).
void choose_tiles(int64_t N, int cols, int kbs, int* bn, int* split) {
  const double fixed = 3000, join = 2500;
  *split = 0;
  double best = 0;
  for (int s = 1; s <= MAX_SPLIT && s <= std::max(kbs, 1); ++s) {
    const int64_t at_once = resident_clusters(s);
    if (at_once < 1) continue;
    const int64_t w0 = ceil_div(ceil_div(N, TILE_N), at_once);             // waves of the widest tiles
    for (int64_t w = w0; w <= w0 + 1; ++w) {
      const int width = (int)std::min<int64_t>(TILE_N, std::max<int64_t>(ceil_div(ceil_div(N, at_once * w), 8) * 8, 32));
      const int64_t tiles = ceil_div(N, width), waves = ceil_div(tiles, at_once);
      const double rate = std::min(50.0, 23.0 * num_sms() / (double)(std::min(tiles, at_once) * s));
      const double block = std::max(420.0, (double)(width + cols) * KB / rate);
      const double t = (double)waves * ((double)ceil_div(kbs, s) * block + fixed + (s > 1 ? join : 0));
      if (*split == 0 || t < best) {
        best = t;
        *split = s;
        *bn = width;
      }
    }
  }
}

}  // namespace gtc

// Calls with more rows of a than this take the pairs of CTAs: 64 x 154880 x 6144 takes 150 us here and 185 there, 64 x
// 6144 x 12288 19.7 and 27. With tiles of 128 columns an earlier form of this kernel took 196 us for 80 x 154880 x 6144
// and 209 for 128 rows, the pairs 185 and 192; 128 x 2048 x 6144 11.5 against 13.3.
constexpr int64_t kPairRows = 64;
static_assert(kPairRows == gtc::COLS, "a tile holds every row of a");

int launch_gemm_fp8(const GemmFp8Plan& g, cudaStream_t st) {
  using namespace gtc;
  if (cc_major() != 10 || !tma_available()) {
    set_error("gemm_fp8_block128: needs a GPU of compute capability 10.x");
    return MTPSD_EUNSUPPORTED;
  }
  if (g.K == 0) {                   // an empty sum
    const size_t es = g.out_f32 ? 4 : 2;
    cudaMemset2DAsync(g.out, (size_t)g.ld_out * es, 0, (size_t)g.N * es, (size_t)g.M, st);
    return check_launch("gemm_fp8_block128");
  }
  if (g.M > kPairRows) return launch_gemm_fp8_pair(g, st);
  Params p;
  p.sa = g.a_scale; p.sw = g.w_scale; p.out = g.out; p.ld_out = g.ld_out;
  p.M = (int)g.M; p.N = (int)g.N; p.kbs = (int)(g.K / KB);
  p.cols = (int)(ceil_div(g.M, 16) * 16);
  p.w_rows = g.w_scale_rows;
  static std::atomic<uint64_t> attr;
  if (!set_smem_limit_once(gemm_fp8_kernel, SMEM_BYTES, attr)) {
    set_error("gemm_fp8_block128: cudaFuncSetAttribute failed");
    return MTPSD_ECUDA;
  }
  choose_tiles(g.N, p.cols, p.kbs, &p.bn, &p.split);
  const int64_t tiles = ceil_div(g.N, p.bn);
  if (tiles > 0x3fffffffLL / MAX_SPLIT) {
    set_error("gemm_fp8_block128: too many output tiles");
    return MTPSD_EUNSUPPORTED;
  }
  p.tiles = (int)tiles;
  p.out_f32 = g.out_f32;
  p.sets = p.cols <= 32 ? 4 : 2;
  p.vec_out = g.ld_out % 4 == 0 && (uintptr_t)g.out % (g.out_f32 ? 16 : 8) == 0;
  p.vec_scales = p.kbs % 4 == 0 && (uintptr_t)g.a_scale % 16 == 0 && (uintptr_t)g.w_scale % 16 == 0;
  p.status = g.status;
  CUtensorMap mw, ma;
  if (!make_tma_2d(&mw, 0, g.w, (uint64_t)g.K, (uint64_t)g.N, (uint64_t)g.K, KB, (uint32_t)p.bn, true) ||
      !make_tma_2d(&ma, 0, g.a, (uint64_t)g.K, (uint64_t)g.M, (uint64_t)g.K, KB, (uint32_t)p.cols, true)) {
    set_error("gemm_fp8_block128: cuTensorMapEncodeTiled failed");
    return MTPSD_ECUDA;
  }
  const unsigned grid = p.split > 1 ? (unsigned)(p.tiles * p.split) : (unsigned)std::min<int64_t>(p.tiles, num_sms());
  cudaLaunchAttribute attrs[2];
  cudaLaunchConfig_t cfg = config(grid, p.split, st, attrs);
  cudaLaunchKernelEx(&cfg, gemm_fp8_kernel, mw, ma, p);
  return check_launch("gemm_fp8_block128");
}

}  // namespace mtpsd
