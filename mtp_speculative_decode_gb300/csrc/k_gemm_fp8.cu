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
// rate, 144 us; 64 rows at 94 %, 153 us), so bn is chosen such that the tiles load every SM alike; TMEM lanes
// past bn hold products of stale operands and are not stored.
//
// The epilogue reads TMEM (lane = output, column = row of a) in the 16x256b
// shape: a thread gets four lanes of every fourth column pair, so one 8-byte
// shared-memory read of two column scales serves eight values.  (With one lane
// per thread every scale is a broadcast read for one value: the reads took more
// shared-memory cycles than the MMAs' operands, 290 against 186 us without them
// at 192 x 154880 x 6144.)
//
// Roles (608 threads, one CTA per SM):
//   warps 0-15  epilogue: warp w takes the TMEM lanes 32 (w % 4) .. +31 and the columns of quarter w / 4
//               (four warps per scheduler hide the latency of the TMEM reads).  A block's scales and the probe
//               of its barrier are fetched before the block in front is added: read after the wait, they made
//               the chain of a block long enough to show (163 us at 64 x 154880 x 6144).
//   warp 16     TMA producer: a ring of stages of one block (128 x 128 bytes of w, cols x 128 of a).
//   warp 17     TMEM allocation and MMA issue.
//   warp 18     scales: a ring of slots of four blocks' scales of the rows of a and of the weight rows.
// With few tiles the blocks of K of a tile are split over a cluster of up to 8 CTAs (consecutive
// runs of blocks), which add their accumulators through distributed shared memory in rank order.
// The order of every sum is fixed by the sizes and the device.  Every mbarrier wait is bounded
// (2 s): on expiry the kernel flags MTPSD_STATUS_WAIT_TIMEOUT, drains its copies, frees TMEM and returns.
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
constexpr int TR_LD = 36;                 // the same for the transposed store of 8 columns x 32 outputs
constexpr int TR_FLOATS = 8 * TR_LD;     // per epilogue warp

constexpr int COLS = 64;                  // most columns (rows of a) of a tile; 16 per epilogue warp
constexpr int STAGE = W_BYTES + COLS * KB;
constexpr int NSTAGE = 192 * 1024 / STAGE;
constexpr int NBUF = TMEM_COLS / COLS;
constexpr int SLOT_FLOATS = SG * (COLS + TILE_N);
constexpr int OFF_SCALE = NSTAGE * STAGE;
constexpr int OFF_TR = OFF_SCALE + NSLOT * SLOT_FLOATS * 4;
constexpr int OFF_BAR = OFF_TR + EPI_WARPS * TR_FLOATS * 4;
constexpr int N_BARS = 2 * NSTAGE + 2 * NBUF + 2 * NSLOT + 1;
constexpr int OFF_MISC = OFF_BAR + N_BARS * 8;
constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;         // + alignment slack
static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
static_assert(COLS * PAD_N * 4 <= NSTAGE * STAGE, "the partial tile fits the stage ring");
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
  int out_f32;
  int vec_scales;         // a block row's scales can be read four at a time
  int32_t* status;
};

__device__ __forceinline__ void store_out(const Params& p, int64_t off, float v) {
  if (p.out_f32) ((float*)p.out)[off] = v;
  else ((__nv_bfloat16*)p.out)[off] = __float2bfloat16_rn(v);
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
  // acc[4 j + 2 h + i]: columns 8 j + 2 (lane % 4), +1 of the warp's, output 16 h + 8 i + lane / 4 of its 32
  uint64_t acc[8];

  if (warp == PRODUCER_WARP) {
    int n = 0;
    bool ok = true;
    const uint32_t bytes = (uint32_t)((p.bn + p.cols) * KB);
    for (int tile = first; tile < p.tiles && ok; tile += step) {
      const int n0 = tile * p.bn;
      for (int kb = kb0; kb < kb1; ++kb, ++n) {
        const int stage = n % NSTAGE, round = n / NSTAGE;
        if (round > 0) ok = wait_all(&empty[stage], (round - 1) & 1, abort_flag, p.status);
        if (!ok) break;
        if (elect_one()) {
          const uint32_t dst = saddr(sm + stage * STAGE);
          mbar_expect_tx(&full[stage], bytes);
          tma_load_2d(dst, &tmap_w, kb * KB, n0, &full[stage]);
          tma_load_2d(dst + W_BYTES, &tmap_a, kb * KB, 0, &full[stage]);
        }
        __syncwarp();
      }
    }
    if (*abort_flag && lane == 0) {   // drain this CTA's copies still in flight (bounded)
      volatile int dummy = 0;
      for (int s = 0; s < NSTAGE; ++s) {
        const int issued = n / NSTAGE + (s < n % NSTAGE ? 1 : 0);   // loads of stage s
        if (issued > 0) mbar::wait<false>(&full[s], (issued - 1) & 1, &dummy, p.status, mbar::DEFAULT_LIMIT_NS);
      }
    }
  } else if (warp == MMA_WARP) {
    int n = 0;
    bool ok = true;
    const uint32_t id = idesc_n(p.cols);
    for (int tile = first; tile < p.tiles && ok; tile += step) {
      for (int kb = kb0; kb < kb1; ++kb, ++n) {
        const int stage = n % NSTAGE, buf = n % NBUF, round = n / NBUF;
        ok = wait_all(&full[stage], (n / NSTAGE) & 1, abort_flag, p.status);
        if (ok && round > 0) ok = wait_all(&t_empty[buf], (round - 1) & 1, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t w_base = saddr(sm + stage * STAGE), a_base = w_base + W_BYTES;
          const uint32_t d = tmem_base + (uint32_t)(buf * COLS);
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
    const int quarter = warp & 3, c0 = (warp >> 2) * 16;           // this warp's TMEM lanes and first column
    const int fr = lane >> 2, fc = 2 * (lane & 3);                 // fragment row and column of this lane
    const bool mine = c0 < p.cols;                                 // the warp has columns
    int n = 0, slot = 0, s_phase = 0;                              // blocks so far, scale slot
    // A wait that gave up makes the warp walk on without waiting, to the end, and store nothing: the blocks' loop then
    // has no exit to test for.
    bool gave_up = false;
    auto finish = [&](uint64_t* bar, uint32_t parity) {            // of a wait whose first probe failed
      if (!gave_up) gave_up = !mbar::wait<false>(bar, parity, abort_flag, p.status, mbar::DEFAULT_LIMIT_NS);
    };
    for (int tile = first; tile < p.tiles; tile += step) {
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = 0ull;
      // The scales of a block and the probe for its products are fetched while the block before is still being added
      float wr[4];                                                 // of the thread's four outputs
      uint64_t cs[2];                                              // of its columns
      bool ready;
      auto fetch = [&](int j, int block) {
        const float* sc = scales + slot * SLOT_FLOATS + j * COLS + c0 + fc;
        const float* sr = scales + slot * SLOT_FLOATS + SG * COLS + j * TILE_N + quarter * 32 + fr;
#pragma unroll
        for (int i = 0; i < 4; ++i) wr[i] = sr[8 * i];
        cs[0] = *(const uint64_t*)sc;
        cs[1] = *(const uint64_t*)(sc + 8);
        ready = mbar::try_wait<false>(&t_full[block % NBUF], block / NBUF & 1);
      };
      auto next_slot = [&]() {
        if (!mbar::try_wait<false>(&s_full[slot], s_phase)) finish(&s_full[slot], s_phase);
        __syncwarp();
      };
      next_slot();
      fetch(0, n);
      for (int kb = kb0, j = 0; kb < kb1; ++kb, ++n) {
        const int buf = n % NBUF;
        uint64_t rw[4];
        const uint64_t s[2] = {cs[0], cs[1]};
#pragma unroll
        for (int i = 0; i < 4; ++i) rw[i] = pack2(make_float2(wr[i], wr[i]));
        if (!ready) finish(&t_full[buf], n / NBUF & 1);
        __syncwarp();
        tc_fence_after();
        uint32_t t[2][8];
        if (mine) {
          const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(buf * COLS + c0);
          tmem_ld_x2(taddr, t[0]);
          tmem_ld_x2(taddr + (16u << 16), t[1]);
          tmem_ld_wait();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&t_empty[buf]);
        if (++j == SG || kb == kb1 - 1) {                          // every lane has read the slot's scales
          if (lane == 0) mbar_arrive(&s_empty[slot]);
          j = 0;
          if (++slot == NSLOT) {
            slot = 0;
            s_phase ^= 1;
          }
          if (kb < kb1 - 1) next_slot();
        }
        if (kb < kb1 - 1) fetch(j, n + 1);
        if (mine) {
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint64_t& q = acc[4 * g + i];
              const uint32_t* v = t[i >> 1] + 4 * g + 2 * (i & 1);
              q = fma2(pack2(v[0], v[1]), mul2(s[g], rw[i]), q);
            }
        }
      }
      if (__any_sync(0xffffffffu, gave_up)) break;
      if (p.split > 1) break;
      // eight columns at a time through the warp's own shared memory, so that a store covers 32 consecutive outputs
      const int o = quarter * 32 + lane;
      const int64_t n_out = (int64_t)tile * p.bn + o;
      const bool mine_out = o < p.bn && n_out < p.N;
      const int m_cols = min(16, p.M - c0);
      float* tr = (float*)(sm + OFF_TR) + warp * TR_FLOATS;
      int64_t off = (int64_t)c0 * p.ld_out + n_out;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (8 * g >= m_cols) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = unpack2(acc[4 * g + i]);
          tr[fc * TR_LD + 8 * i + fr] = v.x;
          tr[(fc + 1) * TR_LD + 8 * i + fr] = v.y;
        }
        __syncwarp();
        if (mine_out) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (8 * g + e < m_cols) store_out(p, off + e * p.ld_out, tr[e * TR_LD + lane]);
        }
        off += 8 * p.ld_out;
        __syncwarp();
      }
    }
  }

  __syncwarp();
  if (p.split > 1) {
    // The cluster's one tile: every rank's accumulators into its own stage ring (its copies and MMAs are
    // done: the epilogue has seen the last block), then each rank sums a part of the columns over the ranks.
    float* part = (float*)sm;                               // [cols][PAD_N]: 128 outputs
    __syncthreads();
    if (warp < EPI_WARPS) {
      const int c0 = (warp >> 2) * 16 + 2 * (lane & 3), o = (warp & 3) * 32 + (lane >> 2);
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = unpack2(acc[4 * g + i]);
          part[(c0 + 8 * g) * PAD_N + o + 8 * i] = v.x;
          part[(c0 + 8 * g + 1) * PAD_N + o + 8 * i] = v.y;
        }
    }
    cluster_sync();
    if (warp < EPI_WARPS) {
      const int r0 = rank * p.M / p.split, r1 = (rank + 1) * p.M / p.split;
      const int o = 4 * lane;                              // this thread's four outputs of a column
      const int n_first = first * p.bn, n_end = min(p.N, n_first + p.bn);
      for (int c = r0 + warp; c < r1; c += EPI_WARPS) {
        float4 v[MAX_SPLIT];                               // every remote read in flight at once
#pragma unroll
        for (int r = 0; r < MAX_SPLIT; ++r)
          v[r] = r < p.split ? ld_cluster4(saddr(part + c * PAD_N + o), r) : make_float4(0.f, 0.f, 0.f, 0.f);
        float4 sum = v[0];
#pragma unroll
        for (int r = 1; r < MAX_SPLIT; ++r)
          if (r < p.split) {
            sum.x += v[r].x; sum.y += v[r].y; sum.z += v[r].z; sum.w += v[r].w;
          }
        const int64_t off = (int64_t)c * p.ld_out + n_first + o;
        const float e[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n_first + o + i < n_end) store_out(p, off + i, e[i]);
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

// Calls with more rows of a than this take the pairs of CTAs: 64 x 154880 x 6144 takes 153 us here and 190 there, 64 x
// 6144 x 12288 24.5 and 27.0.  With tiles of 128 columns (32 per epilogue warp) this kernel took 196 us for 80 x 154880 x
// 6144 and 209 for 128, the pairs 192 and 198; 128 x 2048 x 6144 11.5 against 13.3.
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
