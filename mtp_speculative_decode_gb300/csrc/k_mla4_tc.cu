// Sparse MLA decode over 4-bit latent rows on the 5th-generation tensor cores (tcgen05 kind::f16, bf16 operands, fp32
// accumulators in TMEM).
//
// [P2] "验证段的逐层算子" op 7 / [P3] "稀疏 MLA 的前向路径": per query row r and head h, softmax attention over the selected latent
// rows c[s_j, 0:576] with values c[s_j, 0:512].  The rows are the 416 bytes of latent4.cuh.
//
// A cluster of two CTAs owns (row, 128-head group, split of the selected list); the heads are the MMA's M (heads past H are
// zeros and not stored).  O, 128 heads x 512 dims in fp32, would fill TMEM, so the CTAs share it: rank 0 has value dims 0..255
// and forms the partial scores of dims 0..255 and the 64 rope dims, rank 1 those of dims 256..511.  Per pair of 64
// positions each CTA sends its partial scores (log2 units, fp16) to the other and adds what it receives to its own fp32 ones.
// Every selected row is read, and each half of it dequantized, once per cluster.
//
// A pair's chain (QK^T, read the scores, exchange, maximum, exponentials, P to TMEM, PV, and only then the next QK^T into that
// score buffer) takes several times as long as its MMAs.  Two warpgroups therefore take the pairs in turn, each with a score
// buffer, a receive slot and a staging slot of its own, so that two chains run side by side; the thread that sends a head's scores keeps
// them in registers for the addition, so TMEM is read once.  The only step in order is the running maximum of a head, which passes
// between the two threads of that head through shared memory.  The reference maximum is lazy: O is rescaled only when a head's
// maximum grows by more than 2^8.
// Measured (70 rows, one wave): 1.9 us a pair; 1.5 without the dequantization's arithmetic, 1.07 without the gathers too, 0.77
// without exchange and exponentials; the MMAs need 0.65.  192 rows x 128 heads x 2048 positions: 218 us (FP8 rows: 357).
//
//   TMEM  [0,128) this CTA's 256 query dims (A operand, bf16 pairs); [128,192) [192,256) scores of even and odd pairs (fp32), P
//         over their first 32 columns (bf16 pairs); [256,512) O
//   SMEM  rope query dims (rank 0, 128-byte swizzle); a ring of three pair buffers of 64 positions in chunks of 64 dims (64 rows x 128
//         B, 128-byte swizzle): the K-major B operand of the scores and, for chunks 0..3, the MN-major B operand of PV; two
//         receive slots and two staging slots of 16 KB (two halves of 8 KB: row = head, 32 positions of fp16 in 64 bytes,
//         16-byte piece c at c ^ ((head >> 1) & 3)); a ring of FD gathered tiles
//
// Two warps gather the codes and scales with TMA tile::gather4, FD tiles of 32 positions ahead, and the rope values, which are bf16
// already, straight into their chunk; four warps write the codes as bf16 into the pair buffer.  One warp for both was slower
// (278 us for the 192 rows): its issue, waits and arithmetic add up to more than the rest of a pair's chain.
// A row is dequantized as code * scale * 2^-14: the code's bits are shifted to where a bf16 has them (a factor 2^-126), and
// the scale, times 2^112, is a bf16 too, so one exact multiplication per two values remains.  The factor is taken back in the
// softmax scale and in the output; the rope queries are multiplied by 2^-14 as well, so that both parts of a score have it.
//
// Rounding: scores' halves to fp16 (2^-11 of a half), P to bf16 (2^-8), the output to bf16; sums, maxima and O are fp32.
// Every wait is bounded (2 s) and flags MTPSD_STATUS_WAIT_TIMEOUT on expiry; the CTAs then wait for their copies in flight (settle).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdlib.h>

#include "cache.h"
#include "common.cuh"
#include "head_wait.cuh"
#include "latent4.cuh"

namespace mtpsd {
namespace m4 {

constexpr int DL = 576, DV = 512, DVH = 256;
constexpr int HG = 128;                  // heads per CTA (MMA M)
constexpr int NP = 64;                   // positions per MMA step: a pair (of gathered tiles)
constexpr int NPAIR = 3;                 // pair buffers in the ring
constexpr int CHUNK = NP * 128;          // 64 dims of a pair buffer
constexpr int PAIR_STRIDE = 5 * CHUNK;
constexpr int XHALF = HG * 64, XSLOT = 2 * XHALF;
constexpr int OFF_QR = 0;
constexpr int OFF_C = OFF_QR + HG * 128;
constexpr int OFF_X = OFF_C + NPAIR * PAIR_STRIDE;
constexpr int OFF_STG = OFF_X + 2 * XSLOT;
constexpr int NT = 32, FD = 4;           // positions per gathered tile, gathered tiles in flight
constexpr int F_SCL = NT * 128;          // staging tile: codes [32 rows][128 B], then scales [8 groups of 4 rows][16 B, at 128 B]
constexpr int F_TILE = F_SCL + 8 * 128;
constexpr int OFF_F = OFF_STG + 2 * XSLOT;
constexpr int OFF_MASK = OFF_F + FD * F_TILE;         // [NPAIR] 64 validity bits
constexpr int OFF_MREF = OFF_MASK + 32;               // [128] reference maxima
constexpr int OFF_ML = OFF_MREF + HG * 4;             // [2][128] (reference, sum) of the warpgroups
constexpr int OFF_BAR = OFF_ML + 2 * HG * 8;
constexpr int B_CFULL = 0, B_CEMPTY = B_CFULL + NPAIR, B_SFULL = B_CEMPTY + NPAIR, B_PFULL = B_SFULL + 2, B_PVDONE = B_PFULL + 2,
              B_XFULL = B_PVDONE + 2, B_XFREE = B_XFULL + 4, B_DEC = B_XFREE + 2, B_FFULL = B_DEC + 8, B_FEMPTY = B_FFULL + FD / 2, B_QREADY = B_FEMPTY + FD / 2, B_DRAIN = B_QREADY + 1,
              N_BARS = B_DRAIN + 1;
constexpr int OFF_MISC = OFF_BAR + N_BARS * 8;
// How far each role has come, for a CTA that gives up (settle): tiles whose codes, and whose rope values, a gather warp has fetched;
// pairs that a dequantizing warp has written; pairs that a softmax warp has sent; pairs that a warpgroup has expected.
constexpr int OFF_PROG = OFF_MISC + 16;
constexpr int PG_CODES = 0, PG_ROPE = 2, PG_DEQ = 4, PG_SENT = 8, PG_EXPECTED = 16, N_PROG = 18;
constexpr int SMEM_BYTES = OFF_PROG + 4 * N_PROG + 1024;      // and room to align
static_assert(SMEM_BYTES <= 232448 && OFF_C % 1024 == 0 && OFF_BAR % 8 == 0, "shared memory");
static_assert(4 * 8 * 4096 <= OFF_STG - OFF_C, "the float32 output boxes lie in the drained ring and receive slots");
constexpr int DEQ_WARP = 8, N_DEQ = 4, GATHER_WARP = DEQ_WARP + N_DEQ, N_GATHER = 2, MMA_WARP = GATHER_WARP + N_GATHER;
constexpr int FREE_WARP = MMA_WARP + 1;
constexpr int THREADS = 32 * (FREE_WARP + 1);
constexpr int TM_Q = 0, TM_S0 = 128, TM_O = 256;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float RESCALE_LOG2 = 8.0f;
constexpr float UP = 16384.0f;           // 2^14: what the dequantized values lack
constexpr int MAX_SPLITS = 4;            // splits of a row in one cluster, merged in the kernel

struct Params {
  int B, R, H, n_idx, n_append;
  float sl2;                  // softmax scale * log2(e) * 2^14
  int64_t row_pos_add;
  const __nv_bfloat16* q;
  const uint8_t* latent;
  int64_t pool;
  const int64_t* cache_start;
  const int32_t* bt;          // block table of a paged cache, or null
  int32_t bt_stride, pg_shift;
  const uint32_t* row_offsets;
  const int64_t* row_pos;
  const int32_t* idx;
  const int64_t* append_base;
  __nv_bfloat16* out;
  float* lse;
  float* part_o;              // split partials (O without its normalisation), or null
  float* part_ml;             // [R * H, splits, 2 value halves] (max, sum)
  int n_splits, per_split;    // positions per split: a multiple of NP
  int fused;                  // the splits of a row are one cluster
  int32_t* status;
};

__device__ __forceinline__ uint32_t saddr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint64_t* b, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(b)), "r"(n));
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(b)) : "memory");
}
__device__ __forceinline__ void bar_arrive_tx(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_all(uint64_t* b, uint32_t parity, volatile int* abort_flag, int32_t* status) {
  return __all_sync(0xffffffffu, mbar::wait_head<CLUSTER>(b, parity, abort_flag, status));
}
__device__ __forceinline__ bool elect_one() {
  uint32_t pred = 0;
  asm volatile("{\n .reg .b32 rx;\n .reg .pred px;\n elect.sync rx|px, 0xffffffff;\n selp.b32 %0, 1, 0, px;\n}\n" : "=r"(pred));
  return pred != 0;
}
__device__ __forceinline__ void bar_expect_tx(uint64_t* b, uint32_t bytes) {   // no arrival
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(saddr(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_complete_tx(uint64_t* b, uint32_t bytes) {   // as if so many had come
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(saddr(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void gather4(uint32_t dst, const CUtensorMap* map, int x, const int* y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
      "%6}], [%7];" ::"r"(dst), "l"((uint64_t)map), "r"(x), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(saddr(bar))
      : "memory");
}
__device__ __forceinline__ void store_2d(const CUtensorMap* map, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"((uint64_t)map), "r"(x), "r"(y),
               "r"(src) : "memory");
}
__device__ __forceinline__ void store_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"((uint64_t)map), "r"(x),
               "r"(y), "r"(z), "r"(src) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void commit(uint64_t* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(saddr(b)) : "memory");
}
// 128-byte-swizzle matrix descriptor
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 | (uint64_t)((sbo >> 4) & 0x3FFFu) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// kind::f16, D = F32, A = B = BF16, A K-major; QK: N = 64, PV: B MN-major, N = 256
constexpr uint32_t IDESC_QK = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(NP >> 3) << 17) | ((uint32_t)(HG >> 4) << 24);
constexpr uint32_t IDESC_PV =
    (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(DVH >> 3) << 17) | ((uint32_t)(HG >> 4) << 24);
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
               "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
               "r"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void tm_ld32(uint32_t t, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
               "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                 "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
                 "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
                 "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
               : "r"(t));
}
__device__ __forceinline__ void tm_st32(uint32_t t, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
               "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(t),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
               "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
               "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
               "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
               : "memory");
}
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {   // -inf -> +0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *(const uint32_t*)&v;
}
__device__ __forceinline__ uint32_t pack_f16_sat(float lo, float hi) {   // out of range: +-65504
  uint32_t d;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t map_rank(uint32_t cta_addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(cta_addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Position of an entry, or -1 (padding, past the split, or out of range: flagged).
__device__ __forceinline__ int64_t entry_pos(const Params& p, int64_t s, int64_t limit) {
  if (s == -1) return -1;
  if (s < 0 || s > limit) {
    flag_status(p.status, MTPSD_STATUS_INDEX_RANGE);
    return -1;
  }
  return s;
}
__device__ __forceinline__ int32_t page_entry(const Params& p, int b, int64_t s) {
  if (s < 0 || (s >> p.pg_shift) >= p.bt_stride) return -1;
  return __ldg(p.bt + (int64_t)b * p.bt_stride + (s >> p.pg_shift));
}
template <bool PAGED>
__device__ __forceinline__ int64_t entry_row(const Params& p, int64_t s, int64_t base, int32_t page) {
  if (s < 0) return -1;
  const int64_t row = PAGED ? (page < 0 ? -1 : (((int64_t)page << p.pg_shift) | (s & ((1LL << p.pg_shift) - 1)))) : base + s;
  if (row < 0 || row >= p.pool) {
    flag_status(p.status, MTPSD_STATUS_ROW_RANGE);
    return -1;
  }
  return row;
}

// Merge of a row's S split partials for heads [lo, hi) of the group and this CTA's value half; a warp per head, 8 dims per lane.
template <int S>
__device__ __noinline__ void merge_splits(const Params& p, int r, int h0, int lo, int hi, uint32_t rank) {
  const int warp = threadIdx.x >> 5, d8 = threadIdx.x & 31;
  for (int h = lo + warp; h < hi; h += THREADS / 32) {
    if (h0 + h >= p.H) break;
    const int64_t rh = (int64_t)r * p.H + h0 + h;
    float2 ml[S];
    float4 o[S][2];
#pragma unroll
    for (int t = 0; t < S; ++t) {
      ml[t] = *(const float2*)(p.part_ml + ((rh * S + t) * 2 + rank) * 2);
      const float4* src = (const float4*)(p.part_o + (rh * S + t) * DV + rank * DVH) + 2 * d8;
      o[t][0] = src[0];
      o[t][1] = src[1];
    }
    float m = -INFINITY, l = 0.f;
#pragma unroll
    for (int t = 0; t < S; ++t) m = fmaxf(m, ml[t].x);
    float acc[8] = {};
#pragma unroll
    for (int t = 0; t < S; ++t) {
      const float w = ml[t].x == -INFINITY ? 0.f : ex2(ml[t].x - m);
      l += w * ml[t].y;
      acc[0] += w * o[t][0].x; acc[1] += w * o[t][0].y; acc[2] += w * o[t][0].z; acc[3] += w * o[t][0].w;
      acc[4] += w * o[t][1].x; acc[5] += w * o[t][1].y; acc[6] += w * o[t][1].z; acc[7] += w * o[t][1].w;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    *((uint4*)(p.out + rh * DV + rank * DVH) + d8) =
        make_uint4(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv),
                   pack_bf16(acc[4] * inv, acc[5] * inv), pack_bf16(acc[6] * inv, acc[7] * inv));
    if (rank == 0 && d8 == 0 && p.lse) p.lse[rh] = l > 0.f ? (m + log2f(l)) / LOG2E : -INFINITY;
  }
}

// What a CTA that gives up does about its copies in flight: every barrier that has bytes to come gets the arrivals that the roles left
// out, so that its phase ends with the last of the bytes, and is then waited for (bounded).  peer_prog: the other CTA's OFF_PROG.
__device__ __noinline__ void settle(uint8_t* sm, uint64_t* bars, uint32_t peer_prog, bool rope, int32_t* status) {
  const int* prog = (const int*)(sm + OFF_PROG);
  auto of_pair = [&](int tiles, int P) { return min(max(tiles - 2 * P, 0), 2); };   // tiles of pair P among the first `tiles`
  // codes and scales; the slots hold the last FD / 2 pairs that were begun
  const int codes = (max(prog[PG_CODES], prog[PG_CODES + 1]) + 1) / 2;
  for (int P = max(codes - FD / 2, 0); P < codes; ++P) {
    uint64_t* b = bars + B_FFULL + P % (FD / 2);
    for (int g = 0; g < N_GATHER; ++g)
      if (of_pair(prog[PG_CODES + g], P) < 2) bar_arrive(b);
    mbar::drain<false>(b, (P / (FD / 2)) & 1, status);
  }
  const int ropes = rope ? (max(prog[PG_ROPE], prog[PG_ROPE + 1]) + 1) / 2 : 0;
  for (int P = max(ropes - NPAIR, 0); P < ropes; ++P) {
    uint64_t* b = bars + B_CFULL + P % NPAIR;
    for (int g = 0; g < N_GATHER; ++g)
      if (of_pair(prog[PG_ROPE + g], P) < 2) bar_arrive(b);
    for (int d = 0; d < N_DEQ; ++d)
      if (prog[PG_DEQ + d] <= P) bar_arrive(b);
    mbar::drain<false>(b, (P / NPAIR) & 1, status);
  }
  // scores from the other CTA: of the last pair that any of its warps has sent, 2 KB per warp and half
  for (int w = 0; w < 2; ++w) {
    int sent[4], last = 0;
    uint32_t bytes = 0;
    for (int q = 0; q < 4; ++q) {
      asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(sent[q]) : "r"(peer_prog + 4 * (PG_SENT + 4 * w + q)) : "memory");
      last = max(last, sent[q]);
    }
    if (last == 0) continue;
    for (int q = 0; q < 4; ++q) bytes += sent[q] == last ? XHALF / 4 : 0;
    for (int half = 0; half < 2; ++half) {
      uint64_t* b = bars + B_XFULL + 2 * w + half;
      if (prog[PG_EXPECTED + w] < last) bar_arrive_tx(b, bytes);
      else if (bytes < XHALF) bar_complete_tx(b, XHALF - bytes);
      mbar::drain<true>(b, (last - 1) & 1, status);
    }
  }
}

// tm_codes, tm_scale: the rows as bytes, boxes of 128 and 16; tm_rope: their rope values, bf16, 128-byte swizzle; tm_st: the output
// (bf16) or the split partials (float32).
template <bool PAGED>
__global__ void __launch_bounds__(THREADS, 1)
    sparse_mla4_tc_kernel(const __grid_constant__ CUtensorMap tm_codes, const __grid_constant__ CUtensorMap tm_scale,
                          const __grid_constant__ CUtensorMap tm_rope, const __grid_constant__ CUtensorMap tm_st, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t* bars = (uint64_t*)(sm + OFF_BAR);
  uint64_t *c_full = bars + B_CFULL, *c_empty = bars + B_CEMPTY, *s_full = bars + B_SFULL, *p_full = bars + B_PFULL,
           *pv_done = bars + B_PVDONE, *x_full = bars + B_XFULL, *x_free = bars + B_XFREE, *dec = bars + B_DEC,
           *f_full = bars + B_FFULL, *f_empty = bars + B_FEMPTY, *q_ready = bars + B_QREADY, *drain = bars + B_DRAIN;
  uint32_t* tmem_slot = (uint32_t*)(sm + OFF_MISC);
  volatile int* abort_flag = (volatile int*)(sm + OFF_MISC + 4);
  volatile int* given_up = (volatile int*)(sm + OFF_MISC + 8);   // some CTA of the cluster has aborted
  uint8_t* mask_s = sm + OFF_MASK;
  volatile int* prog = (volatile int*)(sm + OFF_PROG);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t crank;                          // value half + 2 * split of the cluster
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(crank));
  const uint32_t rank = crank & 1u, peer = crank ^ 1u;
  const int r = blockIdx.x, h0 = (int)(blockIdx.y >> 1) * HG, split = blockIdx.z;
  const int64_t total = (int64_t)p.n_idx + p.n_append;
  const int64_t j0 = (int64_t)split * p.per_split, j1 = min(total, j0 + (int64_t)p.per_split);
  const int n_pairs = j1 > j0 ? (int)((j1 - j0 + NP - 1) / NP) : 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NPAIR; ++i) {
      bar_init(&c_full[i], N_DEQ + N_GATHER);
      bar_init(&c_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&s_full[i], 2);             // the MMAs' commit, and the MMA warp (it hands on the validity bits)
      bar_init(&p_full[i], 4);             // one arrival per warp
      bar_init(&pv_done[i], 1);
      bar_init(&x_full[2 * i], 1);
      bar_init(&x_full[2 * i + 1], 1);
      bar_init(&x_free[i], 1);             // the other CTA's FREE_WARP
    }
    for (int i = 0; i < 8; ++i) bar_init(&dec[i], 1);
    for (int i = 0; i < FD / 2; ++i) {     // per pair of tiles
      bar_init(&f_full[i], N_GATHER);
      bar_init(&f_empty[i], N_DEQ);
    }
    bar_init(q_ready, 8);                  // one arrival per warp
    bar_init(drain, 1);
    *abort_flag = 0;
    *given_up = 0;
    for (int i = 0; i < N_PROG; ++i) prog[i] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_slot)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (warp == GATHER_WARP && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&tm_codes) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&tm_scale) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&tm_rope) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&tm_st) : "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  cluster_sync();                          // the barriers of both CTAs exist before any remote arrival
  griddep_wait();                          // everything above overlaps the previous kernel's tail
  griddep_launch_dependents();
  const uint32_t tmem = *tmem_slot;

  if (warp < 8) {
    // ------------------------------------------------ scores, softmax, output: thread = head, warpgroup w = pairs of parity w
    const int w = warp >> 2, quad = warp & 3, h = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const bool head_ok = h0 + h < p.H;
    {   // queries: this warpgroup's 128 of the CTA's 256 dims to TMEM as they are, rank 0's rope dims to shared memory times 2^-14
      const uint4* src = (const uint4*)(p.q + ((int64_t)r * p.H + h0 + h) * DL);
      const uint4 zero = make_uint4(0, 0, 0, 0);
      uint4 x[16], rp[4];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = head_ok ? src[rank * 32 + w * 16 + i] : zero;
      if (rank == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) rp[i] = head_ok ? src[64 + w * 4 + i] : zero;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t v[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[4 * i] = x[8 * c + i].x; v[4 * i + 1] = x[8 * c + i].y; v[4 * i + 2] = x[8 * c + i].z; v[4 * i + 3] = x[8 * c + i].w;
        }
        tm_st32(tmem + lane_off + TM_Q + w * 64 + c * 32, v);
      }
      if (rank == 0) {
        constexpr uint32_t DOWN = 0x38803880u;   // 2^-14, twice
#pragma unroll
        for (int i = 0; i < 4; ++i)
          sts128(saddr(sm + OFF_QR) + h * 128 + (((w * 4 + i) ^ (h & 7)) << 4), mul_bf16x2(rp[i].x, DOWN), mul_bf16x2(rp[i].y, DOWN),
                 mul_bf16x2(rp[i].z, DOWN), mul_bf16x2(rp[i].w, DOWN));
        fence_async();
      }
      tm_wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(q_ready);
    }
    const uint32_t swz = (uint32_t)((h >> 1) & 3);
    const uint32_t x_own = saddr(sm + OFF_X) + w * XSLOT + h * 64;
    const uint32_t stg_own = saddr(sm + OFF_STG) + w * XSLOT + h * 64;
    const uint32_t stg_warp = saddr(sm + OFF_STG) + w * XSLOT + quad * 2048;
    const uint32_t x_peer = map_rank(saddr(sm + OFF_X), peer) + w * XSLOT + quad * 2048;
    const uint32_t xfull_peer = map_rank(saddr(x_full), peer) + w * 16;
    float* mref = (float*)(sm + OFF_MREF);
    const uint32_t tm_s = tmem + lane_off + TM_S0 + w * 64;
    float m_cur = -INFINITY, l = 0.f;      // this warpgroup's sum, relative to m_cur
    bool ok = true;
    int sent = (n_pairs + 1 - w) / 2, expected = sent;      // pairs of this warpgroup; set where it gives up, the loop carries neither
    for (int P = w; P < n_pairs; P += 2) {
      const uint32_t par = (P >> 1) & 1;
      if (h == 0) {
        bar_arrive_tx(&x_full[2 * w], XHALF);
        bar_arrive_tx(&x_full[2 * w + 1], XHALF);
      }
      // the other CTA has taken pair P - 2 out of its slot: slot and staging may be written again
      if (P >= 2) ok = wait_all<true>(&x_free[w], ((P - 2) >> 1) & 1, abort_flag, p.status);
      ok = ok && wait_all(&s_full[w], par, abort_flag, p.status);
      if (!ok) {
        sent = P / 2;
        expected = P / 2 + 1;
        break;
      }
      fence_after();
      uint32_t sr[64];
      tm_ld32(tm_s, sr);
      tm_ld32(tm_s + 32, sr + 32);
      tm_wait_ld();
      // send: lane 0 moves the warp's 32 heads of each half with one bulk copy
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t hx[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
          hx[j] = pack_f16_sat(__uint_as_float(sr[32 * half + 2 * j]) * p.sl2, __uint_as_float(sr[32 * half + 2 * j + 1]) * p.sl2);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          sts128(stg_own + half * XHALF + ((c ^ swz) << 4), hx[4 * c], hx[4 * c + 1], hx[4 * c + 2], hx[4 * c + 3]);
        fence_async();
        __syncwarp();
        if (lane == 0)
          asm volatile(
              "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                  x_peer + half * XHALF), "r"(stg_warp + half * XHALF), "r"(2048), "r"(xfull_peer + half * 8)
              : "memory");
      }
      const uint2 mk2 = *(const uint2*)(mask_s + 8 * (P % NPAIR));
      const uint32_t mk[2] = {mk2.x, mk2.y};
      // the head's reference as pair P - 1 left it (while the other CTA's scores are on their way)
      float m_old = -INFINITY;
      if (P > 0) {
        ok = wait_all(&dec[4 * (w ^ 1) + quad], ((P - 1) >> 1) & 1, abort_flag, p.status);
        if (!ok) {
          sent = expected = P / 2 + 1;
          break;
        }
        m_old = mref[h];
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        ok = ok && wait_all<true>(&x_full[2 * w + half], par, abort_flag, p.status);
        if (!ok) break;
        uint32_t px[16];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(px[4 * c]), "=r"(px[4 * c + 1]), "=r"(px[4 * c + 2]), "=r"(px[4 * c + 3])
                       : "r"(x_own + half * XHALF + ((c ^ swz) << 4)) : "memory");
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float2 o = __half22float2(*(const __half2*)&px[j]);
          float v0 = fmaf(__uint_as_float(sr[32 * half + 2 * j]), p.sl2, o.x);
          float v1 = fmaf(__uint_as_float(sr[32 * half + 2 * j + 1]), p.sl2, o.y);
          if (mk[half] != 0xffffffffu) {   // the same for the whole CTA
            v0 = (mk[half] >> (2 * j)) & 1u ? v0 : -INFINITY;
            v1 = (mk[half] >> (2 * j + 1)) & 1u ? v1 : -INFINITY;
          }
          mx[j & 3] = fmaxf(mx[j & 3], fmaxf(v0, v1));
          sr[32 * half + 2 * j] = __float_as_uint(v0);
          sr[32 * half + 2 * j + 1] = __float_as_uint(v1);
        }
      }
      if (!ok) {
        sent = expected = P / 2 + 1;
        break;
      }
      const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      const bool grow = mt > m_old + RESCALE_LOG2 || (m_old == -INFINITY && mt > -INFINITY);
      const float m_new = grow ? mt : m_old;
      mref[h] = m_new;
      __syncwarp();
      if (lane == 0) bar_arrive(&dec[4 * w + quad]);
      const bool scale_o = grow && m_old > -INFINITY;    // O holds earlier pairs of this head
      if (__any_sync(0xffffffffu, scale_o)) {
        // after PV(P - 1), and before PV(P): P is published below
        ok = wait_all(&pv_done[(P - 1) & 1], ((P - 1) >> 1) & 1, abort_flag, p.status);
        if (!ok) {
          sent = expected = P / 2 + 1;
          break;
        }
        fence_after();
        const float alpha = scale_o ? ex2(m_old - m_new) : 1.f;
#pragma unroll 1
        for (int c = 0; c < DVH / 32; ++c) {
          uint32_t o[32];
          tm_ld32(tmem + lane_off + TM_O + c * 32, o);
          tm_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          tm_st32(tmem + lane_off + TM_O + c * 32, o);
        }
        tm_wait_st();
      }
      if (m_new != m_cur) {
        l *= ex2(m_cur - m_new);
        m_cur = m_new;
      }
      const float mo = m_new == -INFINITY ? 0.f : m_new;
      float ps[4] = {0.f, 0.f, 0.f, 0.f};
      uint32_t pk[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float e0 = ex2(__uint_as_float(sr[2 * j]) - mo), e1 = ex2(__uint_as_float(sr[2 * j + 1]) - mo);
        pk[j] = pack_bf16(e0, e1);
        ps[j & 3] += e0 + e1;
      }
      l += (ps[0] + ps[1]) + (ps[2] + ps[3]);
      tm_st32(tm_s, pk);                   // over the scores, which this thread has read
      tm_wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(&p_full[w]);
    }
    if (lane == 0) {
      prog[PG_SENT + warp] = sent;
      if (quad == 0) prog[PG_EXPECTED + w] = expected;
    }
    // ------------------------------------------------ output
    float2* ml = (float2*)(sm + OFF_ML);
    ml[w * HG + h] = make_float2(m_cur, l);
    if (ok && n_pairs > 0) ok = wait_all(&pv_done[(n_pairs - 1) & 1], ((n_pairs - 1) >> 1) & 1, abort_flag, p.status);
    asm volatile("bar.sync 1, 256;" ::: "memory");
    ok = ok && !*abort_flag;
    fence_after();
    const float m_fin = n_pairs > 0 ? mref[h] : -INFINITY;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 part = ml[i * HG + h];
      if (part.x != -INFINITY) l += part.y * ex2(part.x - m_fin);
    }
    const bool have_o = n_pairs > 0 && ok;
    const bool whole = h0 + quad * 32 + 32 <= p.H;       // the warp's 32 heads are all there: TMA boxes
    const uint32_t sw = (uint32_t)(lane & 7), row_off = (uint32_t)lane * 128u;
    const int64_t rh = (int64_t)r * p.H + h0 + h;
    if (p.n_splits == 1) {
      const float inv = l > 0.f ? UP / l : 0.f;
      const uint32_t stg = saddr(sm + OFF_C) + quad * 16384u;      // 4 boxes of 64 bf16 columns, two per warpgroup
#pragma unroll 1
      for (int c = 4 * w; c < 4 * w + 4; ++c) {
        uint32_t o[32], b[16];
        if (have_o) {
          tm_ld32(tmem + lane_off + TM_O + c * 32, o);
          tm_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0u;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) b[i] = pack_bf16(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
        if (whole) {
          const uint32_t box = stg + (uint32_t)(c >> 1) * 4096u + row_off;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            sts128(box + ((((uint32_t)(c & 1) * 4u + q) ^ sw) << 4), b[4 * q], b[4 * q + 1], b[4 * q + 2], b[4 * q + 3]);
        } else if (head_ok && ok) {
          uint4* dst = (uint4*)(p.out + rh * DV + rank * DVH + c * 32);
#pragma unroll
          for (int q = 0; q < 4; ++q) dst[q] = make_uint4(b[4 * q], b[4 * q + 1], b[4 * q + 2], b[4 * q + 3]);
        }
      }
      if (whole) {
        fence_async();
        __syncwarp();
        if (ok && lane == 0) {
#pragma unroll
          for (int bx = 2 * w; bx < 2 * w + 2; ++bx)
            store_2d(&tm_st, stg + (uint32_t)bx * 4096u, (int)rank * DVH + bx * 64, r * p.H + h0 + quad * 32);
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // the staging is read before exit
        }
        __syncwarp();
      }
      if (ok && head_ok && rank == 0 && w == 0 && p.lse) p.lse[rh] = l > 0.f ? (m_fin + log2f(l)) / LOG2E : -INFINITY;
    } else {
      const uint32_t stg = saddr(sm + OFF_C) + quad * 32768u;      // 8 boxes of 32 float columns, four per warpgroup
#pragma unroll 1
      for (int c = 4 * w; c < 4 * w + 4; ++c) {
        uint32_t o[32];
        if (have_o) {
          tm_ld32(tmem + lane_off + TM_O + c * 32, o);
          tm_wait_ld();
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = have_o ? __float_as_uint(__uint_as_float(o[i]) * UP) : 0u;
        if (whole) {
          const uint32_t box = stg + (uint32_t)c * 4096u + row_off;
#pragma unroll
          for (int q = 0; q < 8; ++q) sts128(box + (((uint32_t)q ^ sw) << 4), o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        } else if (head_ok && ok) {
          uint4* dst = (uint4*)(p.part_o + (rh * p.n_splits + split) * DV + rank * DVH + c * 32);
#pragma unroll
          for (int q = 0; q < 8; ++q) dst[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        }
      }
      if (whole) {
        fence_async();
        __syncwarp();
        if (ok && lane == 0) {
#pragma unroll
          for (int c = 4 * w; c < 4 * w + 4; ++c)
            store_3d(&tm_st, stg + (uint32_t)c * 4096u, (int)rank * DVH + c * 32, split, r * p.H + h0 + quad * 32);
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          // complete in global memory, and ordered before this thread's later accesses (the cluster barrier that releases them)
          asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
          asm volatile("fence.proxy.async.global;" ::: "memory");
        }
        __syncwarp();
      }
      if (ok && head_ok && w == 0)   // each value half carries its own (max, sum)
        *(float2*)(p.part_ml + ((rh * p.n_splits + split) * 2 + rank) * 2) = make_float2(l > 0.f ? m_fin : -INFINITY, l);
    }
  } else if (warp < DEQ_WARP + N_DEQ) {
    // ------------------------------------------------ dequantization: rows 8 dw .. 8 dw + 7 of each tile
    // Eight lanes a row, each with 16 bytes of codes (32 values) and their two scales.
    const int dw = warp - DEQ_WARP, j = lane & 7, sub = lane >> 3;
    // Word m of a lane's four goes out in turn (m + j / 2) mod 4, so that the eight lanes of a row write to all banks.
    const int rot = j >> 1;
    const bool r1 = rot & 1, r2 = rot & 2;
    uint32_t dst[4];                       // byte offsets for row 8 dw + sub; 4 rows further: 512 on, bit 6 of the piece flipped
#pragma unroll
    for (int m = 0; m < 4; ++m)
      dst[m] = (uint32_t)(j >> 1) * CHUNK + (8 * dw + sub) * 128 + (((4 * (j & 1) + ((m + rot) & 3)) ^ sub) << 4);
    const uint32_t src_code = saddr(sm + OFF_F) + (8 * dw + sub) * 128 + 16 * j;
    const uint32_t src_scale = saddr(sm + OFF_F) + F_SCL + 2 * dw * 128 + sub * 16 + 2 * j;
    int written = n_pairs;
    for (int P = 0; P < n_pairs; ++P) {
      const int q = P % NPAIR, n = P / NPAIR, f0 = (2 * P) % FD;
      uint4 cd[4];
      uint32_t scl[4];
      if (!wait_all(&f_full[P % (FD / 2)], (P / (FD / 2)) & 1, abort_flag, p.status)) {
        written = P;
        break;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {        // tile i / 2, rows + 4 (i % 2)
        const uint32_t at = (uint32_t)(f0 + (i >> 1)) * F_TILE;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(cd[i].x), "=r"(cd[i].y), "=r"(cd[i].z), "=r"(cd[i].w)
                     : "r"(src_code + at + (i & 1) * 512) : "memory");
        uint16_t v;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(src_scale + at + (i & 1) * 128) : "memory");
        scl[i] = v;
      }
      if (n > 0 && !wait_all(&c_empty[q], (n - 1) & 1, abort_flag, p.status)) {
        written = P;
        break;
      }
      const uint32_t pair = saddr(sm + OFF_C + q * PAIR_STRIDE);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 c = cd[i];
        const uint32_t a0 = r1 ? c.y : c.x, a1 = r1 ? c.z : c.y, a2 = r1 ? c.w : c.z, a3 = r1 ? c.x : c.w;
        const uint32_t wd[4] = {r2 ? a2 : a0, r2 ? a3 : a1, r2 ? a0 : a2, r2 ? a1 : a3};
        uint32_t sc[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t code = (scl[i] >> (8 * k)) & 255u;
          const uint32_t v = code * 0x00100010u + 0x6f806f80u;   // bf16 of the scale * 2^112, twice: (code + 8 * 223) << 4
          sc[k] = code == 0 ? 0u : (code == 255 ? 0x7fff7fffu : v);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint32_t s = ((m + rot) & 2) ? sc[1] : sc[0];
          sts128(pair + ((dst[m] + (i >> 1) * (NT * 128) + (i & 1) * 512) ^ ((i & 1) * 64)), mul_bf16x2(lat4::pair_bits<0>(wd[m]), s),
                 mul_bf16x2(lat4::pair_bits<1>(wd[m]), s), mul_bf16x2(lat4::pair_bits<2>(wd[m]), s),
                 mul_bf16x2(lat4::pair_bits<3>(wd[m]), s));
        }
      }
      fence_async();                       // the MMAs read these stores; the next gathers overwrite what was read
      __syncwarp();
      if (lane == 0) {
        bar_arrive(&c_full[q]);
        bar_arrive(&f_empty[P % (FD / 2)]);
      }
    }
    if (lane == 0) prog[PG_DEQ + dw] = written;
  } else if (warp < MMA_WARP) {
    // ------------------------------------------------ gathers: positions 16 gw .. 16 gw + 15 of each tile
    // Two tiles' entries are looked up at once, one per lane (lane = 16 * tile + position): loaded two blocks ahead, their pages one.
    const int gw = warp - GATHER_WARP;
    const int n_tiles = 2 * n_pairs;       // a last half pair is filled with rows outside the map: zeros
    const int32_t* idx_row = p.idx + (int64_t)r * p.n_idx;
    auto place = [&](int blk) -> int64_t { return j0 + (int64_t)(2 * blk + (lane >> 4)) * NT + 16 * gw + (lane & 15); };
    auto raw = [&](int blk) -> int32_t { return p.n_idx > 0 ? idx_row[min(place(blk), (int64_t)p.n_idx - 1)] : 0; };
    int32_t e0 = raw(0), e1 = raw(1), e2 = raw(2);       // (clamped: any block may be asked for)
    const int64_t limit = p.row_pos[r] + p.row_pos_add;
    const int64_t abase = p.n_append > 0 ? p.append_base[r] + 1 : 0;
    const int breq = request_of_row_warp(p.row_offsets, p.B, (uint32_t)r);
    const int64_t base = PAGED ? 0 : p.cache_start[breq];
    auto pos_of = [&](int blk, int32_t e) -> int64_t {
      const int64_t at = place(blk);
      if (at >= j1) return -1;
      return entry_pos(p, at < p.n_idx ? (int64_t)e : abase + (at - p.n_idx), limit);
    };
    int64_t s1 = pos_of(0, e0);            // positions and pages of the next block
    int32_t pg1 = PAGED ? page_entry(p, breq, s1) : -1;
    int32_t row = 0;                       // pool rows of the present block (a row outside the map reads zeros)
    uint32_t there = 0;                    // which of them are there
    int codes = n_tiles, ropes = n_tiles;
    for (int t = 0; t < n_tiles; ++t) {
      if (t % 2 == 0) {                    // the next block becomes the present one
        const int blk = t / 2;
        const int64_t rw = entry_row<PAGED>(p, s1, base, pg1);
        row = rw >= 0 ? (int32_t)rw : (int32_t)p.pool;
        there = __ballot_sync(0xffffffffu, rw >= 0);
        if (rank == 0 && rw >= 0) {        // the rope values are fetched a little later
          const uint8_t* rope = p.latent + rw * lat4::ROW + lat4::OFF_ROPE;
          asm volatile("prefetch.global.L2 [%0];" ::"l"(rope));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(rope + 127));
        }
        s1 = pos_of(blk + 1, e1);
        if (PAGED) pg1 = page_entry(p, breq, s1);
        e1 = e2;
        e2 = raw(blk + 3);
      }
      int y[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = __shfl_sync(0xffffffffu, row, 16 * (t & 1) + i);
      const int f = t % FD, P = t >> 1, q = P % NPAIR, n = P / NPAIR;
      if (t >= FD && !(t & 1) && !wait_all(&f_empty[P % (FD / 2)], (t / FD - 1) & 1, abort_flag, p.status)) {
        codes = ropes = t;
        break;
      }
      const uint32_t dst = saddr(sm + OFF_F + f * F_TILE);
      if (elect_one()) {
        uint64_t* const full = &f_full[P % (FD / 2)];
        if (t & 1) bar_arrive_tx(full, 16 * (128 + 16));
        else bar_expect_tx(full, 16 * (128 + 16));
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          gather4(dst + (4 * gw + g) * 512, &tm_codes, (int)rank * 128, y + 4 * g, full);
          gather4(dst + F_SCL + (4 * gw + g) * 128, &tm_scale, lat4::OFF_SCALE + (int)rank * 16, y + 4 * g, full);
        }
      }
      __syncwarp();
      // validity bits and (rank 0) the rope values, straight into their chunk, once the pair buffer is free
      if (n > 0 && !(t & 1) && !wait_all(&c_empty[q], (n - 1) & 1, abort_flag, p.status)) {
        codes = t + 1;
        ropes = t;
        break;
      }
      if (lane == 0) *(uint16_t*)(mask_s + 8 * q + 4 * (t & 1) + 2 * gw) = (uint16_t)(there >> (16 * (t & 1)));
      __syncwarp();
      if (elect_one()) {
        if (rank == 0) {
          if (t & 1) bar_arrive_tx(&c_full[q], 2048);
          else bar_expect_tx(&c_full[q], 2048);
          const uint32_t rope = saddr(sm + OFF_C + q * PAIR_STRIDE + 4 * CHUNK) + (t & 1) * (NT * 128) + gw * 2048;
#pragma unroll
          for (int g = 0; g < 4; ++g) gather4(rope + g * 512, &tm_rope, 0, y + 4 * g, &c_full[q]);
        } else if (t & 1) {
          bar_arrive(&c_full[q]);
        }
      }
      __syncwarp();
    }
    if (lane == 0) {
      prog[PG_CODES + gw] = codes;
      prog[PG_ROPE + gw] = ropes;
    }
  } else if (warp == FREE_WARP) {
    // ------------------------------------------------ receive slots back to the other CTA
    // Its next copy must not overtake the reads of the four warps here, which have to be released at cluster scope.  A warp that does
    // nothing else does so: by the softmax warps it held up the chain (226 us for the 192 rows), by the MMA warp too (232), a
    // relaxed arrival (214) orders nothing.
    const uint32_t xfree_peer = map_rank(saddr(x_free), peer);
    for (int P = 0; P < n_pairs; ++P) {
      // (a warp arrives on dec after its reads)
      if (!wait_all(&dec[4 * (P & 1) + (lane & 3)], (P >> 1) & 1, abort_flag, p.status)) break;
      if (lane == 0) bar_arrive_remote(xfree_peer + (P & 1) * 8);
      __syncwarp();
    }
  } else {
    // ------------------------------------------------ MMA issue: QK(0), then for every pair P QK(P + 1) and PV(P)
    const uint64_t qr_desc = desc_sw128(saddr(sm + OFF_QR), 16, 1024);
    const uint64_t c_desc0 = desc_sw128(saddr(sm + OFF_C), 16, 1024);
    const uint64_t v_desc0 = desc_sw128(saddr(sm + OFF_C), CHUNK, 1024);
    const int nk = rank == 0 ? 20 : 16;
    bool ok = wait_all(q_ready, 0, abort_flag, p.status);
    fence_after();
    auto qk = [&](int n) -> bool {
      const int b = n % NPAIR;
      const uint32_t par = (n / NPAIR) & 1;
      if (!wait_all(&c_full[b], par, abort_flag, p.status)) return false;
      fence_after();
      const uint64_t cd = c_desc0 + (uint64_t)((b * PAIR_STRIDE) >> 4);
      const uint32_t d = tmem + TM_S0 + (n & 1) * 64;
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 20; ++k)
          if (k < nk) {
            const uint32_t off = (uint32_t)((k >> 2) * CHUNK + (k & 3) * 32) >> 4;
            if (k < 16) mma_ts(d, tmem + TM_Q + k * 8, cd + off, IDESC_QK, k > 0 ? 1u : 0u);
            else mma_ss(d, qr_desc + (uint64_t)(((k & 3) * 32) >> 4), cd + off, IDESC_QK, 1u);
          }
        bar_arrive(&s_full[n & 1]);
        commit(&s_full[n & 1]);
      }
      __syncwarp();
      return true;
    };
    if (ok && n_pairs > 0) ok = qk(0);
    for (int P = 0; P < n_pairs && ok; ++P) {
      if (P + 1 < n_pairs) ok = qk(P + 1);       // into the buffer that PV(P - 1), issued before, has read
      ok = ok && wait_all(&p_full[P & 1], (P >> 1) & 1, abort_flag, p.status);
      if (!ok) break;
      fence_after();
      const uint64_t vd = v_desc0 + (uint64_t)(((P % NPAIR) * PAIR_STRIDE) >> 4);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < NP / 16; ++k)
          mma_ts(tmem + TM_O, tmem + TM_S0 + (P & 1) * 64 + k * 8, vd + (uint64_t)((k * 16 * 128) >> 4), IDESC_PV,
                 P > 0 || k > 0 ? 1u : 0u);
        commit(&pv_done[P & 1]);
        commit(&c_empty[P % NPAIR]);
      }
      __syncwarp();
    }
    if (elect_one()) commit(drain);
    __syncwarp();
    volatile int dummy = 0;
    mbar::wait<false>(drain, 0, &dummy, p.status, mbar::DEFAULT_LIMIT_NS);
  }

  fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
  if (threadIdx.x == 0 && *abort_flag)
    for (uint32_t c = 0; c < (p.fused ? 2u * (uint32_t)p.n_splits : 2u); ++c)
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_rank(saddr((const void*)given_up), c)), "r"(1) : "memory");
  // neither CTA starts another copy into the other's shared memory, and with fused splits every partial of the row is written
  cluster_sync();
  if (*given_up) {     // nothing is merged, and no CTA leaves while copies to it, or from it, are on their way
    if (p.n_splits > 1 && !p.fused && threadIdx.x < HG && h0 + (int)threadIdx.x < p.H) {     // (a NaN: not finished)
      const int64_t rh = (int64_t)r * p.H + h0 + threadIdx.x;
      p.part_ml[((rh * p.n_splits + split) * 2 + rank) * 2] = __uint_as_float(0x7fffffffu);
    }
    if (threadIdx.x == 0) settle(sm, bars, map_rank(saddr((const void*)prog), peer), rank == 0, p.status);
    __syncwarp();
    cluster_sync();
    return;
  }
  if (p.fused) {
    const int lo = split * HG / p.n_splits, hi = (split + 1) * HG / p.n_splits;
    if (p.n_splits == 2) merge_splits<2>(p, r, h0, lo, hi, rank);
    else if (p.n_splits == 3) merge_splits<3>(p, r, h0, lo, hi, rank);
    else merge_splits<4>(p, r, h0, lo, hi, rank);
  }
}

namespace {

cudaLaunchConfig_t config(dim3 grid, int cluster_z, cudaStream_t st, cudaLaunchAttribute* attrs) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = st;
  attrs[0].id = cudaLaunchAttributeClusterDimension;
  attrs[0].val.clusterDim.x = 1;
  attrs[0].val.clusterDim.y = 2;
  attrs[0].val.clusterDim.z = cluster_z;
  attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // see launch_k()
  attrs[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = 1;
  return cfg;
}
bool prepare() {
  static std::atomic<uint64_t> attr[2];
  return set_smem_limit_once(sparse_mla4_tc_kernel<false>, SMEM_BYTES, attr[0]) &&
         set_smem_limit_once(sparse_mla4_tc_kernel<true>, SMEM_BYTES, attr[1]);
}
// CTAs that run at once with `z` splits of a row per cluster (cached per device; -1 in the cache stands for none)
int resident_ctas(int z) {
  static std::atomic<int> cache[kMaxCachedDevices][MAX_SPLITS + 1];
  const int dev = current_device();
  const bool cacheable = dev >= 0 && dev < kMaxCachedDevices;
  if (cacheable) {
    const int v = cache[dev][z].load(std::memory_order_relaxed);
    if (v) return v < 0 ? 0 : v;
  }
  int n = 0, clusters = 0;
  cudaLaunchAttribute attrs[2];
  cudaLaunchConfig_t cfg = config(dim3(1, 2, z), z, 0, attrs);
  if (prepare() && cudaOccupancyMaxActiveClusters(&clusters, (void*)sparse_mla4_tc_kernel<false>, &cfg) == cudaSuccess && clusters > 0)
    n = 2 * z * clusters;
  else
    n = z == 1 ? (num_sms() & ~1) : 0;
  cudaGetLastError();
  if (cacheable) cache[dev][z].store(n > 0 ? n : -1, std::memory_order_relaxed);
  return n;
}
// What a CTA takes beyond its pairs, in pairs
constexpr double START_PAIRS = 7.0;

}  // namespace
}  // namespace m4

bool mla4_tc_supported(const MlaPlan& p) {
  if (p.dtype != MTPSD_FP4_MLA || p.d_latent != 576 || p.d_v != 512 || cc_major() != 10) return false;
  const char* env = getenv("MTPSD_MLA");
  if (env && env[0] == 'm') return false;   // "mma": the mma.sync kernel, as for the other formats
  if (p.pool > 0x7ffffffeLL || (int64_t)p.R * p.H > 0x7fffffffLL || p.R > 0x7fffffff / 2 || ceil_div(p.H, m4::HG) * 2 > 65535) return false;
  if (((uintptr_t)p.latent | (uintptr_t)p.q | (uintptr_t)p.out | (uintptr_t)p.ws) % 16) return false;
  return tma_available();
}

bool mla4_tc_fuse(int n_splits) { return n_splits >= 2 && n_splits <= m4::MAX_SPLITS && m4::resident_ctas(n_splits) > 0; }

// Positions per split (a multiple of NP): the split count with the least modelled time, waves of resident CTAs that take their pairs
// and START_PAIRS more.
int mla4_tc_per_split(int R, int H, int64_t total) {
  const int64_t pairs = ceil_div(total, m4::NP), units = (int64_t)R * ceil_div(H, m4::HG) * 2;
  int64_t best = 1;
  double best_cost = 1e30;
  for (int64_t s = 1; s <= 65 && s <= pairs; ++s) {
    const int64_t per = ceil_div(pairs, s);
    if (ceil_div(pairs, per) != s) continue;
    const int slots = mla4_tc_fuse((int)s) ? m4::resident_ctas((int)s) : m4::resident_ctas(1);
    double cost = (double)ceil_div(units * s, slots) * ((double)per + m4::START_PAIRS);
    if (cost < best_cost - 1e-9) {
      best_cost = cost;
      best = s;
    }
  }
  const int64_t per = ceil_div(pairs, best) * m4::NP;
  return (int)(per > 0 ? per : m4::NP);
}

int launch_sparse_mla4_tc(const MlaPlan& p, int n_splits, int per_split, float* part_o, float* part_ml, cudaStream_t st,
                          bool* combined) {
  using namespace m4;
  Params k;
  k.B = p.B; k.R = p.R; k.H = p.H; k.n_idx = p.n_idx; k.n_append = p.n_append;
  k.sl2 = p.scale * LOG2E * UP; k.row_pos_add = p.row_pos_add;
  k.q = (const __nv_bfloat16*)p.q; k.latent = (const uint8_t*)p.latent; k.pool = p.pool;
  k.cache_start = p.cache_start; k.bt = p.pg.bt; k.bt_stride = p.pg.stride; k.pg_shift = p.pg.shift;
  k.row_offsets = p.row_offsets; k.row_pos = p.row_pos; k.idx = p.idx; k.append_base = p.append_base;
  k.out = (__nv_bfloat16*)p.out; k.lse = p.lse; k.part_o = part_o; k.part_ml = part_ml;
  k.n_splits = n_splits; k.per_split = per_split; k.status = p.status;
  k.fused = mla4_tc_fuse(n_splits) ? 1 : 0;
  *combined = k.fused != 0;
  alignas(64) CUtensorMap tm_codes, tm_scale, tm_rope, tm_st;
  const uint64_t rh = (uint64_t)p.R * p.H;
  const uint64_t out_dims[2] = {(uint64_t)DV, rh}, out_strides[1] = {(uint64_t)DV * 2};
  const uint32_t out_box[2] = {64, 32};
  const uint64_t po_dims[3] = {(uint64_t)DV, (uint64_t)n_splits, rh};
  const uint64_t po_strides[2] = {(uint64_t)DV * 4, (uint64_t)DV * 4 * n_splits};
  const uint32_t po_box[3] = {32, 1, 32};
  const bool st_ok = n_splits == 1 ? make_tma_store_map(&tm_st, false, p.out, 2, out_dims, out_strides, out_box)
                                   : make_tma_store_map(&tm_st, true, part_o, 3, po_dims, po_strides, po_box);
  if (!st_ok || !make_tma_2d_plain_u8(&tm_codes, p.latent, lat4::ROW, (uint64_t)p.pool, 128) ||
      !make_tma_2d_plain_u8(&tm_scale, p.latent, lat4::ROW, (uint64_t)p.pool, 16) ||
      !make_tma_2d(&tm_rope, 1, (const uint8_t*)p.latent + lat4::OFF_ROPE, 64, (uint64_t)p.pool, lat4::ROW, 64, 1, false)) {
    set_error("sparse_mla: cuTensorMapEncodeTiled failed");
    return MTPSD_ECUDA;
  }
  if (!prepare()) {
    set_error("sparse_mla4_tc: cudaFuncSetAttribute failed");
    return MTPSD_ECUDA;
  }
  cudaLaunchAttribute attrs[2];
  cudaLaunchConfig_t cfg = config(dim3(p.R, (unsigned)ceil_div(p.H, HG) * 2, n_splits), k.fused ? n_splits : 1, st, attrs);
  cfg.numAttrs = 2;
  const cudaError_t e = p.pg.bt ? cudaLaunchKernelEx(&cfg, sparse_mla4_tc_kernel<true>, tm_codes, tm_scale, tm_rope, tm_st, k)
                                : cudaLaunchKernelEx(&cfg, sparse_mla4_tc_kernel<false>, tm_codes, tm_scale, tm_rope, tm_st, k);
  if (e != cudaSuccess) {
    set_error("sparse_mla4_tc: launch failed: %s", cudaGetErrorString(e));
    return MTPSD_ECUDA;
  }
  return check_launch("sparse_mla4_tc");
}

}  // namespace mtpsd
