// Block tables from the requests' lengths, the free list's other end (release), and the slots of ragged tokens.
//
// Page counts become places in the free list by an exclusive prefix sum over the requests: deterministic, no atomics.  Every
// CTA of the grow kernel makes that sum for itself (16 bytes a request, from L2) and keeps it in shared memory, so the CTAs need
// not wait for one another: each then writes its share of the table entries and of the slots, and a slot in a page that the call
// hands out is taken from the free list directly, not from the table that another CTA writes.
// The bytes written bound the large calls (16 per token, 4 per entry), the launch and three dependent loads the small ones.
#include "cache.h"
#include "common.cuh"

namespace mtpsd {
namespace {

constexpr int THREADS = 1024;
constexpr int COLS = 512;             // table entries per work item
constexpr int TOKENS = 128;           // tokens per warp that are worth another CTA

// Exclusive sum of v over the block's threads; *total the sum of all.  warp_sums: [33] in shared memory (the grow kernel keeps a number behind them).
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warp_sums, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const int64_t s = warp_sums[lane];
    int64_t z = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, z, o);
      if (lane >= o) z += y;
    }
    warp_sums[lane] = z - s;
    if (lane == 31) warp_sums[32] = z;
  }
  __syncthreads();
  *total = warp_sums[32];
  return warp_sums[warp] + x - v;
}

__device__ __forceinline__ int64_t pages_of(int64_t n, int shift) { return (n + (1LL << shift) - 1) >> shift; }

struct Grow {
  int32_t* table;
  int stride, shift, B, free_cap;
  const int64_t* old_len;
  const int64_t* new_len;
  const int32_t* free_pages;
  const int32_t* n_free;
  int32_t* n_free_out;        // null: left to the finish kernel
  int64_t* lengths;           // the same
  const uint32_t* offsets;
  int64_t* slots;
  int64_t* positions;
  int64_t T;
  int64_t step;               // tokens per warp
  int32_t* status;
};

// What a request gets: entries first .. first + need - 1 of its row; from: its first place in the order of the pages handed out, or
// -1 when it is not served.
struct Share { int32_t first, need, from; };

// The shares of all requests into sh (unless null); lengths and the free count are written by the CTA that is told to.
__device__ int32_t plan_shares(const Grow& a, Share* sh, bool write, int64_t* warp_sums) {
  int32_t n_free = *a.n_free;
  if (n_free < 0 || n_free > a.free_cap) {
    if (write && threadIdx.x == 0) flag_status(a.status, MTPSD_STATUS_ROW_RANGE);
    n_free = n_free < 0 ? 0 : a.free_cap;
  }
  const int64_t room = (int64_t)a.stride << a.shift;
  unsigned* taken = (unsigned*)(warp_sums + 33);
  int64_t before = 0;
  if (threadIdx.x == 0) *taken = 0;
  __syncthreads();
  for (int b0 = 0; b0 < a.B; b0 += THREADS) {
    const int b = b0 + threadIdx.x;
    int64_t first = 0, need = 0, len_old = 0, len_new = 0;
    bool bad = false;
    if (b < a.B) {
      len_old = a.old_len ? a.old_len[b] : 0;
      len_new = a.new_len[b];
      bad = len_old < 0 || len_new < 0 || len_new > room || len_old > room;
      if (!bad) {
        first = pages_of(len_old, a.shift);
        need = max((int64_t)0, pages_of(len_new, a.shift) - first);
      }
    }
    int64_t total;
    const int64_t excl = before + block_scan(need, warp_sums, &total);
    before += total;
    const bool served = need == 0 || excl + need <= n_free;
    if (b < a.B) {
      if (sh) sh[b] = Share{(int32_t)first, (int32_t)need, served ? (int32_t)excl : -1};
      if (write) {
        if (bad) flag_status(a.status, MTPSD_STATUS_ROW_RANGE);
        if (!served) flag_status(a.status, MTPSD_STATUS_NO_PAGES);
        if (a.lengths) a.lengths[b] = served && !bad ? max(len_old, len_new) : len_old;
      }
    }
    // the served requests that need pages come first: what they take ends with the last of them
    const unsigned most = __reduce_max_sync(0xffffffffu, served && need > 0 ? (unsigned)(excl + need) : 0u);
    if ((threadIdx.x & 31) == 0 && most) atomicMax(taken, most);
  }
  __syncthreads();
  if (write && a.n_free_out && threadIdx.x == 0) *a.n_free_out = n_free - (int32_t)*taken;
  return n_free;
}

// Slots and positions of the tokens, `step` consecutive ones (a multiple of 32) per warp; page_of(b, p): the page of entry p of
// request b's row, or a negative number.  A run of one request needs one search (one run per warp: searches and lengths are chains of
// loads; 3.4 M tokens of 128 requests took 23.7 us with 128 tokens per step); where requests are short each lane finds its token's among the
// next 32 offsets, which the lanes hold.
template <class PageOf>
__device__ __forceinline__ void map_tokens(const uint32_t* offsets, const int64_t* lengths, int B, int stride, int shift,
                                           int64_t T, int64_t step, int64_t* slots, int64_t* positions, int32_t* status,
                                           PageOf page_of) {
  if (B == 0) return;
  const int lane = threadIdx.x & 31;
  const int64_t warp = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int64_t begin = offsets[0];
  int64_t end = offsets[B];
  if (end > T) {
    if (warp == 0 && lane == 0) flag_status(status, MTPSD_STATUS_ROW_RANGE);
    end = T;
  }
  bool missing = false;
  auto put = [&](int64_t t, int b, int64_t pos) {
    int64_t slot = -1;
    if (pos >= 0 && (pos >> shift) < stride) {
      const int64_t pg = page_of(b, (int32_t)(pos >> shift));
      if (pg >= 0) slot = (pg << shift) | (pos & ((1LL << shift) - 1));
    }
    missing = missing || slot < 0;
    slots[t] = slot;
    if (positions) positions[t] = pos;
  };
  // the warp's tokens, a request after the other: long runs of one request, or 32 tokens of several
  const int64_t t0 = max(begin, warp * step), t1 = min(end, (warp + 1) * step);
  int b = 0;
  int64_t o1 = 0;                              // end of request b
  for (int64_t t = t0; t < t1;) {
    if (o1 <= t) {
      b = request_of_row_warp(offsets, B, (uint32_t)t);
      o1 = offsets[b + 1];
    }
    const int64_t u1 = min(o1, t1);
    if (u1 == t1 || u1 - t >= 32) {
      const int64_t add = lengths[b] - o1;     // position = token + this
#pragma unroll 4
      for (int64_t u = t + lane; u < u1; u += 32) put(u, b, u + add);
      t = u1;
      continue;
    }
    const int64_t u = t + lane;
    int64_t o_end = 0;
    int mine = -1;                             // the lane's request
    for (int b0 = b; b0 < B; b0 += 32) {       // offsets b0 + 1 .. b0 + 32, one per lane
      const int64_t off = offsets[min(b0 + 1 + lane, B)];
      int c = 0;                               // how many of them are <= u (they do not fall)
#pragma unroll
      for (int w = 16; w; w >>= 1) {
        const int64_t v = __shfl_sync(0xffffffffu, off, c + w - 1);
        c += v <= u ? w : 0;
      }
      const int64_t v = __shfl_sync(0xffffffffu, off, c);
      if (mine < 0 && v > u && b0 + c < B) {
        mine = b0 + c;
        o_end = v;
      }
      if (!__any_sync(0xffffffffu, mine < 0 && u < t1)) break;
    }
    if (mine >= 0 && u < t1) put(u, mine, u - o_end + lengths[mine]);
    b = __shfl_sync(0xffffffffu, mine, 31);    // (looked up again where the last lane has none)
    o1 = __shfl_sync(0xffffffffu, o_end, 31);
    t += 32;
  }
  if (__any_sync(0xffffffffu, missing) && lane == 0) flag_status(status, MTPSD_STATUS_ROW_RANGE);
}

__global__ void __launch_bounds__(THREADS) block_table_grow_kernel(Grow a) {
  griddep_wait();                // the previous kernel's writes are visible from here on
  griddep_launch_dependents();
  extern __shared__ Share shares[];
  __shared__ int64_t warp_sums[34];
  const int32_t n_free = plan_shares(a, shares, blockIdx.x == 0, warp_sums);

  // table entries, COLS of one row per warp and step
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (THREADS / 32), warp = (int64_t)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5);
  const int chunks = (a.stride + COLS - 1) / COLS;
  bool bad_id = false;
  for (int64_t w = warp; w < (int64_t)a.B * chunks; w += warps) {
    const int b = (int)(w / chunks);
    const Share s = shares[b];
    const int lo = (int)(w % chunks) * COLS, hi = min(a.stride, lo + COLS);
    const int p0 = a.old_len ? max(lo, s.first) : lo, p1 = a.old_len ? min(hi, s.first + s.need) : hi;
    for (int p = p0 + lane; p < p1; p += 32) {
      int32_t page = -1;
      if (s.from >= 0 && p < s.first + s.need) {
        page = a.free_pages[n_free - 1 - (s.from + (p - s.first))];
        bad_id = bad_id || page < 0;
      }
      a.table[(int64_t)b * a.stride + p] = page;
    }
  }
  if (__any_sync(0xffffffffu, bad_id) && lane == 0) flag_status(a.status, MTPSD_STATUS_INDEX_RANGE);
  if (!a.offsets) return;
  map_tokens(a.offsets, a.new_len, a.B, a.stride, a.shift, a.T, a.step, a.slots, a.positions, a.status,
             [&](int b, int32_t p) -> int32_t {
               const Share s = shares[b];
               if (p >= s.first && p < s.first + s.need)
                 return s.from < 0 ? -1 : a.free_pages[n_free - 1 - (s.from + (p - s.first))];
               return a.old_len ? a.table[(int64_t)b * a.stride + p] : -1;   // an entry that this call does not write
             });
}

// Lengths and free count of a grow call that writes them over its inputs, after every CTA has read those.
__global__ void __launch_bounds__(THREADS) block_table_finish_kernel(Grow a) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ int64_t warp_sums[34];
  a.status = nullptr;            // flagged by the grow kernel
  plan_shares(a, nullptr, true, warp_sums);
}

__global__ void __launch_bounds__(256) slot_map_kernel(const int32_t* table, int stride, int shift, int B, const uint32_t* offsets,
                                                       const int64_t* lengths, int64_t T, int64_t step, int64_t* slots,
                                                       int64_t* positions, int32_t* status) {
  griddep_wait();
  griddep_launch_dependents();
  map_tokens(offsets, lengths, B, stride, shift, T, step, slots, positions, status,
             [&](int b, int32_t p) -> int32_t { return __ldg(table + (int64_t)b * stride + p); });
}

// One CTA: the pages that each request returns are counted (a warp per request), summed, then moved.
__global__ void __launch_bounds__(THREADS) block_table_release_kernel(int32_t* table, int stride, int shift, int B,
                                                                      const int64_t* old_len, const int64_t* keep_len,
                                                                      int32_t* free_pages, int free_cap, int32_t* n_free,
                                                                      int32_t* status) {
  griddep_wait();
  griddep_launch_dependents();
  extern __shared__ int32_t place[];     // [B] pages of the request, then its first place behind the free list (-1: kept)
  __shared__ int64_t warp_sums[34];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto range = [&](int b, int* lo, int* hi) -> bool {
    const int64_t o = old_len[b], k = keep_len ? keep_len[b] : 0;
    if (o < 0 || k < 0 || o > ((int64_t)stride << shift)) return false;
    *hi = (int)pages_of(o, shift);
    *lo = (int)pages_of(min(k, o), shift);   // (a length near 2^63, "all of them", has no page count)
    return true;
  };
  for (int b = warp; b < B; b += THREADS / 32) {
    int lo = 0, hi = 0, n = 0;
    if (!range(b, &lo, &hi)) {
      lo = hi = 0;
      if (lane == 0) flag_status(status, MTPSD_STATUS_ROW_RANGE);
    }
    for (int p = lo + lane; p < hi; p += 32) n += table[(int64_t)b * stride + p] >= 0;
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) place[b] = n;
  }
  const int32_t start = *n_free;
  if (start < 0 || start > free_cap) {   // (uniform) nothing can be placed
    if (threadIdx.x == 0) flag_status(status, MTPSD_STATUS_ROW_RANGE);
    return;
  }
  __syncthreads();
  int64_t before = start, kept = start;
  for (int b0 = 0; b0 < B; b0 += THREADS) {
    const int b = b0 + threadIdx.x;
    const int64_t n = b < B ? place[b] : 0;
    int64_t total;
    const int64_t at = before + block_scan(n, warp_sums, &total);
    before += total;
    const bool fits = at + n <= free_cap;
    if (b < B) {
      place[b] = fits ? (int32_t)at : -1;
      if (!fits) flag_status(status, MTPSD_STATUS_WRITE_RANGE);
    }
    int64_t moved;
    block_scan(fits ? n : 0, warp_sums, &moved);
    kept += moved;
  }
  __syncthreads();
  if (threadIdx.x == 0) *n_free = (int32_t)kept;
  for (int b = warp; b < B; b += THREADS / 32) {
    int lo = 0, hi = 0;
    int at = place[b];
    if (at < 0 || !range(b, &lo, &hi)) continue;
    for (int p = lo; p < hi; p += 32) {
      int32_t* e = table + (int64_t)b * stride + p + lane;
      const int32_t page = p + lane < hi ? *e : -1;
      const uint32_t have = __ballot_sync(0xffffffffu, page >= 0);
      if (page >= 0) {
        free_pages[at + __popc(have & ((1u << lane) - 1))] = page;
        *e = -1;
      }
      at += __popc(have);
    }
  }
}

}  // namespace

int launch_block_table_grow(const mtpsd_block_table_args& c, int shift, cudaStream_t st) {
  Grow a;
  a.table = c.block_table; a.stride = c.bt_stride; a.shift = shift; a.B = c.B; a.free_cap = c.free_cap;
  a.old_len = c.old_len; a.new_len = c.new_len; a.free_pages = c.free_pages; a.n_free = c.n_free;
  a.n_free_out = c.n_free_out; a.lengths = c.lengths; a.offsets = c.token_offsets; a.slots = c.slots; a.positions = c.positions;
  a.T = c.token_offsets ? c.T : 0; a.status = c.dev_status;
  // One CTA for what its 32 warps do in a few steps each; else as many as find work, one per SM.
  const int64_t items = (int64_t)a.B * ((a.stride + COLS - 1) / COLS) + ceil_div(a.T, TOKENS);
  const int64_t want = ceil_div(items, 32);
  const int grid = (int)(want < 1 ? 1 : (want > num_sms() ? num_sms() : want));
  a.step = ceil_div(ceil_div(a.T, 32), (int64_t)grid * (THREADS / 32)) * 32;
  const bool in_place = c.n_free_out == c.n_free || (c.lengths && c.lengths == c.old_len);
  const bool finish = grid > 1 && in_place;
  if (finish) {
    a.n_free_out = nullptr;
    a.lengths = nullptr;
  }
  // (asked for whatever B is: the 48 KB that need no asking hold the kernel's static shared memory too)
  static std::atomic<uint64_t> attr{0};
  if (!set_smem_limit_once(block_table_grow_kernel, (int)(sizeof(Share) * TABLES_MAX_B), attr)) {
    set_error("block_table_grow: cudaFuncSetAttribute failed");
    return MTPSD_ECUDA;
  }
  launch_k(block_table_grow_kernel, grid, THREADS, sizeof(Share) * (size_t)a.B, st, a);
  if (finish) {
    // lengths and the free count move only behind tables that were written
    if (int rc = check_launch("block_table_grow")) return rc;
    a.n_free_out = c.n_free_out;
    a.lengths = c.lengths;
    launch_k(block_table_finish_kernel, 1, THREADS, 0, st, a);
  }
  return check_launch("block_table_grow");
}

int launch_block_table_release(int32_t* table, int stride, int shift, int B, const int64_t* old_len, const int64_t* keep_len,
                               int32_t* free_pages, int free_cap, int32_t* n_free, int32_t* status, cudaStream_t st) {
  launch_k(block_table_release_kernel, 1, THREADS, sizeof(int32_t) * (size_t)B, st, table, stride, shift, B, old_len, keep_len,
           free_pages, free_cap, n_free, status);
  return check_launch("block_table_release");
}

int launch_slot_map(const Paging& pg, int B, const uint32_t* offsets, const int64_t* lengths, int64_t T, int64_t* slots,
                    int64_t* positions, int32_t* status, cudaStream_t st) {
  const int64_t most = 8 * (int64_t)num_sms(), want = ceil_div(T, 8 * 32), grid = want > most ? most : want;
  const int64_t step = ceil_div(ceil_div(T, 32), grid * 8) * 32;
  launch_k(slot_map_kernel, (unsigned)grid, 256, 0, st, pg.bt, pg.stride, pg.shift, B, offsets, lengths, T,
           step, slots, positions, status);
  return check_launch("slot_map");
}

}  // namespace mtpsd
