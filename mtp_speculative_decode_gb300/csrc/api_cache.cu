// C ABI of the calls that fill the caches: argument checks and dispatch.  Nothing here allocates device memory.
#include "cache.h"
#include "common.cuh"

namespace mtpsd {
namespace {

template <class... A>
int fail(int code, const char* fmt, A... args) {
  set_error(fmt, args...);
  return code;
}
bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// log2 of a page size, or -1 when it is none
int page_shift(int32_t ps) {
  if (ps < 1 || ps > 65536 || (ps & (ps - 1))) return -1;
  int s = 0;
  while ((1 << s) < ps) ++s;
  return s;
}

int check_side(const mtpsd_head_side* c, const char* who, bool key, int64_t T, int32_t rot_dim, const int64_t* slots) {
  if (!c) return MTPSD_OK;
  if (c->heads < 1 || c->heads > 65535 || c->D < 1 || c->D > 1024)
    return fail(MTPSD_EINVAL, "norm_rope: %s: need 1 <= heads <= 65535, 1 <= D <= 1024", who);
  if (c->dtype != MTPSD_BF16 && c->dtype != MTPSD_F32)
    return fail(MTPSD_EUNSUPPORTED, "norm_rope: %s: dtype must be MTPSD_BF16 or MTPSD_F32", who);
  if (c->norm != MTPSD_NORM_NONE && c->norm != MTPSD_NORM_RMS && c->norm != MTPSD_NORM_LAYER)
    return fail(MTPSD_EINVAL, "norm_rope: %s: unknown norm", who);
  if (c->norm && (c->norm_dim < 1 || c->norm_dim > c->D))
    return fail(MTPSD_EINVAL, "norm_rope: %s: need 1 <= norm_dim <= D", who);
  if (c->norm == MTPSD_NORM_NONE && (c->weight || c->bias))
    return fail(MTPSD_EINVAL, "norm_rope: %s: weight or bias without a norm", who);
  if (rot_dim && (c->rot_start < 0 || c->rot_start > c->D - rot_dim))
    return fail(MTPSD_EINVAL, "norm_rope: %s: the turned dims do not fit D", who);
  const bool rows = c->out_dtype == MTPSD_FP8_DS_MLA || c->out_dtype == MTPSD_FP4_MLA;
  const int in_size = c->dtype == MTPSD_F32 ? 4 : 2;
  const int out_size = c->out_dtype == MTPSD_F32 ? 4 : (c->out_dtype == MTPSD_BF16 ? 2 : 1);
  if (rows) {
    if (!key || c->heads != 1 || c->D != 576 || (rot_dim && (rot_dim != 64 || c->rot_start != 512)) ||
        (c->norm && (c->norm_dim > 512 || c->norm_dim % 8)))
      return fail(MTPSD_EUNSUPPORTED, "norm_rope: %s: cache rows need keys of one head, D 576, rot_start 512 and rot_dim 64 (or no "
                  "rotation), and a norm of at most 512 values, a multiple of 8", who);
    if (c->out_token_stride < (c->out_dtype == MTPSD_FP4_MLA ? 416 : 656) || c->out_token_stride % 16)
      return fail(MTPSD_EINVAL, "norm_rope: %s: cache rows need a stride of their bytes, a multiple of 16", who);
  } else if (c->out_dtype == MTPSD_FP8_E4M3) {
    if (c->D != 128) return fail(MTPSD_EUNSUPPORTED, "norm_rope: %s: FP8 needs D 128 (one scale per head)", who);
  } else if (c->out_dtype != MTPSD_BF16 && c->out_dtype != MTPSD_F32) {
    return fail(MTPSD_EUNSUPPORTED, "norm_rope: %s: unknown output type", who);
  }
  if (c->x_token_stride < 0 || c->x_head_stride < 0 || c->out_token_stride < 0 || c->out_head_stride < 0)
    return fail(MTPSD_EINVAL, "norm_rope: %s: negative stride", who);
  if (T * (int64_t)c->heads > (1LL << 31) - 1) return fail(MTPSD_EUNSUPPORTED, "norm_rope: %s: more than 2^31 - 1 heads in a call", who);
  if (T == 0) return MTPSD_OK;
  if (!c->x || !c->out) return fail(MTPSD_EINVAL, "norm_rope: %s: null pointer", who);
  if (c->out_dtype == MTPSD_FP8_E4M3 && !c->scale) return fail(MTPSD_EINVAL, "norm_rope: %s: FP8 needs scale", who);
  if (!aligned(c->x, in_size) || !aligned(c->out, rows ? 16 : (c->out_dtype == MTPSD_FP8_E4M3 ? 4 : out_size)) ||
      !aligned(c->weight, 4) || !aligned(c->bias, 4) || !aligned(c->scale, 4))
    return fail(MTPSD_EINVAL, "norm_rope: %s: misaligned pointer", who);
  if (rows && (!aligned(c->x, 16) || (c->x_token_stride * in_size) % 16 || !aligned(c->weight, 16) || !aligned(c->bias, 16)))
    return fail(MTPSD_EUNSUPPORTED, "norm_rope: %s: cache rows need x, its token stride, weight and bias aligned to 16 bytes", who);
  if (c->out == c->x) {
    if (slots || c->out_dtype != c->dtype || c->out_token_stride != c->x_token_stride || c->out_head_stride != c->x_head_stride)
      return fail(MTPSD_EINVAL, "norm_rope: %s: in place needs the same type and strides and no slots", who);
  }
  return MTPSD_OK;
}

}  // namespace
}  // namespace mtpsd

using namespace mtpsd;

extern "C" {

int mtpsd_block_table_grow(const mtpsd_block_table_args* a, void* stream) {
  set_error("");
  if (!a) return fail(MTPSD_EINVAL, "block_table_grow: null args");
  const int shift = page_shift(a->page_size);
  if (shift < 0) return fail(MTPSD_EINVAL, "block_table_grow: page_size must be a power of two in 1..65536");
  if (a->bt_stride < 1 || a->B < 0 || a->free_cap < 0) return fail(MTPSD_EINVAL, "block_table_grow: need bt_stride >= 1, B >= 0, free_cap >= 0");
  if (a->B > TABLES_MAX_B) return fail(MTPSD_EUNSUPPORTED, "block_table_grow: more than %d requests", TABLES_MAX_B);
  if (a->token_offsets && (a->T < 0 || a->T > 0xffffffffLL)) return fail(MTPSD_EINVAL, "block_table_grow: need 0 <= T < 2^32");
  if (!a->n_free || !a->n_free_out) return fail(MTPSD_EINVAL, "block_table_grow: null pointer");
  if (a->B > 0 && (!a->block_table || !a->new_len || (a->free_cap > 0 && !a->free_pages)))
    return fail(MTPSD_EINVAL, "block_table_grow: null pointer");
  if (a->token_offsets && a->T > 0 && !a->slots) return fail(MTPSD_EINVAL, "block_table_grow: token_offsets without slots");
  if (!aligned(a->block_table, 4) || !aligned(a->old_len, 8) || !aligned(a->new_len, 8) || !aligned(a->free_pages, 4) ||
      !aligned(a->n_free, 4) || !aligned(a->n_free_out, 4) || !aligned(a->lengths, 8) || !aligned(a->token_offsets, 4) ||
      !aligned(a->slots, 8) || !aligned(a->positions, 8) || !aligned(a->dev_status, 4))
    return fail(MTPSD_EINVAL, "block_table_grow: misaligned pointer");
  if (a->lengths && a->lengths == a->new_len) return fail(MTPSD_EINVAL, "block_table_grow: lengths must not be new_len");
  return launch_block_table_grow(*a, shift, (cudaStream_t)stream);
}

int mtpsd_block_table_release(int32_t* block_table, int32_t bt_stride, int32_t page_size, int32_t B, const int64_t* old_len,
                              const int64_t* keep_len, int32_t* free_pages, int32_t free_cap, int32_t* n_free,
                              int32_t* dev_status, void* stream) {
  set_error("");
  const int shift = page_shift(page_size);
  if (shift < 0) return fail(MTPSD_EINVAL, "block_table_release: page_size must be a power of two in 1..65536");
  if (bt_stride < 1 || B < 0 || free_cap < 0) return fail(MTPSD_EINVAL, "block_table_release: need bt_stride >= 1, B >= 0, free_cap >= 0");
  if (B > TABLES_MAX_B) return fail(MTPSD_EUNSUPPORTED, "block_table_release: more than %d requests", TABLES_MAX_B);
  if (B == 0) return MTPSD_OK;
  if (!block_table || !old_len || !n_free || (free_cap > 0 && !free_pages)) return fail(MTPSD_EINVAL, "block_table_release: null pointer");
  if (!aligned(block_table, 4) || !aligned(old_len, 8) || !aligned(keep_len, 8) || !aligned(free_pages, 4) || !aligned(n_free, 4) ||
      !aligned(dev_status, 4))
    return fail(MTPSD_EINVAL, "block_table_release: misaligned pointer");
  return launch_block_table_release(block_table, bt_stride, shift, B, old_len, keep_len, free_pages, free_cap, n_free, dev_status,
                                    (cudaStream_t)stream);
}

int mtpsd_slot_map(const mtpsd_paged_kv* paged, int32_t B, const uint32_t* token_offsets, const int64_t* lengths, int64_t T,
                   int64_t* slots, int64_t* positions, int32_t* dev_status, void* stream) {
  set_error("");
  if (!paged || paged->bt_stride < 1) return fail(MTPSD_EINVAL, "slot_map: needs a block table with bt_stride >= 1");
  Paging pg;
  pg.bt = paged->block_table;
  pg.stride = paged->bt_stride;
  pg.shift = page_shift(paged->page_size);
  if (pg.shift < 0) return fail(MTPSD_EINVAL, "slot_map: page_size must be a power of two in 1..65536");
  if (B < 0 || T < 0 || T > 0xffffffffLL) return fail(MTPSD_EINVAL, "slot_map: need B >= 0, 0 <= T < 2^32");
  if (B == 0 || T == 0) return MTPSD_OK;
  if (!paged->block_table || !token_offsets || !lengths || !slots) return fail(MTPSD_EINVAL, "slot_map: null pointer");
  if (!aligned(paged->block_table, 4) || !aligned(token_offsets, 4) || !aligned(lengths, 8) || !aligned(slots, 8) ||
      !aligned(positions, 8) || !aligned(dev_status, 4))
    return fail(MTPSD_EINVAL, "slot_map: misaligned pointer");
  return launch_slot_map(pg, B, token_offsets, lengths, T, slots, positions, dev_status, (cudaStream_t)stream);
}

int mtpsd_norm_rope(const mtpsd_head_side* q, const mtpsd_head_side* k, int64_t T, const int64_t* positions,
                    const float* cos_sin, int64_t n_pos, int32_t rot_dim, int32_t interleaved, float eps, const int64_t* slots,
                    int64_t pool_tokens, int32_t* dev_status, void* stream) {
  set_error("");
  if (!q && !k) return fail(MTPSD_EINVAL, "norm_rope: neither q nor k");
  if (T < 0 || T > 0x7fffffffLL) return fail(MTPSD_EINVAL, "norm_rope: need 0 <= T < 2^31");
  if (rot_dim < 0 || rot_dim > 1024 || rot_dim % 2) return fail(MTPSD_EINVAL, "norm_rope: rot_dim must be even, 0..1024");
  if (!(eps >= 0.f)) return fail(MTPSD_EINVAL, "norm_rope: eps must not be negative");
  if (slots && (!k || pool_tokens < 0)) return fail(MTPSD_EINVAL, "norm_rope: slots need k and pool_tokens >= 0");
  if (int rc = check_side(q, "q", false, T, rot_dim, nullptr)) return rc;
  if (int rc = check_side(k, "k", true, T, rot_dim, slots)) return rc;
  if (T == 0) return MTPSD_OK;
  if (rot_dim && (!positions || !cos_sin || n_pos < 0)) return fail(MTPSD_EINVAL, "norm_rope: a rotation needs positions and cos_sin");
  if (!aligned(positions, 8) || !aligned(cos_sin, 4) || !aligned(slots, 8) || !aligned(dev_status, 4))
    return fail(MTPSD_EINVAL, "norm_rope: misaligned pointer");
  if (k && (k->out_dtype == MTPSD_FP8_DS_MLA || k->out_dtype == MTPSD_FP4_MLA) && !aligned(cos_sin, 16))
    return fail(MTPSD_EUNSUPPORTED, "norm_rope: cache rows need cos_sin aligned to 16 bytes");
  NormRopePlan p;
  p.q = q; p.k = k; p.T = T; p.positions = positions; p.cos_sin = cos_sin; p.n_pos = n_pos; p.rot_dim = rot_dim;
  p.interleaved = interleaved != 0; p.eps = eps; p.slots = slots; p.pool = pool_tokens; p.status = dev_status;
  return launch_norm_rope(p, (cudaStream_t)stream);
}

int mtpsd_pack_latent_fp4(const void* latent, int32_t dtype, int64_t T, uint8_t* packed, const int64_t* slots,
                          int64_t pool_tokens, int32_t* dev_status, void* stream) {
  set_error("");
  if (T < 0 || pool_tokens < 0 || (!slots && T > pool_tokens)) return fail(MTPSD_EINVAL, "pack_latent_fp4: need T >= 0 and a row for each token");
  if (dtype != MTPSD_BF16 && dtype != MTPSD_F32) return fail(MTPSD_EUNSUPPORTED, "pack_latent_fp4: dtype must be MTPSD_BF16 or MTPSD_F32");
  if (T == 0) return MTPSD_OK;
  if (!latent || !packed) return fail(MTPSD_EINVAL, "pack_latent_fp4: null pointer");
  if (!aligned(latent, 16) || !aligned(packed, 16)) return fail(MTPSD_EINVAL, "pack_latent_fp4: buffers must be 16-byte aligned");
  if (!aligned(slots, 8) || !aligned(dev_status, 4)) return fail(MTPSD_EINVAL, "pack_latent_fp4: misaligned pointer");
  return launch_pack_latent_fp4(latent, dtype == MTPSD_F32, T, packed, slots, pool_tokens, dev_status, (cudaStream_t)stream);
}

}  // extern "C"
