// Launchers of the kernels that fill the caches: block tables and slots, norms with rotation, 4-bit latent rows; and the attention
// over 4-bit rows (internal header).
#pragma once

#include "../../include/mtpsd.h"
#include "internal.h"

namespace mtpsd {

constexpr int TABLES_MAX_B = 8192;   // requests of one grow or release: their page counts are kept in shared memory

int launch_block_table_grow(const mtpsd_block_table_args& a, int shift, cudaStream_t st);
int launch_block_table_release(int32_t* table, int stride, int shift, int B, const int64_t* old_len, const int64_t* keep_len,
                               int32_t* free_pages, int free_cap, int32_t* n_free, int32_t* status, cudaStream_t st);
int launch_slot_map(const Paging& pg, int B, const uint32_t* offsets, const int64_t* lengths, int64_t T, int64_t* slots,
                    int64_t* positions, int32_t* status, cudaStream_t st);

struct NormRopePlan {
  const mtpsd_head_side* q; const mtpsd_head_side* k;   // null: absent
  int64_t T;
  const int64_t* positions; const float* cos_sin; int64_t n_pos;
  int rot_dim; bool interleaved; float eps;
  const int64_t* slots; int64_t pool;
  int32_t* status;
};
int launch_norm_rope(const NormRopePlan& p, cudaStream_t st);

int launch_pack_latent_fp4(const void* latent, bool f32_in, int64_t T, uint8_t* out, const int64_t* slots, int64_t pool,
                           int32_t* status, cudaStream_t st);

// Sparse MLA over 4-bit rows on the tensor cores: whether this call can take it, the positions per split, whether that many splits
// of a row are merged in the kernel.
bool mla4_tc_supported(const MlaPlan& p);
int mla4_tc_per_split(int R, int H, int64_t total);
bool mla4_tc_fuse(int n_splits);
int launch_sparse_mla4_tc(const MlaPlan& p, int n_splits, int per_split, float* part_o, float* part_ml, cudaStream_t st,
                          bool* combined);

}  // namespace mtpsd
