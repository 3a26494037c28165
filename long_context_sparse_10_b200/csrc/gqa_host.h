// Host-side checks and tensor maps shared by the grouped-head (GQA) calls.
#pragma once

#include <cmath>
#include <cstring>

#include "host_util.h"

namespace csa {
namespace gqa {

struct Heads {
  int Hkv, G, dqk, dv;
};

inline bool dims_ok(int dqk, int dv) {
  return (dqk == 192 && dv == 128) || (dqk == 128 && dv == 128) || (dqk == 64 && dv == 64);
}

inline csa_status check_dims(const char* what, int32_t H_kv, int32_t d_qk, int32_t d_v) {
  CSA_REQUIRE(H_kv >= 1 && H_kv <= 65535, "%s: kv heads must be in [1, 65535] (got %d)", what, H_kv);
  if (!dims_ok(d_qk, d_v))
    return fail(CSA_ERR_UNSUPPORTED, "%s: channel widths (d_qk, d_v) must be (192, 128), (128, 128) or (64, 64), got "
                "(%d, %d)", what, d_qk, d_v);
  return CSA_OK;
}

inline csa_status check_heads(const char* what, int32_t H, int32_t H_kv, int32_t d_qk, int32_t d_v, Heads* h) {
  if (csa_status st = check_dims(what, H_kv, d_qk, d_v); st != CSA_OK) return st;
  CSA_REQUIRE(H >= 1 && H <= 65535 && H % H_kv == 0, "%s: query heads must be a multiple of the kv heads (H %d, H_kv %d)",
              what, H, H_kv);
  if (H / H_kv > 128) return fail(CSA_ERR_UNSUPPORTED, "%s: at most 128 query heads per kv head (got %d)", what, H / H_kv);
  h->Hkv = H_kv;
  h->G = H / H_kv;
  h->dqk = d_qk;
  h->dv = d_v;
  return CSA_OK;
}

inline csa_status check_scale(const char* what, float scale) {
  // far inside what keeps scale * log2(e) and 8 / scale finite
  CSA_REQUIRE(scale >= 0x1p-100f && scale <= 0x1p100f, "%s: scale must be in [2^-100, 2^100]", what);
  return CSA_OK;
}

inline csa_status check_batch(const char* what, const gqa_cache* cache, const gqa_batch* batch) {
  CSA_REQUIRE(cache != nullptr, "%s: cache is NULL", what);
  CSA_REQUIRE(batch != nullptr, "%s: batch is NULL", what);
  CSA_REQUIRE(batch->reserved == 0, "%s: batch->reserved must be 0", what);
  CSA_REQUIRE(batch->n_seqs >= 0 && batch->max_pages >= 0 && batch->max_q >= 0, "%s: negative sizes in batch", what);
  CSA_REQUIRE(batch->total_q >= 0 && batch->total_q < (int64_t(1) << 31), "%s: total_q must be in [0, 2^31)", what);
  CSA_REQUIRE(cache->page_size == 16 || cache->page_size == 32 || cache->page_size == 64 || cache->page_size == 128,
              "%s: page_size must be 16, 32, 64 or 128 (got %d)", what, cache->page_size);
  return check_dims(what, cache->n_kv_heads, cache->d_qk, cache->d_v);
}

inline csa_status check_paged(const char* what, const gqa_cache* cache, const gqa_batch* batch, int32_t H, Heads* h) {
  if (csa_status st = check_batch(what, cache, batch); st != CSA_OK) return st;
  return check_heads(what, H, cache->n_kv_heads, cache->d_qk, cache->d_v, h);
}

// The pool and the batch's arrays of a call that has work to do.
inline csa_status check_pool(const char* what, const gqa_cache* cache, const gqa_batch* batch, bool rows) {
  CSA_REQUIRE(cache->n_pages >= 1 &&
                  cache->n_pages < ((int64_t(1) << 31) - 128) / (static_cast<int64_t>(cache->n_kv_heads) * cache->page_size),
              "%s: n_pages must be at least 1, and n_pages * H_kv * page_size below 2^31 - 128", what);
  CSA_REQUIRE(batch->max_pages >= 1, "%s: max_pages must be at least 1", what);
  CSA_REQUIRE(static_cast<int64_t>(batch->max_pages) * cache->page_size < (int64_t(1) << 31) - 65536,
              "%s: max_pages * page_size must be below 2^31 - 65536", what);
  CSA_REQUIRE_PTR(cache->k);
  CSA_REQUIRE_PTR(cache->v);
  CSA_REQUIRE_PTR(batch->block_table);
  CSA_REQUIRE_PTR(batch->cache_len);
  if (rows) {
    CSA_REQUIRE(batch->max_q >= 1, "%s: max_q is 0 but there are rows", what);
    CSA_REQUIRE_PTR(batch->cu_q);
  }
  return CSA_OK;
}

inline int max_len(const gqa_cache* cache, const gqa_batch* batch) { return batch->max_pages * cache->page_size; }

inline csa_status encode(const char* what, CUtensorMap* map, int rank, const void* base, const cuuint64_t* dims,
                         const cuuint64_t* strides, const cuuint32_t* box) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (enc == nullptr) return fail(CSA_ERR_CUDA, "%s: cuTensorMapEncodeTiled unavailable", what);
  const cuuint32_t es[3] = {1u, 1u, 1u};
  memset(map, 0, sizeof(*map));
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, es,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(CSA_ERR_CUDA, "%s: tensor map encoding failed (%d)", what, static_cast<int>(r));
  return CSA_OK;
}

// [rows, heads, d]: boxes of box_rows tokens x box_heads heads x 64 channels.
inline csa_status map_tokens(const char* what, CUtensorMap* map, const void* base, int d, int heads, uint64_t rows,
                             int box_heads, int box_rows) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), rows};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(d) * 2 * heads};
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_rows)};
  return encode(what, map, 3, base, dims, strides, box);
}

// [rows, d]: boxes of box_rows rows x 64 channels.
inline csa_status map_rows(const char* what, CUtensorMap* map, const void* base, int d, uint64_t rows, int box_rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(d), rows};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(d) * 2};
  const cuuint32_t box[2] = {64u, static_cast<cuuint32_t>(box_rows)};
  return encode(what, map, 2, base, dims, strides, box);
}

}  // namespace gqa
}  // namespace csa
