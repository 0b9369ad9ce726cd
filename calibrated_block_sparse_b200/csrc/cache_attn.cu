// Attention of new tokens over a paged 8-bit cache (e4m3 values, one scale
// per page of 128 tokens and head):
//   o = softmax(scale * q (2^ek k8)^T) (2^ev v8),  lse = ln sum exp(scale * q k^T).
//
// The query rows that share a key head (its group of query heads, times the
// new tokens of a stream) are taken together, so a cached byte is read once
// for all of them: up to 16 rows by cache_few.cu, bound by the cache's bytes,
// more by cache_tile.cu, bound by the tensor core. Both split the cache over
// CTAs along its length; a split leaves its running maximum, sum and
// unnormalised output in a workspace, and a second kernel joins them.
// This file holds the entry points and the plan.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "cache.cuh"
#include "calibatt.h"
#include "kernels.h"
#include "ptx.cuh"
#include "sched.cuh"

namespace calibatt {

int make_page_map(CUtensorMap* map, const void* pool, const CacheAttnParams& p) {
  EncodeTiledFn enc = get_encode();
  if (!enc) return CALIBATT_ERR_CUDA;
  int64_t rows = static_cast<int64_t>(p.n_pages) * p.heads_kv * kPage;
  if (rows > INT32_MAX) return CALIBATT_ERR_UNSUPPORTED;
  if (rows == 0) {  // an empty pool is never read: the map needs an address all the same
    pool = p.q;
    rows = kPage;
  }
  cuuint64_t dims[2] = {128, static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {128};
  cuuint32_t box[2] = {128, kPage};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(pool), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? CALIBATT_OK : CALIBATT_ERR_CUDA;
}

namespace {

// ------------------------------------------------------------------ plan
// Which kernel, and how its work is shared out, from the host's bounds alone.
struct CachePlan {
  bool few;
  FewPlan fp;
  TilePlan tp;
};

CachePlan cache_plan(int batch, int heads_q, int heads_kv, int n, int max_new, int max_kv) {
  CachePlan c{};
  const int64_t rows = static_cast<int64_t>(std::min(max_new, n)) * (heads_q / heads_kv);
  const int64_t pages = std::max<int64_t>(1, (static_cast<int64_t>(max_kv) + kPage - 1) / kPage);
  c.few = rows <= kFewRows;
  if (c.few)
    c.fp = few_plan(batch, heads_kv, static_cast<int>(rows), pages, sm_count());
  else
    c.tp = tile_plan(batch, heads_kv, rows, pages, sm_count());
  return c;
}

int check_shape(int batch, int heads_q, int heads_kv, int n, int max_new, int max_kv) {
  if (batch < 0 || heads_q < 1 || heads_kv < 1 || heads_q % heads_kv || n < 0 || max_new < 0 || max_kv < 0)
    return CALIBATT_ERR_ARG;
  const int64_t group = heads_q / heads_kv;
  // row numbers of a stream fit 32 bits, the grid's dimensions their limits
  if (std::min(max_new, n) * group > INT_MAX / 2 || batch > 65535 || heads_q > 65535) return CALIBATT_ERR_UNSUPPORTED;
  return CALIBATT_OK;
}

size_t workspace_bytes(const CachePlan& c) {
  return c.few ? few_workspace_bytes(c.fp) : tile_workspace_bytes(c.tp);
}

}  // namespace
}  // namespace calibatt

extern "C" {

size_t calibatt_cache_attn_workspace_size(int batch, int heads_q, int heads_kv, int n, int max_new, int max_kv) {
  using namespace calibatt;
  if (check_shape(batch, heads_q, heads_kv, n, max_new, max_kv) != CALIBATT_OK) return 0;
  if (batch == 0 || n == 0 || max_new == 0) return 0;
  return workspace_bytes(cache_plan(batch, heads_q, heads_kv, n, max_new, max_kv));
}

int calibatt_cache_attn_fwd(const calibatt_bf16* q, int heads_q, int heads_kv, int n, int d, float scale,
                            int causal_unit, const int32_t* tok_start, const int32_t* kv_len, int batch, int max_new,
                            int max_kv, const int32_t* table, int table_stride, int n_pages, const uint8_t* k8,
                            const uint8_t* v8, const float* k_scale, const float* v_scale, calibatt_bf16* o,
                            float* lse, void* ws, size_t ws_bytes, calibatt_stream_t stream_) {
  using namespace calibatt;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (d != CALIBATT_HEAD_DIM) return CALIBATT_ERR_UNSUPPORTED;
  int rc = check_shape(batch, heads_q, heads_kv, n, max_new, max_kv);
  if (rc != CALIBATT_OK) return rc;
  if (causal_unit < 0 || !(std::isfinite(scale) && scale > 0.f) || table_stride < 0 || n_pages < 0)
    return CALIBATT_ERR_ARG;
  if (batch == 0 || n == 0 || max_new == 0) return CALIBATT_OK;
  if (!q || !o || !tok_start || !kv_len || (table_stride > 0 && !table) ||
      (n_pages > 0 && (!k8 || !v8 || !k_scale || !v_scale)))
    return CALIBATT_ERR_ARG;
  for (const void* x : {static_cast<const void*>(q), static_cast<const void*>(o), static_cast<const void*>(k8),
                        static_cast<const void*>(v8), static_cast<const void*>(ws)})
    if (reinterpret_cast<uintptr_t>(x) & 15u) return CALIBATT_ERR_ALIGN;
  for (const void* x : {static_cast<const void*>(tok_start), static_cast<const void*>(kv_len),
                        static_cast<const void*>(table), static_cast<const void*>(k_scale),
                        static_cast<const void*>(v_scale), static_cast<const void*>(lse)})
    if (reinterpret_cast<uintptr_t>(x) & 3u) return CALIBATT_ERR_ALIGN;
  const CachePlan plan = cache_plan(batch, heads_q, heads_kv, n, max_new, max_kv);
  const size_t need = workspace_bytes(plan);
  if (need > 0 && (!ws || ws_bytes < need)) return CALIBATT_ERR_ARG;
  CacheAttnParams p{};
  p.status = status_word();
  if (!p.status) return CALIBATT_ERR_CUDA;
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.o = reinterpret_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.tok_start = tok_start;
  p.kv_len = kv_len;
  p.table = table;
  p.k8 = k8;
  p.v8 = v8;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.heads_q = heads_q;
  p.heads_kv = heads_kv;
  p.group = heads_q / heads_kv;
  p.n = n;
  p.batch = batch;
  p.max_new = max_new;
  p.table_stride = table_stride;
  p.n_pages = n_pages;
  p.unit = causal_unit;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.wait_limit_ns = wait_limit_ns();
  return plan.few ? launch_cache_attn_few(p, plan.fp, ws, stream) : launch_cache_attn_tiles(p, plan.tp, ws, stream);
}

}  // extern "C"
