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
// This file holds the entry points, the plan and the tiles' join.
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
namespace {

// ------------------------------------------------------------------ joining the splits
// A warp per row: weights 2^(m_s - max m), then the weighted sum of the
// splits' outputs over the weighted sum of their sums.
__global__ void __launch_bounds__(128) cache_attn_join_kernel(const __grid_constant__ CacheAttnParams p) {
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.z;
  const Stream st = stream_of(p.tok_start, p.kv_len, b, p.n, p.table_stride);
  if (st.bad || st.n_new > p.max_new) return;
  const int tok = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (tok >= st.n_new) return;
  const int64_t at = static_cast<int64_t>(blockIdx.y) * p.n + st.t0 + tok;
  const int64_t step = static_cast<int64_t>(p.heads_q) * p.n;
  float mx = -INFINITY;
  for (int s = lane; s < p.splits; s += 32) mx = fmaxf(mx, p.part_ml[s * step + at].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float use = mx == -INFINITY ? 0.f : mx;
  float sum = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < p.splits; ++s) {
    const float2 ml = p.part_ml[s * step + at];
    if (ml.y == 0.f) continue;  // no key of the split is visible: its output was not written
    const float f = ex2_approx(ml.x - use);
    const float4 x = *reinterpret_cast<const float4*>(p.part_o + (s * step + at) * 128 + lane * 4);
    sum += ml.y * f;
    o.x += x.x * f;
    o.y += x.y * f;
    o.z += x.z * f;
    o.w += x.w * f;
  }
  const bool some = sum != 0.f;
  const float inv = some ? 1.f / sum : 0.f;
  uint2 w = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (!some) w = make_uint2(0, 0);
  *reinterpret_cast<uint2*>(p.o + at * 128 + lane * 4) = w;
  if (p.lse && lane == 0) p.lse[at] = some ? (mx + log2f(sum)) * kLn2 : -INFINITY;
}

// ------------------------------------------------------------------ plan
struct CachePlan {
  bool few, alternate;  // the kernel for up to 16 rows; tiles of 128 rows instead of 256
  int tiles, splits;    // of the tile kernel
  FewPlan fp;
};

// Which kernel, how many row tiles, and into how many splits a tile's pages
// are cut, from the host's bounds alone.
// Tiles: one CTA per SM, so the splits that give the shortest schedule: waves
// of CTAs times the pages of one (plus its start and end, about 3 pages' time),
// plus the joining's traffic (8 bytes per output value and split; a page takes
// a tile about 1.1 us).
CachePlan cache_plan(int batch, int heads_q, int heads_kv, int n, int max_new, int max_kv) {
  CachePlan c;
  const int64_t rows = static_cast<int64_t>(std::min(max_new, n)) * (heads_q / heads_kv);
  c.few = rows <= kFewRows;
  c.alternate = rows <= 128;
  const int64_t pages = std::max<int64_t>(1, (static_cast<int64_t>(max_kv) + kPage - 1) / kPage);
  const int sms = sm_count();
  if (c.few) {
    c.tiles = c.splits = 1;
    c.fp = few_plan(batch, heads_kv, static_cast<int>(rows), pages, sms);
    return c;
  }
  const int tile = c.alternate ? 128 : 256;
  c.tiles = static_cast<int>((rows + tile - 1) / tile);
  const int64_t units = static_cast<int64_t>(batch) * heads_kv * c.tiles;
  const double join = static_cast<double>(heads_q) * std::min<int64_t>(static_cast<int64_t>(batch) * max_new, n) *
                      1024.0 / 6.5e12 / 1.1e-6;
  double best = 0.0;
  c.splits = 1;
  for (int s = 1; s <= 64 && s <= pages; ++s) {
    const double waves = static_cast<double>((units * s + sms - 1) / sms);
    const double time = waves * ((pages + s - 1) / s + 3.0) + (s > 1 ? 4.0 + s * join : 0.0);
    if (s == 1 || time < best) {
      best = time;
      c.splits = s;
    }
  }
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

size_t workspace_bytes(const CachePlan& c, int heads_q, int n) {
  if (c.few) return few_workspace_bytes(c.fp);
  if (c.splits <= 1) return 0;
  return static_cast<size_t>(c.splits) * heads_q * n * (128 * sizeof(float) + sizeof(float2));
}

}  // namespace
}  // namespace calibatt

extern "C" {

size_t calibatt_cache_attn_workspace_size(int batch, int heads_q, int heads_kv, int n, int max_new, int max_kv) {
  using namespace calibatt;
  if (check_shape(batch, heads_q, heads_kv, n, max_new, max_kv) != CALIBATT_OK) return 0;
  if (batch == 0 || n == 0 || max_new == 0) return 0;
  return workspace_bytes(cache_plan(batch, heads_q, heads_kv, n, max_new, max_kv), heads_q, n);
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
  const size_t need = workspace_bytes(plan, heads_q, n);
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
  p.tiles = plan.tiles;
  p.splits = plan.splits;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.part_o = static_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + static_cast<int64_t>(plan.splits) * heads_q * n * 128);
  const int64_t y = static_cast<int64_t>(heads_kv) * plan.tiles;
  if (y > 65535) return CALIBATT_ERR_UNSUPPORTED;
  p.wait_limit_ns = wait_limit_ns();
  if (plan.few) return launch_cache_attn_few(p, plan.fp, ws, stream);
  rc = launch_cache_attn_tiles(p, plan.alternate, stream);
  if (rc != CALIBATT_OK) return rc;
  if (plan.splits > 1) {
    const unsigned gx = (std::min(max_new, n) + 3) / 4;
    cache_attn_join_kernel<<<dim3(gx, heads_q, batch), 128, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return CALIBATT_ERR_CUDA;
  }
  return CALIBATT_OK;
}

}  // extern "C"
