// Attention of new tokens over a paged 8-bit cache (e4m3 values, one scale
// per page of 128 tokens and head):
//   o = softmax(scale * q (2^ek k8)^T) (2^ev v8),  lse = ln sum exp(scale * q k^T).
//
// The query rows that share a key head (its group of query heads, times the
// new tokens of a stream) are taken together, so a cached byte is read once
// for all of them: up to 16 rows by cache_few.cu, bound by the cache's bytes,
// up to 128 by cache_mid.cu, more by cache_tile.cu, bound by the tensor core
// and the softmax beside it. All split the cache over CTAs along its length; a
// part leaves its running maximum, sum and unnormalised output in a workspace,
// and a second kernel joins them. This file holds the entry points, the plan
// and the join.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "cache.cuh"
#include "cache_list.cuh"
#include "calibatt.h"
#include "kernels.h"
#include "ptx.cuh"
#include "sched.cuh"

namespace calibatt {
namespace {

// Joins the stretches of one (stream, key head): those of the CTAs whose
// shares meet its pages. A warp per row, 8 rows per CTA.
constexpr int kJoinRows = 8;
__global__ void __launch_bounds__(32 * kJoinRows)
    cache_join_kernel(const __grid_constant__ CacheAttnParams p, int ctas, const float* part, int cap) {
  const int lane = threadIdx.x & 31, row = blockIdx.z * kJoinRows + (threadIdx.x >> 5);
  const int head = blockIdx.x, b = blockIdx.y;
  const Stream st = stream_of(p.tok_start, p.kv_len, b, p.n, p.table_stride);
  const int pages = stream_pages(p, st);
  int64_t before = 0, total = 0;
  if (pages > 0) {
    for (int i = lane; i < p.batch; i += 32) {
      const int64_t x = stream_pages(p, stream_of(p.tok_start, p.kv_len, i, p.n, p.table_stride));
      total += x;
      if (i < b) before += x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      total += __shfl_xor_sync(0xffffffffu, total, o);
      before += __shfl_xor_sync(0xffffffffu, before, o);
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (pages == 0 || row >= st.n_new * p.group) return;
  total *= p.heads_kv;
  const int64_t u0 = before * p.heads_kv + static_cast<int64_t>(head) * pages, u1 = u0 + pages;
  // the last CTA whose share begins at or before u0
  int c = static_cast<int>(u0 * ctas / total);
  while (c + 1 < ctas && share_begin(total, c + 1, ctas) <= u0) ++c;
  while (c > 0 && share_begin(total, c, ctas) > u0) --c;
  if (share_begin(total, c + 1, ctas) >= u1) return;  // one CTA had all of them and wrote the result
  const int last = static_cast<int>(min(static_cast<int64_t>(ctas), (u1 * ctas + total - 1) / total + 1));
  join_row(
      p, static_cast<int64_t>(head * p.group + row % p.group) * p.n + st.t0 + row / p.group, lane, c, last,
      [&](int i) -> const float* {
        const int64_t w0 = share_begin(total, i, ctas);
        if (w0 >= u1 || w0 == share_begin(total, i + 1, ctas)) return nullptr;  // behind, or an empty share
        return part_of(const_cast<float*>(part), i, w0 > u0, cap);
      },
      row, cap);
}

}  // namespace

int launch_cache_join(const CacheAttnParams& p, const SharePlan& plan, const float* part, int cap,
                      cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.heads_kv, p.batch, (plan.rows + kJoinRows - 1) / kJoinRows);
  cfg.blockDim = dim3(32 * kJoinRows);
  cfg.stream = stream;
  // it may be resident while the pages are still read: it waits in the kernel
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_join_kernel, p, plan.ctas, part, cap) == cudaSuccess ? CALIBATT_OK
                                                                                             : CALIBATT_ERR_CUDA;
}

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
  int rows;  // the most that share a key head, in one stream
  SharePlan share;
  TilePlan tile;
  bool fits = true;  // the grid's limits
};

// Shares for `slots` CTAs that run at the same time. Up to 5 pages the join
// costs more than the split saves, and up to 8 if there are several streams,
// whose shares begin and end inside others' (measured whole and split: 40 heads
// of one stream, a row each, 5 pages 10.0 and 11.5 us, 8 pages 13.1 and 12.0;
// 16 streams of 8 heads, 5 pages 10.0 and 15.3 us, 8 pages 13.7 and 16.4; 4
// streams of 8 heads with 5 rows each, 8 pages 15.6 and 17.5, 12 pages 19.7 and
// 17.8). Where the streams' key heads fit a whole
// number of times, their pages are cut alike and no share crosses from one to
// the next, which costs about 4 pages' time (its start and end once more);
// ragged streams cross anyway. A share has at least two pages.
bool share_plan(SharePlan& f, int batch, int heads_kv, int rows, int64_t pages, int slots) {
  const int64_t units = static_cast<int64_t>(batch) * heads_kv;
  f.rows = rows;
  f.whole = pages <= (batch > 1 ? 8 : 5);
  int64_t ctas = units;
  if (!f.whole) {
    ctas = slots;
    if (units <= slots) {
      const int64_t each = slots / units;
      if ((pages + each - 1) / each <= (pages * units + slots - 1) / slots + 4) ctas = units * each;
    }
    ctas = std::min<int64_t>(ctas, units * ((pages + 1) / 2));
  }
  f.ctas = static_cast<int>(std::min<int64_t>(ctas, INT_MAX));
  return ctas <= INT_MAX;
}

// One CTA per SM. Full waves of tiles are taken whole; the tiles behind them
// are split so that the schedule is shortest, in a tile's time for a page
// (about 2 us): rounds of CTAs times the pages of one (plus its start and end,
// about 3), the joining's launch and its traffic. A pair's last tile, if it has
// up to 128 rows, takes about 0.75 of a tile's time and fills gaps. All SMs at
// work at the same time run into the power limit, so a schedule without gaps is
// no shorter than 1 / 0.88 of the work: splitting 92 of the 240 full tiles of a
// 480p frame to fill its second wave was slower (1095 -> 1140 us), splitting the
// 12 behind a wave faster (40 heads, 1024 rows, 20000 keys: 639 -> 427 us).
bool tile_plan(TilePlan& t, int batch, int heads_kv, int64_t rows, int64_t pages, int sms) {
  const int64_t tiles = (rows + kTileRows - 1) / kTileRows, pairs = static_cast<int64_t>(batch) * heads_kv;
  if (pairs > INT_MAX / 2 / tiles) return false;
  t.tiles = static_cast<int>(tiles);
  // two waves of tiles: the pages of a pair are read from memory about twice
  t.chunk = static_cast<int>(std::min(pairs, (2 * sms + tiles - 1) / tiles));
  const int64_t units = pairs * tiles, whole = units / sms * sms;
  t.units = static_cast<int>(units);
  t.whole = t.units;
  t.splits = 1;
  const int64_t rest = units - whole;
  if (rest == 0) return true;
  const bool odd = rows % kTileRows > 0 && rows % kTileRows <= kTileRows / 2;
  const int64_t small = odd ? std::min(rest, pairs) : 0;
  const double page = 2e-6;
  const double join = 2.0 * kTileRows * 520 / 6.5e12 / page * static_cast<double>(rest);
  const double waves = static_cast<double>(whole / sms);
  const double least = (static_cast<double>(units) - (odd ? 0.5 * static_cast<double>(pairs) : 0.0)) / sms / 0.88 *
                       static_cast<double>(pages);
  double best = 0.0;
  for (int s = 1; s <= 64 && s <= pages; ++s) {
    // whole tiles' parts, then the last tiles' into the gaps
    const int64_t full = (rest - small) * s, over = full % sms, gaps = sms - over, m = small * s;
    double last = over > 0 ? 1.0 : 0.0;
    if (m > 0)
      last = std::max(last, m <= gaps              ? 0.75
                            : m <= 2 * gaps        ? 1.5
                            : m <= 2 * gaps + over ? 1.75
                                                   : 2.5);
    const double rounds = static_cast<double>(full / sms) + last;
    const double each = static_cast<double>((pages + s - 1) / s) + 3.0;
    const double time = std::max(least, waves * static_cast<double>(pages + 3) + rounds * each) +
                        (s > 1 ? 2.5 + s * join : 0.0);
    if (s == 1 || time < best) {
      best = s == 1 ? 0.95 * time : time;  // a split is worth its join if it saves 5 %
      t.splits = s;
    }
  }
  if (t.splits > 1) t.whole = static_cast<int>(whole);
  return true;
}

CachePlan cache_plan(int batch, int heads_q, int heads_kv, int n, int max_new, int max_kv) {
  CachePlan c{};
  const int64_t rows = static_cast<int64_t>(std::min(max_new, n)) * (heads_q / heads_kv);
  const int64_t pages = std::max<int64_t>(1, (static_cast<int64_t>(max_kv) + kPage - 1) / kPage);
  const int sms = sm_count();
  c.rows = static_cast<int>(rows);
  if (rows <= kMidRows)
    c.fits = share_plan(c.share, batch, heads_kv, c.rows, pages, rows <= kFewRows ? 2 * sms : sms);
  else
    c.fits = tile_plan(c.tile, batch, heads_kv, rows, pages, sms);
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

// Memory that a call reads or writes.
struct Span {
  const void* at;
  size_t bytes;
};
bool meet(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  return a.at && b.at && x < y + b.bytes && y < x + a.bytes;
}

size_t workspace_bytes(const CachePlan& c) {
  if (c.rows <= kMidRows) {
    if (c.share.whole) return 0;
    const int cap = c.rows <= kFewRows ? kFewRows : kMidRows;
    return 2 * static_cast<size_t>(c.share.ctas) * part_floats(cap) * sizeof(float);
  }
  return static_cast<size_t>(c.tile.units - c.tile.whole) * c.tile.splits * part_floats(kTileRows) * sizeof(float);
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
  CachePlan plan = cache_plan(batch, heads_q, heads_kv, n, max_new, max_kv);
  if (!plan.fits) return CALIBATT_ERR_UNSUPPORTED;
  const size_t need = workspace_bytes(plan);
  if (need > 0 && (!ws || ws_bytes < need)) return CALIBATT_ERR_ARG;
  // a stream's parts are written while other CTAs still read
  const size_t rows = static_cast<size_t>(heads_q) * n, pages = static_cast<size_t>(n_pages) * heads_kv;
  const Span written[] = {{o, rows * 256}, {lse, rows * 4}, {need > 0 ? ws : nullptr, need}};
  const Span read[] = {{q, rows * 256}, {k8, pages * kPage * 128}, {v8, pages * kPage * 128},
                       {k_scale, pages * 4}, {v_scale, pages * 4}};
  for (int i = 0; i < 3; ++i) {
    for (const Span& r : read)
      if (meet(written[i], r)) return CALIBATT_ERR_ARG;
    for (int j = 0; j < i; ++j)
      if (meet(written[i], written[j])) return CALIBATT_ERR_ARG;
  }
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
  p.max_rows = plan.rows <= kFewRows   ? kFewRows
               : plan.rows <= 32       ? 32
               : plan.rows <= 64       ? 64
               : plan.rows <= kMidRows ? kMidRows
                                       : INT_MAX;
  if (plan.rows <= kFewRows) return launch_cache_attn_few(p, plan.share, ws, stream);
  if (plan.rows <= kMidRows) return launch_cache_attn_mid(p, plan.share, ws, stream);
  // under a causal mask over mostly new tokens the last tiles are short as they are
  if (causal_unit > 0 && plan.tile.whole > 0 && max_new > max_kv / 2) plan.tile.whole = plan.tile.units;
  return launch_cache_attn_tiles(p, plan.tile, ws, stream);
}

}  // extern "C"
