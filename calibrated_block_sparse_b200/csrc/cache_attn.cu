// Attention of new tokens over a paged 8-bit cache (e4m3 values, one scale
// per page of 128 tokens and head):
//   o = softmax(scale * q (2^ek k8)^T) (2^ev v8),  lse = ln sum exp(scale * q k^T).
//
// The query rows that share a key head (its group of query heads, times the
// new tokens of a stream) are taken together, so a cached byte is read once
// for all of them, and the cache is split over CTAs along its length when
// there are few rows: each split leaves its running maximum, sum and
// unnormalised output in a workspace, and a second kernel joins them.
//
// K and V stay in fp16 as the matrix operands: every e4m3 value is an fp16
// value, so the conversion is exact. A row of Q is brought to fp16 by a power
// of two that puts its largest value into [1, 2) (rounding only what is below
// 2^-14 of it, by 2^-25 at most); that power, the page's key scale and the
// softmax scale multiply the fp32 score. P is rounded to fp16 (2^-12
// relative), and a page's P V is accumulated in fp32 from zero and joined to
// the output with the page's value scale, which may be any fp32 number.
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

// ------------------------------------------------------------------ few rows
constexpr int kFewRows = 16;   // rows of one mma tile
constexpr int kFewWarps = 4;   // each takes 32 of a page's 128 keys
constexpr int kFewThreads = 32 * kFewWarps;

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Makes the NaN bytes of a word zero; nonzero if there was one.
__device__ __forceinline__ uint32_t take_nan(uint32_t& w) {
  const uint32_t hit = e4m3_nan_bytes(w);
  w &= ~((hit >> 7) * 0xffu);
  return hit;
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Loads a lane's 2 x 16 channels of a query row and returns their largest magnitude.
__device__ __forceinline__ float load_q_row(const __nv_bfloat16* row, int t, float (&x)[32]) {
  float amax = 0.f;
#pragma unroll
  for (int l = 0; l < 2; ++l)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 v = *reinterpret_cast<const uint4*>(row + l * 64 + t * 16 + i * 8);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[l * 16 + i * 8 + 2 * j] = __uint_as_float(w[j] << 16);
        x[l * 16 + i * 8 + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    }
#pragma unroll
  for (int i = 0; i < 32; ++i) amax = fmaxf(amax, fabsf(x[i]));
  return amax;
}

// CTA: one split of one tile of 16 rows of one key head of one stream.
// Each warp takes 32 keys of every page with its own running softmax; the
// four are joined at the end. Fragments come straight from global memory: the
// order of the contracted channels, and of the output channels, is free as
// long as both operands agree, so it is chosen to make each lane's share 16
// consecutive bytes of a key row.
__global__ void __launch_bounds__(kFewThreads)
    cache_attn_few_kernel(const __grid_constant__ CacheAttnParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int split = blockIdx.x;
  const int head = blockIdx.y / p.tiles, tile = blockIdx.y % p.tiles;
  const int b = blockIdx.z;
  const Stream st = stream_of(p.tok_start, p.kv_len, b, p.n, p.table_stride);
  if (st.bad || st.n_new > p.max_new) {
    if (threadIdx.x == 0) record_error(p.status, CALIBATT_ERR_CSR);
    return;
  }
  const int rows = st.n_new * p.group;
  const int r0 = tile * kFewRows;
  if (r0 >= rows) return;

  // rows g and g + 8 of the tile: token r / group, query head head * group + r % group
  const __nv_bfloat16* qrow[2];
  int limit[2];
  float c[2];
  uint32_t qa[8][4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = min(r0 + g + 8 * i, rows - 1);
    const int tok = r / p.group, h = head * p.group + r % p.group;
    qrow[i] = p.q + (static_cast<int64_t>(h) * p.n + st.t0 + tok) * 128;
    limit[i] = r0 + g + 8 * i < rows ? visible(st.len - st.n_new + tok, st.len, p.unit) : 0;
    float x[32];
    float amax = load_q_row(qrow[i], t, x);
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const float shrink = row_shrink(amax);
    c[i] = p.scale_log2 / shrink;
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      // step ks: slots 2t, 2t+1 hold channels 4w, 4w+1 of the lane's sixteen, slots 2t+8, 2t+9 the next two
      const int at = (ks >> 2) * 16 + (ks & 3) * 4;
      qa[ks][i] = pack_half2(x[at] * shrink, x[at + 1] * shrink);
      qa[ks][2 + i] = pack_half2(x[at + 2] * shrink, x[at + 3] * shrink);
    }
  }
  int most = max(limit[0], limit[1]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  const int pages = (most + kPage - 1) / kPage;
  const int per = (pages + p.splits - 1) / p.splits;
  const int pg0 = split * per, pg1 = min(pages, pg0 + per);

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float acc[16][4];
#pragma unroll
  for (int j = 0; j < 16; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
  const int32_t* table = p.table + static_cast<int64_t>(b) * p.table_stride;

  for (int pg = pg0; pg < pg1; ++pg) {
    const int page = __ldg(table + pg);
    if (page < 0 || page >= p.n_pages) {
      if (lane == 0) record_error(p.status, CALIBATT_ERR_CSR);
      continue;
    }
    const int64_t at = static_cast<int64_t>(page) * p.heads_kv + head;
    const float ks = __ldg(p.k_scale + at), vs = __ldg(p.v_scale + at);
    const int key0 = pg * kPage + warp * 32;
    if (key0 >= st.len) continue;
    const uint8_t* kp = p.k8 + (at * kPage + warp * 32) * 128;
    const uint8_t* vp = p.v8 + (at * kPage + warp * 32) * 128;
    uint4 kw[4][2], vw[2][4];
#pragma unroll
    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) kw[nt][h] = ld_stream(kp + (nt * 8 + g) * 128 + h * 64 + t * 16);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        vw[s][i] = ld_stream(vp + (s * 16 + 2 * t + (i & 1) + (i >> 1) * 8) * 128 + g * 16);

    // S = Q K^T
    float s[4][4];
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t w = word_of(kw[nt][k >> 2], k & 3);
        mma_f16(s[nt], qa[k], e4m3x2_to_half2(w & 0xffffu), e4m3x2_to_half2(w >> 16));
      }
    }
    const bool whole = __all_sync(0xffffffffu, key0 + 32 <= limit[0] && key0 + 32 <= limit[1]);
    if (!whole) {
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (key0 + nt * 8 + 2 * t + (i & 1) >= limit[i >> 1]) s[nt][i] = -INFINITY;
      // slots that no token has reached may hold anything
#pragma unroll
      for (int st2 = 0; st2 < 2; ++st2)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (key0 + st2 * 16 + 2 * t + (i & 1) + (i >> 1) * 8 >= st.len) vw[st2][i] = make_uint4(0, 0, 0, 0);
      // a product takes every key for every row, and 0 * NaN is NaN: a NaN
      // value of a key that some rows do not see is taken out of the product
      // and put into the rows that see it
      uint32_t nan = 0;
#pragma unroll
      for (int st2 = 0; st2 < 2; ++st2)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          nan |= take_nan(vw[st2][i].x) | take_nan(vw[st2][i].y);
          nan |= take_nan(vw[st2][i].z) | take_nan(vw[st2][i].w);
        }
      if (__any_sync(0xffffffffu, nan != 0)) {
        for (int key = 0; key < 32 && key0 + key < st.len; ++key) {
          const uint8_t* row = vp + key * 128 + 32 * t;
#pragma unroll
          for (int j = 0; j < 16; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (key0 + key < limit[i >> 1] && (row[16 * (i & 1) + j] & 0x7f) == 0x7f) acc[j][i] = NAN;
        }
      }
    }
    // online softmax of the warp's 32 keys
    float alpha[2];
    uint32_t pa[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) mx = fmaxf(mx, fmaxf(s[nt][2 * i], s[nt][2 * i + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float ck = score_factor(c[i], ks);
      const float now = fmaxf(m[i], mx * ck);
      const float use = now == -INFINITY ? 0.f : now;
      alpha[i] = ex2_approx(m[i] - use);
      // relative to the page's own largest score first: scores of 2^24 and
      // more would leave the rounding of mx * ck in the exponent
      const float off = mx * ck - use;
      if (mx == -INFINITY) mx = 0.f;
      float sum = 0.f;
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        const float e0 = ex2_approx((s[nt][2 * i] - mx) * ck + off), e1 = ex2_approx((s[nt][2 * i + 1] - mx) * ck + off);
        sum += e0 + e1;
        pa[nt >> 1][(nt & 1) * 2 + i] = pack_half2(e0, e1);
      }
      l[i] = l[i] * alpha[i] + sum;
      m[i] = now;
    }
    // O = O * alpha + (P V) * vs, one group of 8 output channels at a time
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t pair[2][2][2][2];  // k16 step, operand half, pair of channels, packed fp16 of two keys
#pragma unroll
      for (int s2 = 0; s2 < 2; ++s2)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint32_t x = word_of(vw[s2][2 * hf], w), y = word_of(vw[s2][2 * hf + 1], w);
          const uint32_t lo = __byte_perm(x, y, 0x5140), hi = __byte_perm(x, y, 0x7362);
          pair[s2][hf][0][0] = e4m3x2_to_half2(lo & 0xffffu);
          pair[s2][hf][0][1] = e4m3x2_to_half2(lo >> 16);
          pair[s2][hf][1][0] = e4m3x2_to_half2(hi & 0xffffu);
          pair[s2][hf][1][1] = e4m3x2_to_half2(hi >> 16);
        }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s2 = 0; s2 < 2; ++s2) mma_f16(d, pa[s2], pair[s2][0][j >> 1][j & 1], pair[s2][1][j >> 1][j & 1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[w * 4 + j][i] = acc[w * 4 + j][i] * alpha[i >> 1] + d[i] * vs;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
  }

  // join the four warps: rows of 128 channels in shared memory (padded to
  // 132), lane t of a quad holds channels 32t .. 32t+31
  __shared__ float so[kFewWarps][kFewRows][132];
  __shared__ float sm[kFewWarps][kFewRows], sl[kFewWarps][kFewRows];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (t == 0) {
      sm[warp][g + 8 * i] = m[i];
      sl[warp][g + 8 * i] = l[i];
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int j = 0; j < 16; ++j) so[warp][g + 8 * i][32 * t + 16 * e + j] = acc[j][2 * i + e];
  }
  __syncthreads();
  for (int r = warp; r < kFewRows && r0 + r < rows; r += kFewWarps) {
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) mx = fmaxf(mx, sm[w][r]);
    const float use = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) {
      const float f = ex2_approx(sm[w][r] - use);
      const float4 x = *reinterpret_cast<const float4*>(&so[w][r][lane * 4]);
      sum += sl[w][r] * f;
      o.x += x.x * f;
      o.y += x.y * f;
      o.z += x.z * f;
      o.w += x.w * f;
    }
    const int row = r0 + r;
    const int64_t at = static_cast<int64_t>(head * p.group + row % p.group) * p.n + st.t0 + row / p.group;
    if (p.splits == 1) {
      const bool some = sum != 0.f;
      const float inv = some ? 1.f / sum : 0.f;
      uint2 w = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
      if (!some) w = make_uint2(0, 0);
      *reinterpret_cast<uint2*>(p.o + at * 128 + lane * 4) = w;
      if (p.lse && lane == 0) p.lse[at] = some ? (mx + log2f(sum)) * kLn2 : -INFINITY;
    } else {
      const int64_t pt = static_cast<int64_t>(split) * p.heads_q * p.n + at;
      if (sum != 0.f) *reinterpret_cast<float4*>(p.part_o + pt * 128 + lane * 4) = o;
      if (lane == 0) p.part_ml[pt] = make_float2(mx, sum);
    }
  }
}

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
  int tiles, splits;
};

// Which kernel, how many row tiles, and into how many splits a tile's pages
// are cut, from the host's bounds alone.
// Few rows: enough CTAs to fill the card twice, and at least 4 pages for a
// split to be worth its joining.
// Tiles: one CTA per SM, so the splits that give the shortest schedule: waves
// of CTAs times the pages of one (plus its start and end, about 3 pages' time),
// plus the joining's traffic (8 bytes per output value and split; a page takes
// a tile about 1.1 us).
CachePlan cache_plan(int batch, int heads_q, int heads_kv, int n, int max_new, int max_kv) {
  CachePlan c;
  const int64_t rows = static_cast<int64_t>(std::min(max_new, n)) * (heads_q / heads_kv);
  c.few = rows <= kFewRows;
  c.alternate = rows <= 128;
  const int tile = c.few ? kFewRows : c.alternate ? 128 : 256;
  c.tiles = static_cast<int>((rows + tile - 1) / tile);
  const int64_t units = static_cast<int64_t>(batch) * heads_kv * c.tiles;
  const int64_t pages = std::max<int64_t>(1, (static_cast<int64_t>(max_kv) + kPage - 1) / kPage);
  const int sms = sm_count();
  if (c.few) {
    int64_t s = (4ll * sms + units - 1) / std::max<int64_t>(units, 1);
    s = std::min(s, pages / 4);
    c.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(s, 128)));
    return c;
  }
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
  if (plan.few) {
    cache_attn_few_kernel<<<dim3(plan.splits, static_cast<unsigned>(y), batch), kFewThreads, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return CALIBATT_ERR_CUDA;
  } else {
    rc = launch_cache_attn_tiles(p, plan.alternate, stream);
    if (rc != CALIBATT_OK) return rc;
  }
  if (plan.splits > 1) {
    const unsigned gx = (std::min(max_new, n) + 3) / 4;
    cache_attn_join_kernel<<<dim3(gx, heads_q, batch), 128, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return CALIBATT_ERR_CUDA;
  }
  return CALIBATT_OK;
}

}  // extern "C"
