// Pieces shared by the kernels of the paged 8-bit cache: a stream's share of
// the packed tokens, and e4m3 conversions.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "calibatt.h"
#include "ptx.cuh"

namespace calibatt {

constexpr int kPage = 128;  // tokens per cache page
// Tokens of a stream: the kernels round a length up to whole pages and look a
// page ahead in 32 bits.
constexpr int kMaxTokens = INT32_MAX - 2 * kPage + 1;

// New tokens [t0, t0 + n_new) of stream b and the tokens its cache holds.
struct Stream {
  int t0, n_new, len;
  bool bad;  // the lists do not fit: nothing may be read through them
};

__device__ __forceinline__ Stream stream_of(const int32_t* tok_start, const int32_t* kv_len, int b, int n,
                                            int table_stride) {
  Stream s;
  s.t0 = __ldg(tok_start + b);
  const int t1 = __ldg(tok_start + b + 1);
  s.len = __ldg(kv_len + b);
  s.bad = s.t0 < 0 || t1 < s.t0 || t1 > n || s.len < 0 || s.len > kMaxTokens ||
          s.len > static_cast<int64_t>(table_stride) * kPage;
  s.n_new = t1 - s.t0;
  return s;
}

// 16 bytes that are read once.
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Bit 7 of every byte that holds a NaN.
__device__ __forceinline__ uint32_t e4m3_nan_bytes(uint32_t four) {
  return ((four & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// Makes the NaN bytes of a word zero; nonzero if there was one.
__device__ __forceinline__ uint32_t take_nan(uint32_t& w) {
  const uint32_t hit = e4m3_nan_bytes(w);
  w &= ~((hit >> 7) * 0xffu);
  return hit;
}

// Writes to shared memory become visible to TMA and the tensor core.
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 2D tiled load of one box into shared memory, completing on `bar`.
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y)
      : "memory");
}

// Two packed e4m3 values to packed fp16: exact, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}

__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two) {
  const uint32_t h = e4m3x2_to_half2(two);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// fp16 operands, fp32 accumulation (operand formats 0); V has its channels (N) contiguous.
constexpr uint32_t kIdescQK = (1u << 4) | (16u << 17) | (8u << 24);
constexpr uint32_t kIdescPVh = kIdescQK | (1u << 16);

__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// 16 e4m3 values as two 16-byte chunks j, j + 1 of fp16 of row r, with the
// 128-byte swizzle (chunk j is at j ^ (r & 7)).
__device__ __forceinline__ void store_half(uint32_t row_addr, int r, int j, const uint4& w) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[2 * i] = e4m3x2_to_half2(x[i] & 0xffffu);
    h[2 * i + 1] = e4m3x2_to_half2(x[i] >> 16);
  }
  st_shared16(row_addr + ((j ^ (r & 7)) << 4), h[0], h[1], h[2], h[3]);
  st_shared16(row_addr + (((j + 1) ^ (r & 7)) << 4), h[4], h[5], h[6], h[7]);
}

// One row's power of two: 2^(to - x) for a largest magnitude in [2^x, 2^(x+1)).
__device__ __forceinline__ float row_shrink(float amax, int to) {
  const int x = (__float_as_int(amax) >> 23) - 127;  // amax >= 0; NaN and inf: 128
  return x >= 128 ? 1.f : __int_as_float((min(max(to - x, -126), 126) + 127) << 23);
}

// Factor of a raw score, never 0 (a masked score is -inf, and -inf * 0 is NaN).
__device__ __forceinline__ float score_factor(float row, float key_scale) {
  const float f = row * key_scale;
  return f == 0.f ? 1.17549435e-38f : f;
}

// Units of an output that is summed over pages with different value scales
// (one state for all rows): it is kept as O / (2^-kLog * ref). A page whose
// scale is 2^kLow .. 2 of the reference multiplies P by 2^kLog times the
// ratio, in the exponent, at no cost; outside that range the reference moves
// and O is multiplied by what page() returns. kLog leaves P room above 1 for a
// running maximum that is up to kStale (a power of two) behind; kLow keeps
// weights down to 2^-24 of the largest. The reference is never more than 2^-70
// below the largest scale met: O, at most 2^55 in units of that
// (2^15 * 448 * 2^31 keys), stays finite.
template <int kLog, int kLow>
struct VRef {
  float ref = 0.f, top = 0.f, ref_inv = 0.f;
  float vs = 0.f, log = 0.f, inv = 0.f;  // the page's: its scale, P's factor as a log2, 1 / that factor

  static constexpr float kUnit = 1.f / (1 << kLog);
  // Scales change from page to page, so this is kept to a few instructions:
  // the approximate logarithm and reciprocal are exact for powers of two, and
  // within 2^-22 for others.
  __device__ __forceinline__ float page(float scale) {
    vs = scale == 0.f ? 1.17549435e-38f : scale;
    float ratio = 1.f;
    if (ref == 0.f) {
      ref = top = vs;
      ref_inv = 1.f / ref;
    } else if (vs > 2.f * ref || vs * (1 << -kLow) < ref) {
      top = fmaxf(top, vs);
      const float now = fmaxf(vs, top * 8.470329472543003e-22f);
      ratio = ref / now;
      ref = now;
      ref_inv = 1.f / ref;
    }
    // At 2^-40 P, 2^14 times that at most (kLog and a stale maximum), rounds to
    // zero already: under half of fp16's smallest value. Further down it would
    // stay so, but f and its reciprocal would leave fp32's range and make the
    // sum of the weights NaN.
    const float f = fmaxf(vs * ref_inv, 9.094947017729282e-13f);
    float l2, r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(l2) : "f"(f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(f));
    log = l2 + kLog;
    inv = kUnit * r;
    return ratio;
  }
  // Outputs leave the units of the reference before they are divided by their
  // weights' sum, and a sum of values next to the largest leaves fp32's range
  // although their mean is inside it. From a reference of 1 on, outputs and sums
  // are therefore kept times 2^-40 (2^31 keys with weights up to 2^8, twice)
  // and the maximum is 40 more: the same row in other units.
  __device__ __forceinline__ float damp() const { return ref > 1.f ? 9.094947017729282e-13f : 1.f; }
  __device__ __forceinline__ float raise() const { return ref > 1.f ? 40.f : 0.f; }
  __device__ __forceinline__ float unit() const { return ref * kUnit * damp(); }
};

// Tile t of the ring's order -> (V?, page of the range): K0 V0 K1 V1 ..., or
// with the next page's K before a page's V: K0 K1 V0 K2 V1 ...
template <bool kAhead>
__device__ __forceinline__ void ring_tile(int t, int np, bool& is_v, int& page) {
  if (!kAhead) {
    is_v = t & 1;
    page = t >> 1;
  } else if (t & 1) {
    page = (t + 1) >> 1;
    is_v = page >= np;
    if (is_v) page = (t - 1) >> 1;
  } else {
    is_v = t > 0;
    page = t > 0 ? (t >> 1) - 1 : 0;
  }
}

struct CacheAttnParams {
  const __nv_bfloat16* q;  // [heads_q][n][128]
  __nv_bfloat16* o;
  float* lse;              // [heads_q][n] or NULL
  const int32_t* tok_start;
  const int32_t* kv_len;
  const int32_t* table;
  const uint8_t* k8;
  const uint8_t* v8;
  const float* k_scale;
  const float* v_scale;
  int heads_q, heads_kv, group, n, batch, max_new, table_stride, n_pages, unit;
  int max_rows;            // of a stream and key head that the kernel is laid out for
  float scale_log2;
  int* status;
  uint64_t wait_limit_ns;
};

// Keys that the token at position pos sees (pos may be negative).
__device__ __forceinline__ int visible(int pos, int len, int unit) {
  if (unit == 0) return len;
  const int u = pos >= 0 ? pos / unit : -((unit - 1 - pos) / unit);
  const int64_t end = (static_cast<int64_t>(u) + 1) * unit;
  return static_cast<int>(end < 0 ? 0 : end > len ? len : end);
}

// Page numbers of 32 consecutive pages of a stream, one per lane, fetched a
// chunk of 32 ahead; kScales: with their key and value scales. A page outside
// the pool is reported and gets id -1, and so does one behind the last token.
template <bool kScales>
struct PageWindow {
  const CacheAttnParams& p;
  const int32_t* table;
  int head, count;
  int id = -1, id_next = -1;
  float ks = 1.f, vs = 1.f, ks_next = 1.f, vs_next = 1.f;

  // `pages` pages of stream b from its page pg on
  __device__ __forceinline__ PageWindow(const CacheAttnParams& params, int b, int key_head, int pg, int pages, int len)
      : p(params), table(params.table + static_cast<int64_t>(b) * params.table_stride + pg), head(key_head) {
    count = min(pages, (len + kPage - 1) / kPage - pg);
  }
  __device__ __forceinline__ void fetch(int at, int* status) {
    id_next = -1;
    ks_next = vs_next = 1.f;
    if (at < count) {
      id_next = __ldg(table + at);
      if (id_next < 0 || id_next >= p.n_pages) {
        record_error(status, CALIBATT_ERR_CSR);
        id_next = -1;
      } else if (kScales) {
        const int64_t i = static_cast<int64_t>(id_next) * p.heads_kv + head;
        ks_next = __ldg(p.k_scale + i);
        vs_next = __ldg(p.v_scale + i);
      }
    }
  }
  // call before using page i = 0, 32, 64, ...
  __device__ __forceinline__ void advance(int i, int lane, int* status) {
    id = id_next;
    ks = ks_next;
    vs = vs_next;
    fetch(i + 32 + lane, status);
  }
};

// Normalises and stores a row's four channels of a lane; no key seen: 0 and -inf.
__device__ __forceinline__ void store_row(const CacheAttnParams& p, int64_t at, int lane, float mx, float sum,
                                          const float4& o) {
  const bool some = sum != 0.f;
  const float inv = some ? 1.f / sum : 0.f;
  uint2 w = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (!some) w = make_uint2(0, 0);
  *reinterpret_cast<uint2*>(p.o + at * 128 + lane * 4) = w;
  if (p.lse && lane == 0) p.lse[at] = some ? (mx + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

// Joins one row's partial results (a warp): those of parts c0 .. c1 - 1 for
// which `slot` gives an address, each [rows][128] outputs, then maximum (log2
// units) and sum per row. The lanes fetch 32 parts' maxima and sums at a time;
// the outputs are then loaded independently of each other.
template <class Slot>
__device__ __forceinline__ void join_row(const CacheAttnParams& p, int64_t at, int lane, int c0, int c1,
                                         const Slot& slot, int64_t row, int64_t rows) {
  float mx = -INFINITY, sum = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int base = c0; base < c1; base += 32) {
    const float* mine = base + lane < c1 ? slot(base + lane) : nullptr;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (mine) ml = *reinterpret_cast<const float2*>(mine + rows * 128 + 2 * row);
    float top = ml.x;
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
    const float now = fmaxf(mx, top), use = now == -INFINITY ? 0.f : now;
    const float keep = ex2_approx(mx - use), w = ex2_approx(ml.x - use);
    mx = now;
    float add = ml.y * w;
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) add += __shfl_xor_sync(0xffffffffu, add, i);
    sum = sum * keep + add;
    o.x *= keep;
    o.y *= keep;
    o.z *= keep;
    o.w *= keep;
    unsigned have = __ballot_sync(0xffffffffu, mine != nullptr);
    while (have) {
      constexpr int kBatch = 4;
      float4 x[kBatch];
      float f[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int l = have ? __ffs(have) - 1 : 0;
        const float* src =
            reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), l));
        f[i] = __shfl_sync(0xffffffffu, w, l);
        x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (have)
          x[i] = *reinterpret_cast<const float4*>(src + row * 128 + lane * 4);
        else
          f[i] = 0.f;
        have &= have - 1;
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        o.x += x[i].x * f[i];
        o.y += x[i].y * f[i];
        o.z += x[i].z * f[i];
        o.w += x[i].w * f[i];
      }
    }
  }
  store_row(p, at, lane, mx, sum, o);
}

// 128-byte rows of a pool's pages, boxes of one page with the 128-byte swizzle.
int make_page_map(CUtensorMap* map, const void* pool, const CacheAttnParams& p);

// Up to 16, up to 128 and more query rows that share a key head.
constexpr int kFewRows = 16, kMidRows = 128, kTileRows = 256;

// Few and mid rows: the streams' pages, key head by key head, cut into equal
// shares for `ctas` CTAs; or, with `whole`, a CTA for each key head of each
// stream, and nothing to join.
struct SharePlan {
  bool whole;
  int ctas;
  int rows;  // the most that a key head has
};
int launch_cache_attn_few(const CacheAttnParams& p, const SharePlan& plan, void* ws, cudaStream_t stream);
int launch_cache_attn_mid(const CacheAttnParams& p, const SharePlan& plan, void* ws, cudaStream_t stream);
// Joins their partial results, for kernels laid out for `cap` rows.
int launch_cache_join(const CacheAttnParams& p, const SharePlan& plan, const float* part, int cap,
                      cudaStream_t stream);

// More rows: tiles of 256 of them; those behind the first `whole` are split over
// the keys and joined.
struct TilePlan {
  int tiles;  // of a stream and key head, at most
  int chunk;  // (stream, key head) pairs whose tiles are taken together
  int units;  // tiles of all pairs
  int whole;
  int splits;
};
int launch_cache_attn_tiles(const CacheAttnParams& p, const TilePlan& plan, void* ws, cudaStream_t stream);

}  // namespace calibatt
