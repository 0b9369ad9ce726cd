// Writing keys and values into a paged 8-bit cache: pages of 128 tokens, e4m3
// values, one scale per page and head.
//
//   x = q * 2^e,  q = round_e4m3(x / 2^e),
//   e = the least integer with max|x| <= 448 * 2^e over the page's tokens.
// A power of two as the scale makes x / 2^e and q * 2^e exact, so a value is
// rounded once (to e4m3's 4 significant bits), and costs no accuracy: e4m3 is
// a floating format whose relative step does not depend on the scale. It also
// lets a page that is written in several calls take a larger exponent later:
// the entries it holds are re-encoded with q / 2^(e' - e), which is exact
// down to e4m3's subnormals (they round once more).
//
// Bound by memory: 2 bytes read and 1 written per value. One CTA takes the
// new tokens of one page and head (of K or of V): every value is held in
// registers between the maximum and the rounding, so it is read once.
// Measured on B200: 4 x 10800 tokens of 40 heads (1.03 GB) in 159 us, the rate
// of a plain copy (161 with four CTAs per SM instead of five, 179 with 512
// threads per CTA); one 480p frame (1560 tokens, 48 MB) in 9.7 us, of which 7.4
// are its bytes and the rest the launch and one CTA's chain of load, maximum,
// rounding and store.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "cache.cuh"
#include "calibatt.h"
#include "kernels.h"
#include "ptx.cuh"

namespace calibatt {
namespace {

constexpr int kWriteThreads = 256;
constexpr int kRowsPerPass = kWriteThreads / 16;    // 16 threads hold a row of 128 channels
constexpr int kPasses = kPage / kRowsPerPass;       // 8 channels of 8 rows per thread
constexpr int kMinExp = -117;  // 2^-9 * 2^-117, the smallest value a page stands for, is still normal in fp32

struct WriteParams {
  const __nv_bfloat16* x[2];  // keys, values
  int64_t ts[2], hs[2];
  uint8_t* c[2];
  float* scale[2];
  const int32_t* tok_start;
  const int32_t* kv_len;
  const int32_t* table;
  int heads, n, batch, max_new, table_stride, n_pages;
  int* status;
};

// Two fp32 values to packed e4m3, round to nearest even. With kFinite false
// what is not finite becomes NaN (the conversion alone would turn an infinity
// into 448).
template <bool kFinite>
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  if (!kFinite) {
    lo = fabsf(lo) <= 3.4028235e38f ? lo : __int_as_float(0x7fffffff);
    hi = fabsf(hi) <= 3.4028235e38f ? hi : __int_as_float(0x7fffffff);
  }
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

template <bool kFinite>
__device__ __forceinline__ uint2 to_e4m3x8(const uint4& v, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    q[j] = to_e4m3x2<kFinite>(__uint_as_float(w[j] << 16) * inv, __uint_as_float(w[j] & 0xffff0000u) * inv);
  return make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
}

// The least exponent e >= kMinExp with a <= 448 * 2^e (a >= 0, finite).
__device__ __forceinline__ int page_exponent(float a) {
  const int bits = __float_as_int(a);
  // a = 1.m * 2^x: 448 * 2^e = 1.75 * 2^(e + 8)
  const int e = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000);
  return max(e, kMinExp);
}

__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }

__global__ void __launch_bounds__(kWriteThreads, 5) cache_write_kernel(const __grid_constant__ WriteParams p) {
  const int which = blockIdx.x & 1, head = blockIdx.x >> 1;
  const int b = blockIdx.z;
  const Stream st = stream_of(p.tok_start, p.kv_len, b, p.n, p.table_stride);
  if (st.bad || st.n_new > p.max_new || st.len < st.n_new) {
    if (threadIdx.x == 0) record_error(p.status, CALIBATT_ERR_CSR);
    return;
  }
  if (st.n_new == 0) return;
  const int begin = st.len - st.n_new;  // position of the first new token
  const int pg = begin / kPage + static_cast<int>(blockIdx.y);
  if (static_cast<int64_t>(pg) * kPage >= st.len) return;  // pages that max_new allows for may pass 32 bits
  const int page = __ldg(p.table + static_cast<int64_t>(b) * p.table_stride + pg);
  if (page < 0 || page >= p.n_pages) {
    if (threadIdx.x == 0) record_error(p.status, CALIBATT_ERR_CSR);
    return;
  }
  const int lo = max(begin - pg * kPage, 0), hi = min(st.len - pg * kPage, kPage);  // new slots of the page
  const int chunk = threadIdx.x & 15, row0 = threadIdx.x >> 4;
  const int64_t first = st.t0 + (static_cast<int64_t>(pg) * kPage - begin);  // token of slot 0
  const __nv_bfloat16* x = p.x[which] + head * p.hs[which] + chunk * 8;
  const int64_t ts = p.ts[which];

  // The largest magnitude, as the bit pattern of a bf16 value without its sign
  // (they are ordered like the values). 0x7f80 and more is not finite: then,
  // rarely, the page is looked through again without those.
  uint4 v[kPasses];
  uint32_t top = 0;  // two 16-bit maxima
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = row0 + i * kRowsPerPass;
    v[i] = make_uint4(0, 0, 0, 0);
    if (r >= lo && r < hi) v[i] = ld_stream(x + (first + r) * ts);
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    top = __vmaxu2(top, __vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu));
    top = __vmaxu2(top, __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu));
  }
  __shared__ uint32_t part[2][kWriteThreads / 32];
  auto block_max = [&](uint32_t t, uint32_t* at) {
    t = max(t & 0xffffu, t >> 16);
    t = __reduce_max_sync(0xffffffffu, t);
    if ((threadIdx.x & 31) == 0) at[threadIdx.x >> 5] = t;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWriteThreads / 32; ++i) t = max(t, at[i]);
    return t;
  };
  // the page's scale is read by every thread before thread 0 replaces it
  float* scale = p.scale[which] + static_cast<int64_t>(page) * p.heads + head;
  const float old = lo > 0 ? *scale : 0.f;
  top = block_max(top, part[0]);
  const bool finite = top < 0x7f80u;
  if (!finite) {
    top = 0;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a = w[j] & 0x7fffu, c = w[j] >> 16 & 0x7fffu;
        top = max(top, max(a < 0x7f80u ? a : 0u, c < 0x7f80u ? c : 0u));
      }
    }
    top = block_max(top, part[1]);
  }
  const int e = page_exponent(__uint_as_float(top << 16));
  const float now = fmaxf(exp2_int(e), old);
  const float inv = 1.f / now;  // exact: a power of two
  uint8_t* c = p.c[which] + (static_cast<int64_t>(page) * p.heads + head) * (kPage * 128) + chunk * 8;
  if (lo > 0 && now != old) {
    // entries written earlier, in units of the larger scale
    const float ratio = old * inv;
#pragma unroll 1
    for (int r = row0; r < lo; r += kRowsPerPass) {
      uint2* at = reinterpret_cast<uint2*>(c + r * 128);
      const uint2 w = *at;
      uint32_t in[2] = {w.x, w.y}, out[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 a = e4m3x2_to_float2(in[j] & 0xffffu), d = e4m3x2_to_float2(in[j] >> 16);
        out[j] = to_e4m3x2<false>(a.x * ratio, a.y * ratio) | to_e4m3x2<false>(d.x * ratio, d.y * ratio) << 16;
      }
      *at = make_uint2(out[0], out[1]);
    }
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = row0 + i * kRowsPerPass;
    if (r < lo || r >= hi) continue;
    *reinterpret_cast<uint2*>(c + r * 128) = finite ? to_e4m3x8<true>(v[i], inv) : to_e4m3x8<false>(v[i], inv);
  }
  if (threadIdx.x == 0 && now != old) *scale = now;
}

}  // namespace
}  // namespace calibatt

extern "C" int calibatt_cache_write(const calibatt_bf16* k, int64_t k_token_stride, int64_t k_head_stride,
                                    const calibatt_bf16* v, int64_t v_token_stride, int64_t v_head_stride, int heads,
                                    int n, int d, const int32_t* tok_start, const int32_t* kv_len, int batch,
                                    int max_new, const int32_t* table, int table_stride, int n_pages, uint8_t* k8,
                                    uint8_t* v8, float* k_scale, float* v_scale, calibatt_stream_t stream) {
  using namespace calibatt;
  if (heads < 1 || heads > (1 << 20) || n < 0 || batch < 0 || max_new < 0 || table_stride < 0 || n_pages < 0)
    return CALIBATT_ERR_ARG;
  if (d != CALIBATT_HEAD_DIM) return CALIBATT_ERR_UNSUPPORTED;
  if (batch > 65535) return CALIBATT_ERR_UNSUPPORTED;
  if (n == 0 || batch == 0 || max_new == 0) return CALIBATT_OK;
  if (!k || !v || !tok_start || !kv_len || !table || !k8 || !v8 || !k_scale || !v_scale || table_stride < 1 ||
      n_pages < 1 || k_token_stride < 0 || k_head_stride < 0 || v_token_stride < 0 || v_head_stride < 0 ||
      k8 == v8 || k_scale == v_scale)
    return CALIBATT_ERR_ARG;
  for (const int64_t s : {k_token_stride, v_token_stride})
    if (s > (INT64_MAX >> 24) / n) return CALIBATT_ERR_ARG;
  for (const int64_t s : {k_head_stride, v_head_stride})
    if (s > (INT64_MAX >> 24) / heads) return CALIBATT_ERR_ARG;
  for (const void* x : {static_cast<const void*>(k), static_cast<const void*>(v), static_cast<const void*>(k8),
                        static_cast<const void*>(v8)})
    if (reinterpret_cast<uintptr_t>(x) & 15u) return CALIBATT_ERR_ALIGN;
  if ((k_token_stride | k_head_stride | v_token_stride | v_head_stride) & 7) return CALIBATT_ERR_ALIGN;
  for (const void* x : {static_cast<const void*>(tok_start), static_cast<const void*>(kv_len),
                        static_cast<const void*>(table), static_cast<const void*>(k_scale),
                        static_cast<const void*>(v_scale)})
    if (reinterpret_cast<uintptr_t>(x) & 3u) return CALIBATT_ERR_ALIGN;
  WriteParams p{};
  p.status = status_word();
  if (!p.status) return CALIBATT_ERR_CUDA;
  p.x[0] = reinterpret_cast<const __nv_bfloat16*>(k);
  p.x[1] = reinterpret_cast<const __nv_bfloat16*>(v);
  p.ts[0] = k_token_stride;
  p.hs[0] = k_head_stride;
  p.ts[1] = v_token_stride;
  p.hs[1] = v_head_stride;
  p.c[0] = k8;
  p.c[1] = v8;
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  p.tok_start = tok_start;
  p.kv_len = kv_len;
  p.table = table;
  p.heads = heads;
  p.n = n;
  p.batch = batch;
  p.max_new = max_new;
  p.table_stride = table_stride;
  p.n_pages = n_pages;
  // pages that max_new tokens can touch, wherever in a page they start
  const int64_t most = (static_cast<int64_t>(std::min(max_new, n)) + kPage - 2) / kPage + 1;
  if (most > 65535) return CALIBATT_ERR_UNSUPPORTED;
  const dim3 grid(2u * heads, static_cast<unsigned>(most), static_cast<unsigned>(batch));
  cache_write_kernel<<<grid, kWriteThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? CALIBATT_OK : CALIBATT_ERR_CUDA;
}
