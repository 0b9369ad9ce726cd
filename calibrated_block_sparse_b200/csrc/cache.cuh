// Pieces shared by the kernels of the paged 8-bit cache: a stream's share of
// the packed tokens, and e4m3 conversions.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace calibatt {

constexpr int kPage = 128;  // tokens per cache page

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
  s.bad = s.t0 < 0 || t1 < s.t0 || t1 > n || s.len < 0 || s.len > static_cast<int64_t>(table_stride) * kPage;
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

}  // namespace calibatt
