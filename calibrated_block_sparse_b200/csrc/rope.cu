// Rotary positions over several axes (time, height, width) for the queries
// and keys of an attention call, and the gradient (the inverse rotation).
//
// Pair i of channels (a, b) of a token at position p is rotated by the angle
// p[axis(i)] * freq(i):
//   y_a = x_a cos - x_b sin,   y_b = x_a sin + x_b cos.
// The angle is taken in 64 bits and in turns (freq / 2 pi): the product with
// the position is reduced to a fraction of a turn exactly there, and only the
// fraction is rounded to fp32 for sincospi, so far positions lose nothing.
// The rotation is fp32, rounded once to bf16.
//
// Bound by memory: 2 bytes read and 2 written per value. A thread keeps one
// token's sines and cosines of its channels in registers and walks the heads
// (queries, then keys) with them, so their cost is shared by all heads; reads
// and writes are whole 256-byte rows, which makes the change between the
// projections' token-major layout and the attention's head-major one free.
// Measured on B200: 32760 tokens x 80 heads (1.34 GB) in 211 us, 98 % of the
// rate of a plain copy.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "calibatt.h"
#include "kernels.h"
#include "ptx.cuh"
#include "sched.cuh"

namespace calibatt {
namespace {

constexpr int kRopeThreads = 64;

struct RopeView {
  const __nv_bfloat16* in;
  __nv_bfloat16* out;
  int64_t in_ts, in_hs, out_ts, out_hs;  // token and head strides, elements
  int heads;
};

struct RopeParams {
  RopeView t[2];  // queries, keys
  int64_t n;
  int pairs;
  int inverse;
  const int32_t* pos;  // [n][3] or NULL: the grid
  int64_t hw;
  int W;
  int start[3];
  int heads_per_cta;  // heads (queries and keys together) of one CTA
  int head_lanes;     // heads that a CTA works on at the same time
  double turns[64];
  uint8_t axis[64];
};

__device__ __forceinline__ void pair_angle(const RopeParams& p, const double (&pos)[3], int i, float& c, float& s) {
  if (i >= p.pairs) {
    c = 1.f;
    s = 0.f;
    return;
  }
  const int ax = p.axis[i];
  const double t = (ax == 0 ? pos[0] : ax == 1 ? pos[1] : pos[2]) * p.turns[i];
  const float f = static_cast<float>(t - rint(t));  // fraction of a turn, |f| <= 1/2
  sincospif(2.f * f, &s, &c);
  if (p.inverse) s = -s;
}

// Rotates the pairs of two packed words (interleaved: a word is a pair).
__device__ __forceinline__ uint32_t rotate_word(uint32_t w, float c, float s, bool on) {
  const float a = __uint_as_float(w << 16), b = __uint_as_float(w & 0xffff0000u);
  return on ? pack_bf16x2(a * c - b * s, a * s + b * c) : w;
}

// Rotates two pairs whose first channels are packed in a, second ones in b.
__device__ __forceinline__ void rotate_words(uint32_t& a, uint32_t& b, const float* c, const float* s) {
  const float a0 = __uint_as_float(a << 16), a1 = __uint_as_float(a & 0xffff0000u);
  const float b0 = __uint_as_float(b << 16), b1 = __uint_as_float(b & 0xffff0000u);
  a = pack_bf16x2(a0 * c[0] - b0 * s[0], a1 * c[1] - b1 * s[1]);
  b = pack_bf16x2(a0 * s[0] + b0 * c[0], a1 * s[1] + b1 * c[1]);
}

// kHalves: pair i is channels (i, i + pairs), else (2i, 2i + 1).
// Interleaved: 16 threads per token, one 16-byte chunk (4 pairs) each.
// Halves: 8 threads per token, two chunks each: a chunk and its partner
// (8 pairs), or two chunks behind the rotated channels.
template <bool kHalves>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kLanes = kHalves ? 8 : 16;
  constexpr int kPairs = kHalves ? 8 : 4;
  const int lane = threadIdx.x % kLanes;
  const int slot = threadIdx.x / kLanes;
  const int head_lane = slot % p.head_lanes;
  const int tokens = (kRopeThreads / kLanes) / p.head_lanes;
  const int64_t token = static_cast<int64_t>(blockIdx.x) * tokens + slot / p.head_lanes;
  if (token >= p.n) return;

  double pos[3];
  if (p.pos) {
    for (int a = 0; a < 3; ++a) pos[a] = __ldg(p.pos + token * 3 + a);
  } else {
    const int64_t f = token / p.hw;
    const int rem = static_cast<int>(token - f * p.hw);
    pos[0] = static_cast<double>(p.start[0]) + static_cast<double>(f);
    pos[1] = static_cast<double>(p.start[1]) + rem / p.W;
    pos[2] = static_cast<double>(p.start[2]) + rem % p.W;
  }
  const int rot = p.pairs >> 3;  // halves: chunks of the first half
  const bool on_h = lane < rot;
  const int c0 = kHalves ? (on_h ? lane : 2 * rot + 2 * (lane - rot)) : lane;
  const int c1 = kHalves ? (on_h ? lane + rot : c0 + 1) : 0;
  const int heads = p.t[0].heads + p.t[1].heads;
  const int h_end = min(heads, (static_cast<int>(blockIdx.y) + 1) * p.heads_per_cta);
  // kBatch heads are loaded at a time, and the next ones before these are
  // stored: the output may be the input's own memory, so the compiler cannot
  // move a load over a store. The first loads run beside the sines. With half
  // as many heads at a time 24.4 and 34.4 us instead of 21.6 and 32.6 (the
  // sizes named at the launch), with more of them 24 and 32.
  constexpr int kBatch = kHalves ? 4 : 8;
  constexpr int kChunks = kHalves ? 2 : 1;
  uint4 v[kBatch][kChunks], next[kBatch][kChunks];
  auto load = [&](int h0, uint4 (&w)[kBatch][kChunks]) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i * p.head_lanes;
      if (h >= h_end) break;
      const bool second = h >= p.t[0].heads;
      const __nv_bfloat16* in = second ? p.t[1].in + (h - p.t[0].heads) * p.t[1].in_hs + token * p.t[1].in_ts
                                       : p.t[0].in + h * p.t[0].in_hs + token * p.t[0].in_ts;
      w[i][0] = reinterpret_cast<const uint4*>(in)[c0];
      if constexpr (kHalves) w[i][1] = reinterpret_cast<const uint4*>(in)[c1];
    }
  };
  int h0 = blockIdx.y * p.heads_per_cta + head_lane;
  load(h0, v);
  float cs[kPairs], sn[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) pair_angle(p, pos, (kHalves ? lane * 8 : lane * 4) + i, cs[i], sn[i]);
  for (; h0 < h_end; h0 += kBatch * p.head_lanes) {
    load(h0 + kBatch * p.head_lanes, next);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i * p.head_lanes;
      if (h >= h_end) break;
      const bool second = h >= p.t[0].heads;
      __nv_bfloat16* out = second ? p.t[1].out + (h - p.t[0].heads) * p.t[1].out_hs + token * p.t[1].out_ts
                                  : p.t[0].out + h * p.t[0].out_hs + token * p.t[0].out_ts;
      uint4& x = v[i][0];
      if constexpr (!kHalves) {
        x.x = rotate_word(x.x, cs[0], sn[0], lane * 4 + 0 < p.pairs);
        x.y = rotate_word(x.y, cs[1], sn[1], lane * 4 + 1 < p.pairs);
        x.z = rotate_word(x.z, cs[2], sn[2], lane * 4 + 2 < p.pairs);
        x.w = rotate_word(x.w, cs[3], sn[3], lane * 4 + 3 < p.pairs);
      } else if (on_h) {
        uint4& y = v[i][1];
        rotate_words(x.x, y.x, cs + 0, sn + 0);
        rotate_words(x.y, y.y, cs + 2, sn + 2);
        rotate_words(x.z, y.z, cs + 4, sn + 4);
        rotate_words(x.w, y.w, cs + 6, sn + 6);
      }
      reinterpret_cast<uint4*>(out)[c0] = x;
      if constexpr (kHalves) reinterpret_cast<uint4*>(out)[c1] = v[i][1];
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
#pragma unroll
      for (int j = 0; j < kChunks; ++j) v[i][j] = next[i][j];
  }
}

// Extent in elements of a view [n][heads][128] with the given strides.
int64_t extent(int64_t n, int heads, int64_t ts, int64_t hs) { return (n - 1) * ts + (heads - 1) * hs + 128; }

struct View {
  uintptr_t base;
  int64_t n, ts, hs;
  int heads;
};

// Whether no byte belongs to both views: disjoint ranges, or interleaved rows
// of one buffer (one token stride that holds every head of a row, as in a
// fused projection's output).
bool disjoint(const View& a, const View& b) {
  if (!a.base || !b.base) return true;
  const uintptr_t ae = a.base + 2 * extent(a.n, a.heads, a.ts, a.hs);
  const uintptr_t be = b.base + 2 * extent(b.n, b.heads, b.ts, b.hs);
  if (ae <= b.base || be <= a.base) return true;
  const int64_t row_a = (a.heads - 1) * a.hs + 128, row_b = (b.heads - 1) * b.hs + 128;
  if (a.n == 1) return false;
  if (a.ts != b.ts || row_a > a.ts || row_b > b.ts) return false;
  const View& lo = a.base <= b.base ? a : b;
  const View& hi = a.base <= b.base ? b : a;
  const int64_t off = static_cast<int64_t>(hi.base - lo.base) / 2 % a.ts;
  const int64_t row_lo = &lo == &a ? row_a : row_b, row_hi = &lo == &a ? row_b : row_a;
  return off >= row_lo && off + row_hi <= a.ts;
}

bool same(const View& a, const View& b) { return a.base == b.base && a.ts == b.ts && a.hs == b.hs; }

// A view that is written names every element once.
bool writable(const View& v) {
  if (v.n > 1 && v.ts < 128) return false;
  if (v.heads > 1 && v.hs < 128) return false;
  if (v.n == 1 || v.heads == 1) return true;
  return v.ts >= (v.heads - 1) * v.hs + 128 || v.hs >= (v.n - 1) * v.ts + 128;
}

int check_view(const void* ptr, int heads, int64_t n, int64_t ts, int64_t hs) {
  if (!ptr || ts < 0 || hs < 0) return CALIBATT_ERR_ARG;
  // extents stay far from 64 bits
  if (ts > (INT64_MAX >> 24) / n || hs > (INT64_MAX >> 24) / heads) return CALIBATT_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(ptr) & 15u) || (ts & 7) || (hs & 7)) return CALIBATT_ERR_ALIGN;
  return CALIBATT_OK;
}

int rope(const calibatt_rope_plan* plan, const void* q, int64_t q_ts, int64_t q_hs, int heads_q, const void* k,
         int64_t k_ts, int64_t k_hs, int heads_k, int64_t n, int d, const int32_t* pos, int H, int W,
         const int32_t* start, void* q_out, int64_t qo_ts, int64_t qo_hs, void* k_out, int64_t ko_ts, int64_t ko_hs,
         bool inverse, cudaStream_t stream) {
  if (!plan || n < 0 || heads_q < 0 || heads_k < 0 || heads_q + static_cast<int64_t>(heads_k) < 1 ||
      heads_q > 65535 || heads_k > 65535 || n > INT_MAX)
    return CALIBATT_ERR_ARG;
  if (d != CALIBATT_HEAD_DIM) return CALIBATT_ERR_UNSUPPORTED;
  if (plan->pairs < 1 || plan->pairs > 64 || (plan->pairing != CALIBATT_ROPE_INTERLEAVED &&
                                              plan->pairing != CALIBATT_ROPE_HALVES))
    return CALIBATT_ERR_ARG;
  const bool halves = plan->pairing == CALIBATT_ROPE_HALVES;
  if (halves && (plan->pairs & 7)) return CALIBATT_ERR_UNSUPPORTED;
  for (int i = 0; i < plan->pairs; ++i)
    if (plan->axis[i] > 2 || !std::isfinite(plan->turns[i])) return CALIBATT_ERR_ARG;
  if (!pos && (H < 1 || W < 1)) return CALIBATT_ERR_ARG;
  if (pos && (reinterpret_cast<uintptr_t>(pos) & 3u)) return CALIBATT_ERR_ALIGN;
  if (n == 0) return CALIBATT_OK;
  RopeParams p;
  std::memset(&p, 0, sizeof p);
  View in[2] = {}, out[2] = {};
  const void* ins[2] = {q, k};
  void* outs[2] = {q_out, k_out};
  const int64_t its[2] = {q_ts, k_ts}, ihs[2] = {q_hs, k_hs}, ots[2] = {qo_ts, ko_ts}, ohs[2] = {qo_hs, ko_hs};
  const int heads[2] = {heads_q, heads_k};
  for (int i = 0; i < 2; ++i) {
    if (heads[i] == 0) continue;
    int rc = check_view(ins[i], heads[i], n, its[i], ihs[i]);
    if (rc == CALIBATT_OK) rc = check_view(outs[i], heads[i], n, ots[i], ohs[i]);
    if (rc != CALIBATT_OK) return rc;
    in[i] = View{reinterpret_cast<uintptr_t>(ins[i]), n, its[i], ihs[i], heads[i]};
    out[i] = View{reinterpret_cast<uintptr_t>(outs[i]), n, ots[i], ohs[i], heads[i]};
    if (!writable(out[i])) return CALIBATT_ERR_ARG;
    p.t[i] = RopeView{static_cast<const __nv_bfloat16*>(ins[i]), static_cast<__nv_bfloat16*>(outs[i]), its[i], ihs[i],
                      ots[i], ohs[i], heads[i]};
  }
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j)
      if (!disjoint(out[i], in[j]) && !(i == j && same(out[i], in[j]))) return CALIBATT_ERR_ARG;
  if (!disjoint(out[0], out[1])) return CALIBATT_ERR_ARG;
  p.n = n;
  p.pairs = plan->pairs;
  p.inverse = inverse;
  p.pos = pos;
  p.hw = static_cast<int64_t>(H) * W;
  p.W = W;
  if (pos) p.hw = p.W = 1;
  for (int a = 0; a < 3; ++a) p.start[a] = start ? start[a] : 0;
  for (int i = 0; i < plan->pairs; ++i) {
    p.turns[i] = plan->turns[i];
    p.axis[i] = plan->axis[i];
  }
  const int all = heads_q + heads_k;
  const int slots = kRopeThreads / (halves ? 8 : 16);
  // few tokens: a CTA's slots take several heads of a token instead of several tokens
  p.head_lanes = 1;
  while (p.head_lanes < slots && static_cast<int64_t>(slots / p.head_lanes) > n) p.head_lanes *= 2;
  const int64_t gx = (n * p.head_lanes + slots - 1) / slots;
  // and the heads are spread over CTAs until there are 12 per SM: fewer leave
  // SMs idle, more repeat the sines. Measured at 7421 tokens x 32 heads with
  // halves paired: 21.6 us with 12, 22.7 with 16, 25.1 with 32; at 4680 x 80
  // (192 MB): 32.6, 32.9, 33.5 (CTAs of 128 threads, 8 per SM: 23.0 and 33.1).
  const int64_t want = 12ll * sm_count();
  int64_t gy = (want + gx - 1) / gx;
  const int64_t most = (all + p.head_lanes - 1) / p.head_lanes;
  if (gy > most) gy = most;
  p.heads_per_cta = static_cast<int>((all + gy - 1) / gy);
  p.heads_per_cta = (p.heads_per_cta + p.head_lanes - 1) / p.head_lanes * p.head_lanes;
  gy = (all + p.heads_per_cta - 1) / p.heads_per_cta;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
  if (halves)
    rope_kernel<true><<<grid, kRopeThreads, 0, stream>>>(p);
  else
    rope_kernel<false><<<grid, kRopeThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? CALIBATT_OK : CALIBATT_ERR_CUDA;
}

}  // namespace
}  // namespace calibatt

extern "C" {

int calibatt_rope_plan_init(const int32_t* dims, double theta, int pairing, int ladder, calibatt_rope_plan* plan) {
  if (!dims || !plan || !std::isfinite(theta) || theta <= 0.0 ||
      (pairing != CALIBATT_ROPE_INTERLEAVED && pairing != CALIBATT_ROPE_HALVES) ||
      (ladder != CALIBATT_ROPE_LADDER_AXIS && ladder != CALIBATT_ROPE_LADDER_SHARED))
    return CALIBATT_ERR_ARG;
  int64_t sum = 0;
  for (int a = 0; a < 3; ++a) {
    if (dims[a] < 0 || (dims[a] & 1)) return CALIBATT_ERR_ARG;
    sum += dims[a];
  }
  if (sum < 2 || sum > CALIBATT_HEAD_DIM) return CALIBATT_ERR_ARG;
  if (pairing == CALIBATT_ROPE_HALVES && (sum / 2) % 8) return CALIBATT_ERR_UNSUPPORTED;
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  std::memset(plan, 0, sizeof *plan);
  plan->pairs = static_cast<int32_t>(sum / 2);
  plan->pairing = pairing;
  int i = 0;
  for (int a = 0; a < 3; ++a)
    for (int j = 0; j < dims[a] / 2; ++j, ++i) {
      const double e = ladder == CALIBATT_ROPE_LADDER_AXIS ? 2.0 * j / dims[a] : 2.0 * i / static_cast<double>(sum);
      plan->turns[i] = std::pow(theta, -e) / kTwoPi;
      plan->axis[i] = static_cast<uint8_t>(a);
    }
  return CALIBATT_OK;
}

int calibatt_rope_fwd(const calibatt_rope_plan* plan, const calibatt_bf16* q, int64_t q_token_stride,
                      int64_t q_head_stride, int heads_q, const calibatt_bf16* k, int64_t k_token_stride,
                      int64_t k_head_stride, int heads_k, int64_t n, int d, const int32_t* pos, int H, int W,
                      const int32_t* start, calibatt_bf16* q_out, int64_t q_out_token_stride,
                      int64_t q_out_head_stride, calibatt_bf16* k_out, int64_t k_out_token_stride,
                      int64_t k_out_head_stride, calibatt_stream_t stream) {
  return calibatt::rope(plan, q, q_token_stride, q_head_stride, heads_q, k, k_token_stride, k_head_stride, heads_k, n,
                        d, pos, H, W, start, q_out, q_out_token_stride, q_out_head_stride, k_out, k_out_token_stride,
                        k_out_head_stride, false, reinterpret_cast<cudaStream_t>(stream));
}

int calibatt_rope_bwd(const calibatt_rope_plan* plan, const calibatt_bf16* dq_out, int64_t dq_out_token_stride,
                      int64_t dq_out_head_stride, int heads_q, const calibatt_bf16* dk_out,
                      int64_t dk_out_token_stride, int64_t dk_out_head_stride, int heads_k, int64_t n, int d,
                      const int32_t* pos, int H, int W, const int32_t* start, calibatt_bf16* dq,
                      int64_t dq_token_stride, int64_t dq_head_stride, calibatt_bf16* dk, int64_t dk_token_stride,
                      int64_t dk_head_stride, calibatt_stream_t stream) {
  return calibatt::rope(plan, dq_out, dq_out_token_stride, dq_out_head_stride, heads_q, dk_out, dk_out_token_stride,
                        dk_out_head_stride, heads_k, n, d, pos, H, W, start, dq, dq_token_stride, dq_head_stride, dk,
                        dk_token_stride, dk_head_stride, true, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
