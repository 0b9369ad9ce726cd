// Attention over the paged 8-bit cache for few query rows (up to 16 that share
// a key head: one token of up to 16 query heads, a few tokens of a head).
//
// Bound by reading the cache once. Its pages are one list, stream by stream,
// key head by key head, cut into equal shares: two CTAs per SM, whatever the
// streams' lengths are (they are read on the device), so no SM waits for a
// long stream. A stretch of a share that is not all of its stream's pages
// leaves maximum, sum and unnormalised output in the workspace, and
// cache_join_kernel joins them.
//
// The tensor core multiplies the cache's bytes as they are: a page is the
// 128-row operand A, K as it lies in memory and V transposed, and the few rows
// are operand B:
//   S^T [key][row] = K Q^T,   O^T [channel][row] += V^T P^T   (kind::f8f6f4)
// so nothing of the cache passes through registers (converting it to fp16
// there, for mma.sync, took ~500 ALU instructions per warp and 8 KB and held
// the kernel at 52 % of the DRAM rate). Q and P are written as sums of e5m2
// values: three parts of 3 significant bits hold a bf16 value's 8 exactly, four
// parts hold P to 2^-12. The products of Q's parts are accumulated into the
// same columns of S^T; those of P's parts have columns of their own (one
// product instead of four), which are added up at the end of a stretch.
// e5m2 spans 2^-16 .. 2^15, so a row of Q, scaled by a power of two to a
// largest value in [2^13, 2^14), is exact down to 2^-22 of it and within 2^-31
// of it below, and weights keep a bit down to 2^-24 of the largest.
//
// CTA:
//   warp  0    TMA producer: K and V tiles (16 KB) into a 5-stage ring
//   warp  1    MMA issuer: S^T of the next page before O^T of this one
//   4 warps    softmax; thread = key of the page = TMEM lane of S^T, and
//              channel = TMEM lane of O^T at the end
// More than 4 rows are shared out to two such groups of 4 warps, 4 or 8 rows
// each: the softmax of 16 rows in one thread is a chain of ~4000 cycles a page
// (8 rows of 30000 keys, 2 streams: 34 us in one group, 32 in two; 15 rows in
// four groups, whose registers do not fit: 8 us more than in two).
// Two CTAs of 320 threads leave 96 registers a thread: with 8 rows a group
// ptxas spills 100 bytes, with 1 and 4 rows none.
// The running maximum of a row moves only if it grew by more than 2^4, which a
// page finds out with one vote of a group's warps.
//
// Measured on B200: one token of 40 heads over 32760 cached (335 MB) in 60 us,
// 86 % of the rate of a plain copy; 16 streams of 20000 tokens, 40 query heads
// on 8, 3 tokens each (15 rows a key head, 437 MB) in 99 us, 68 %: there each
// page is a chain of score, vote, exponential, parts, store and product, and
// four of them (two CTAs with two groups) run on an SM at a time.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
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

constexpr int few_threads(int groups) { return 64 + 128 * groups; }
constexpr int kFewRing = 5;
constexpr int kPageBytes = kPage * 128;
constexpr float kFewStale = 4.0f;                              // log2 units
constexpr float kNoMax = -3e38f;                               // of a row that has seen no key
constexpr int kQParts = 3, kPParts = 4;

// Columns (N) of a product with `parts` columns per row: a multiple of 16.
__host__ __device__ constexpr int few_cols(int rows, int parts) { return (rows * parts + 15) / 16 * 16; }

struct FewBarriers {
  uint64_t full[kFewRing], empty[kFewRing];
  uint64_t q_full;
  uint64_t s_full[2], p_full[2];  // per buffer of S^T and P^T
  uint64_t pv_done;               // every page's O^T product
  uint64_t o_full;                // the last one of a stretch
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
  int nan_seen;
  int limit[kFewRows];            // keys that a row sees
  float c[kFewRows];              // a raw score's factor, without the key scale
  Walk walk[10];                  // per warp: it would hold 14 registers from one stretch to the next
  float top[4][kFewRows];         // per warp of a group, of a page
  float sum[4][kFewRows];         // per warp of a group, at a stretch's end
};

struct FewLayout {
  static constexpr int kRingOff = 0;
  static constexpr int kQOff = kFewRing * kPageBytes;                  // Q^T's operand: rows of 128 channels, part by part
  static constexpr int kPOff = kQOff + kQParts * few_cols(kFewRows, 1) * 128;  // P^T's two buffers
  static constexpr int kPBytes = few_cols(kFewRows, kPParts) * 128;
  static constexpr int kBarOff = kPOff + 2 * kPBytes;
  static constexpr int kDynSmem = kBarOff + static_cast<int>(sizeof(FewBarriers)) + 1024;
};
// two CTAs on an SM (228 KB, of which each takes 1 KB more)
static_assert(2 * (FewLayout::kDynSmem + 1024) <= 233472, "shared memory budget");

// Tensor memory: S^T in two buffers of 16 columns, O^T in up to 64.
constexpr uint32_t kFewCols = 128, kSBuf = 32, kOCol = 64;

// kind::f8f6f4, A e4m3, B e5m2, fp32 accumulation, M = 128; with mn_major A (V)
// has its channels and B (P^T) its rows contiguous.
__host__ __device__ constexpr uint32_t idesc_f8(int N, bool mn_major) {
  return (1u << 4) | (0u << 7) | (1u << 10) | ((mn_major ? 3u : 0u) << 15) | (static_cast<uint32_t>(N >> 3) << 17) |
         (8u << 24);
}

// P^T as operand B with its rows contiguous and no swizzle: planes of 16 rows,
// a plane 16 bytes of each of the page's keys. A thread, which holds one key's
// weights, then writes them 16 at a time and consecutive lanes write
// consecutive bytes (byte by byte into rows of keys, 32 stores a page: 2 us
// more with 15 rows).
constexpr int kPPlane = kPage * 16;
__device__ __forceinline__ uint64_t desc_p(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) |
         static_cast<uint64_t>(128 >> 4) << 16 |      // from 8 keys to the next
         static_cast<uint64_t>(kPPlane >> 4) << 32 |  // from 16 rows to the next
         1ull << 46;
}

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Vote of a group's four warps.
__device__ __forceinline__ bool vote_128(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x)), "r"(id)
      : "memory");
  return r != 0;
}

// The kParts columns of RG rows, added up: column part * RG + r, of one lane.
template <int RG, int kParts>
__device__ __forceinline__ void tmem_rows(uint32_t taddr, float (&x)[RG]) {
  uint32_t c[few_cols(RG, kParts)];
  tmem_ld16s_wait(taddr, c);
#pragma unroll
  for (int r = 0; r < RG; ++r) {
    float sum = __uint_as_float(c[(kParts - 1) * RG + r]);  // the small parts first
#pragma unroll
    for (int i = kParts - 2; i >= 0; --i) sum += __uint_as_float(c[i * RG + r]);
    x[r] = sum;
  }
}

// The leading three significant bits of x, exactly an e5m2 value down to 2^-14.
__device__ __forceinline__ float three_bits(float x) { return __uint_as_float(__float_as_uint(x) & 0xffe00000u); }

__device__ __forceinline__ uint32_t to_e5m2x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E5M2);
}

// Where V of page i of a stretch of `count` is in the ring's order.
__device__ __forceinline__ uint32_t v_tile(int i, int count) { return i + 1 < count ? 2 * i + 2 : 2 * i + 1; }

// Whether a row that sees `limit` keys has a NaN value in this channel among
// the stretch's pages that not every row sees whole.
__device__ __forceinline__ bool stretch_nan(const CacheAttnParams& p, const Stretch& s, int limit, int least,
                                            int channel) {
  const int32_t* table = p.table + static_cast<int64_t>(s.b) * p.table_stride;
  for (int k = max(least / kPage, s.pg) * kPage; k < min(limit, (s.pg + s.count) * kPage); ++k) {
    const int id = __ldg(table + k / kPage);
    if (id < 0 || id >= p.n_pages) continue;
    if ((p.v8[((static_cast<int64_t>(id) * p.heads_kv + s.head) * kPage + k % kPage) * 128 + channel] & 0x7f) == 0x7f)
      return true;
  }
  return false;
}

template <bool SW, int RG, int G>  // G groups of softmax warps, each laid out for RG rows
__global__ void __launch_bounds__(few_threads(G), 2)
    cache_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ CacheAttnParams p, bool whole, float* part) {
  using L = FewLayout;
  constexpr int RB = RG * G, kAll = 128 * G;
  static_assert(few_threads(G) / 32 <= sizeof(FewBarriers::walk) / sizeof(Walk), "a walk per warp");
  constexpr int kQCols = few_cols(RG * G, 1), kPCols = few_cols(RG * G, kPParts);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const uint32_t sbase = smem_u32(smem);
  FewBarriers& bar = *reinterpret_cast<FewBarriers*>(smem + L::kBarOff);
  volatile int* abort_flag = &bar.abort;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kFewRing; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 1);
    }
    mbar_init(&bar.q_full, kAll);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_full[i], kAll);
    }
    mbar_init(&bar.pv_done, 1);
    mbar_init(&bar.o_full, 1);
    mbar_init(&bar.mma_done, 1);
    bar.abort = 0;
    bar.nan_seen = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(&bar.tmem_base, kFewCols);
  {  // the lists are on their way while the barriers and tensor memory are made
    Walk walk;
    walk.start(p, whole, lane);
    if (lane == 0) bar.walk[warp] = walk;
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bar.tmem_base, 0);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // for all lanes of a warp, or its lane 0 alone
  auto next_stretch = [&](Stretch& s, unsigned lanes) -> bool {
    Walk walk = bar.walk[warp];
    const bool more = walk.next(p, s);
    __syncwarp(lanes);
    if (lane == 0) bar.walk[warp] = walk;
    __syncwarp(lanes);
    return more;
  };
  Stretch s;
  if (warp == 0) {
    // ---------------------------------------------------------- TMA producer
    uint32_t stage = 0, phase = 0;
    int used = 0;
    bool ok = true;
    while (ok && next_stretch(s, 0xffffffffu)) {
      PageWindow<false> win(p, s.b, s.head, s.pg, s.count, s.st.len);
      win.fetch(lane, p.status);
      int id_now = -1, id_before = -1, k_at = 0;
      for (int t = 0; t < 2 * s.count && ok; ++t) {
        bool is_v;
        int i, id;
        ring_tile<true>(t, s.count, is_v, i);
        if (!is_v) {
          if ((i & 31) == 0) win.advance(i, lane, p.status);
          id_before = id_now;
          id_now = id = __shfl_sync(0xffffffffu, win.id, i & 31);
          k_at = i;
        } else {
          id = k_at == i ? id_now : id_before;
        }
        if (lane == 0) {
          ok = mbar_wait<SW>(&bar.empty[stage], phase ^ 1, abort_flag, p.status, p.wait_limit_ns);
          if (ok) {
            if (id >= 0) {
              mbar_arrive_expect_tx(&bar.full[stage], kPageBytes);
              tma_load_2d(smem + L::kRingOff + stage * kPageBytes, is_v ? &tm_v : &tm_k, &bar.full[stage], 0,
                          (id * p.heads_kv + s.head) * kPage);
            } else {
              mbar_arrive(&bar.full[stage]);  // nothing to read: the softmax warps leave the page out
            }
            ++used;
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (++stage == kFewRing) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    // streams that do not fit are reported once
    if (blockIdx.x == 0)
      for (int b = lane; b < p.batch; b += 32) {
        const Stream st = stream_of(p.tok_start, p.kv_len, b, p.n, p.table_stride);
        if (!stream_fits(p, st)) record_error(p.status, CALIBATT_ERR_CSR);
      }
    // no copy may still be landing when the CTA leaves
    __syncwarp();
    if (lane == 0)
      for (int i = used > kFewRing ? used - kFewRing : 0; i < used; ++i) {
        volatile int never = 0;
        mbar_wait(&bar.full[i % kFewRing], (i / kFewRing) & 1, &never, p.status);
      }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0) {
      uint32_t stage = 0, phase = 0, turn = 0, stretch = 0;
      const uint64_t ring0 = smem_desc_sw128(sbase + L::kRingOff, 16, 1024);
      const uint64_t q0 = smem_desc_sw128(sbase + L::kQOff, 16, 1024);
      const uint64_t p0 = desc_p(sbase + L::kPOff);
      constexpr uint32_t kIdescS = idesc_f8(kQCols, false), kIdescO = idesc_f8(kPCols, true);
      bool ok = true;
      auto wait = [&](uint64_t* b, uint32_t parity) {
        return mbar_wait<SW>(b, parity, abort_flag, p.status, p.wait_limit_ns);
      };
      auto ring_next = [&]() {
        mma_commit(&bar.empty[stage]);
        if (++stage == kFewRing) {
          stage = 0;
          phase ^= 1;
        }
      };
      // S^T of the page that is `turn` number t: 4 steps of 32 channels (32 bytes of a row)
      auto issue_s = [&](uint32_t t) -> bool {
        if (!wait(&bar.full[stage], phase)) return false;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < kQParts; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f8(tmem + (t & 1) * kSBuf, ring0 + stage * (kPageBytes >> 4) + k * 2,
                   q0 + i * (kQCols * 128 >> 4) + k * 2, kIdescS, (i > 0 || k > 0) ? 1u : 0u);
        mma_commit(&bar.s_full[t & 1]);
        ring_next();
        return true;
      };
      while (ok && next_stretch(s, 1u)) {
        if (!(ok = wait(&bar.q_full, stretch & 1))) break;
        ++stretch;
        if (!(ok = issue_s(turn))) break;
        for (int i = 0; i < s.count; ++i, ++turn) {
          if (i + 1 < s.count && !(ok = issue_s(turn + 1))) break;
          if (!(ok = wait(&bar.p_full[turn & 1], (turn >> 1) & 1))) break;
          if (!(ok = wait(&bar.full[stage], phase))) break;
          tc_fence_after();
          // 4 steps of 32 keys: 32 rows of V (4 KB), 512 bytes of a plane of P^T
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f8(tmem + kOCol, ring0 + stage * (kPageBytes >> 4) + k * (4096 >> 4),
                   p0 + (turn & 1) * (L::kPBytes >> 4) + k * (512 >> 4), kIdescO, (i > 0 || k > 0) ? 1u : 0u);
          mma_commit(&bar.pv_done);
          if (i + 1 == s.count) mma_commit(&bar.o_full);
          ring_next();
        }
      }
      // every issued MMA has finished before tensor memory is released
      mma_commit(&bar.mma_done);
      volatile int never = 0;
      mbar_wait(&bar.mma_done, 0, &never, p.status);
    }
  } else {
    // ---------------------------------------------------------- softmax
    // a warp reaches the 32 lanes of tensor memory that its number modulo 4 names
    const int quarter = warp & 3, g = G == 1 ? 0 : (warp - 2) >> 2;
    const int key = quarter * 32 + lane;  // of a page; channel of the output
    const int r0 = g * RG;                // the group's first row
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const int all = threadIdx.x - 64;
    uint32_t turn = 0;
    int seg = 0;
    // after a failed wait the warps go on without waiting or touching tensor
    // memory, so that they still meet at every barrier
    bool ok = true;  // warp-uniform
    auto wait_warp = [&](uint64_t* b, uint32_t parity) -> bool {
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait<SW>(b, parity, abort_flag, p.status, p.wait_limit_ns));
      return ok;
    };
    uint32_t stage_v = 0;  // ring stages passed: V of this page, for the pages that are cleaned
    while (next_stretch(s, 0xffffffffu)) {
      const int rows = s.st.n_new * p.group;
      PageWindow<true> win(p, s.b, s.head, s.pg, s.count, s.st.len);
      win.fetch(lane, p.status);
      // rows that the stretch does not have see no key
      if (all >= rows && all < RB) {
        bar.c[all] = 0.f;
        bar.limit[all] = 0;
      }
      // the rows of Q as operand B of each part, channels contiguous
      for (int r = warp - 2; r < rows; r += 4 * G) {
        const int tok = r / p.group, h = s.head * p.group + r % p.group;
        const uint2 w = *reinterpret_cast<const uint2*>(
            p.q + (static_cast<int64_t>(h) * p.n + s.st.t0 + tok) * 128 + lane * 4);
        float x[4] = {__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                      __uint_as_float(w.y & 0xffff0000u)};
        float amax = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const float shrink = row_shrink(amax, 13);
        if (lane == 0) {
          bar.c[r] = p.scale_log2 / shrink;
          bar.limit[r] = visible(s.st.len - s.st.n_new + tok, s.st.len, p.unit);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] *= shrink;
#pragma unroll
        for (int part_i = 0; part_i < kQParts; ++part_i) {
          float y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[e] = part_i + 1 < kQParts ? three_bits(x[e]) : x[e];
            x[e] -= y[e];
          }
          const int row = part_i * kQCols + r;
          *reinterpret_cast<uint32_t*>(smem + L::kQOff + row * 128 + ((lane * 4) ^ ((row & 7) << 4))) =
              to_e5m2x2(y[0], y[1]) | to_e5m2x2(y[2], y[3]) << 16;
        }
      }
      fence_proxy_async();
      mbar_arrive(&bar.q_full);
      named_bar_sync(1, kAll);  // c and limit
      float m[RG], l[RG];
#pragma unroll
      for (int r = 0; r < RG; ++r) {
        m[r] = kNoMax;
        l[r] = 0.f;
      }
      const int least = bar.limit[0];  // the first token's rows come first
      VRef<10, -3> vref;  // P below 2^4 (stale maximum) * 2^10 * 2; 2^-24 * 2^10 * 2^-3 is below its smallest value
      const uint32_t ring_base = stage_v;
      for (int i = 0; i < s.count; ++i, ++turn) {
        if ((i & 31) == 0) win.advance(i, lane, p.status);
        const int id = __shfl_sync(0xffffffffu, win.id, i & 31);
        const float ks = __shfl_sync(0xffffffffu, win.ks, i & 31);
        const float o_ratio = vref.page(__shfl_sync(0xffffffffu, win.vs, i & 31));
        const int key0 = (s.pg + i) * kPage;
        const bool partial = id < 0 || key0 + kPage > least;
        wait_warp(&bar.s_full[turn & 1], (turn >> 1) & 1);
        tc_fence_after();
        float t[RG];
        if (ok) tmem_rows<RG, 1>(tmem + lane_off + (turn & 1) * kSBuf + r0, t);
        bool need = o_ratio != 1.f;
#pragma unroll
        for (int r = 0; r < RG; ++r) t[r] *= bar.c[r0 + r] * ks;
        if (partial) {
          // Slots that no token has reached may hold anything, and a product
          // takes every key for every row although 0 * NaN is NaN: those
          // slots become zero in the tile, and so does a NaN, which the rows
          // that see it get back at the end.
#pragma unroll
          for (int r = 0; r < RG; ++r)
            if (id < 0 || key0 + key >= bar.limit[r0 + r]) t[r] = -INFINITY;
        }
        if (partial && g == 0) {
          const uint32_t at = ring_base + v_tile(i, s.count);
          wait_warp(&bar.full[at % kFewRing], (at / kFewRing) & 1);
          uint4* row = reinterpret_cast<uint4*>(smem + L::kRingOff + (at % kFewRing) * kPageBytes + key * 128);
          const bool drop = id < 0 || key0 + key >= s.st.len;
          uint32_t nan = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (!ok) break;
            uint4 v = drop ? make_uint4(0, 0, 0, 0) : row[j];
            uint32_t hit = take_nan(v.x) | take_nan(v.y);
            hit |= take_nan(v.z) | take_nan(v.w);
            if (drop || hit) row[j] = v;
            nan |= hit;
          }
          if (nan) *const_cast<volatile int*>(&bar.nan_seen) = 1;
        }
        float d[RG];
#pragma unroll
        for (int r = 0; r < RG; ++r) {
          d[r] = t[r] - m[r];
          need |= d[r] > kFewStale;
        }
        if (vote_128(2 + g, need)) {
          // new maxima over the page, the same for the four warps; O is
          // rescaled, once its product with the page before is complete (the
          // one before that is: S^T of this page was issued after it)
#pragma unroll
          for (int r = 0; r < RG; ++r) {
            float top = t[r];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (lane == 0) bar.top[quarter][r0 + r] = top;
          }
          named_bar_sync(4 + g, 128);
          float by[RG];
#pragma unroll
          for (int r = 0; r < RG; ++r) {
            const float now = fmaxf(fmaxf(m[r], fmaxf(bar.top[0][r0 + r], bar.top[1][r0 + r])),
                                    fmaxf(bar.top[2][r0 + r], bar.top[3][r0 + r]));
            const float alpha = ex2_approx(m[r] - now);
            m[r] = now;
            d[r] = t[r] - now;
            l[r] *= alpha;
            by[r] = alpha * o_ratio;
          }
          if (i > 0 && wait_warp(&bar.pv_done, (turn - 1) & 1)) {
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < kPParts * RG; j += 16) {
              const uint32_t col = tmem + lane_off + kOCol + g * kPParts * RG + j;
              uint32_t o[16];
              tmem_ld16_wait(col, o);
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (j + e < kPParts * RG) o[e] = __float_as_uint(__uint_as_float(o[e]) * by[(j + e) % RG]);
              tmem_st16(col, o);
            }
            tmem_wait_st();
          }
          named_bar_sync(4 + g, 128);  // top has been read
        }
        // P^T's row part * RG + r of a group. An e5m2 value is the upper byte of
        // an fp16 value, so the parts are that byte of the fp16 weight, of what
        // remains, and so on, the last one rounded; two rows at a time.
        constexpr int kOne = RG == 1;
        uint32_t x[(RG + 1) / 2][kPParts];  // bytes 1 and 3: rows r and r + 1
#pragma unroll
        for (int r = 0; r < RG; r += 2) {
          const float w0 = ex2_approx(d[r] + vref.log), w1 = kOne ? 0.f : ex2_approx(d[r + 1 - kOne] + vref.log);
          l[r] = __fmaf_rn(w0, vref.inv, l[r]);
          if (!kOne) l[r + 1 - kOne] = __fmaf_rn(w1, vref.inv, l[r + 1 - kOne]);
          __half2 rest = __floats2half2_rn(w0, w1);
#pragma unroll
          for (int i = 0; i < kPParts; ++i) {
            uint32_t& y = x[r / 2][i];
            y = *reinterpret_cast<const uint32_t*>(&rest);
            if (i + 1 == kPParts) y += 0x00800080u;
            if (i + 1 < kPParts) {
              y &= 0xff00ff00u;
              rest = __hsub2(rest, *reinterpret_cast<const __half2*>(&y));
            }
          }
        }
        uint8_t* pt = smem + L::kPOff + (turn & 1) * L::kPBytes + g * (kPParts * RG / 16) * kPPlane + key * 16;
        if constexpr (kOne) {
          const uint32_t y0 = __byte_perm(x[0][0], x[0][1], 0x51), y1 = __byte_perm(x[0][2], x[0][3], 0x51);
          *reinterpret_cast<uint32_t*>(pt) = __byte_perm(y0, y1, 0x5410);
        } else {
          static_assert(kOne || RG == 4 || RG == 8, "16 rows and parts fill 16 bytes");
#pragma unroll
          for (int j = 0; j < kPParts * RG / 16; ++j) {
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int row = j * 16 + e * 4, i = row / RG, r = row % RG / 2;
              y[e] = __byte_perm(x[r][i], x[r + 1][i], 0x7531);
            }
            *reinterpret_cast<uint4*>(pt + j * kPPlane) = make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
        fence_proxy_async();
        tc_fence_before();
        mbar_arrive(&bar.p_full[turn & 1]);
      }
      stage_v += 2 * s.count;
      // the stretch's result: every lane has its channel of all rows
      wait_warp(&bar.o_full, seg & 1);
      tc_fence_after();
      float o[RG];
      if (ok) tmem_rows<RG, kPParts>(tmem + lane_off + kOCol + g * kPParts * RG, o);
#pragma unroll
      for (int r = 0; r < RG; ++r) {
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], x);
        if (lane == 0) bar.sum[quarter][r0 + r] = l[r] * vref.damp();
      }
      named_bar_sync(1, kAll);
      const bool complete = s.count == s.pages;
      const bool patch = *const_cast<volatile int*>(&bar.nan_seen) != 0;
      float* out = part_of(part, blockIdx.x, s.pg > 0, kFewRows);
      if (ok && *abort_flag == 0) {
#pragma unroll
        for (int rr = 0; rr < RG; ++rr) {
          const int r = r0 + rr;
          if (r >= rows) break;
          const float sum = (bar.sum[0][r] + bar.sum[1][r]) + (bar.sum[2][r] + bar.sum[3][r]);
          float x = o[rr] * vref.unit();
          if (patch && stretch_nan(p, s, bar.limit[r], least, key)) x = NAN;
          if (complete) {
            const int64_t at = static_cast<int64_t>(s.head * p.group + r % p.group) * p.n + s.st.t0 + r / p.group;
            const bool some = sum != 0.f;
            p.o[at * 128 + key] = __float2bfloat16_rn(some ? x / sum : 0.f);
            if (p.lse && key == 0) p.lse[at] = some ? (m[rr] + vref.raise() + log2f(sum)) * kLn2 : -INFINITY;
          } else {
            out[r * 128 + key] = sum != 0.f ? x : 0.f;
            if (key == 0)
              *reinterpret_cast<float2*>(out + kFewRows * 128 + 2 * r) =
                  make_float2(sum != 0.f ? m[rr] + vref.raise() : -INFINITY, sum);
          }
        }
      }
      tc_fence_before();
      named_bar_sync(1, kAll);  // limit, sum and nan_seen have been read
      if (all == 0) bar.nan_seen = 0;
      ++seg;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem, kFewCols);
  }
}

template <bool SW, int RG, int G>
int launch_few(const CUtensorMap& mk, const CUtensorMap& mv, const CacheAttnParams& p, const SharePlan& plan, float* ws,
               cudaStream_t stream) {
  static PerDeviceOnce once;
  const int rc =
      set_max_smem_once(reinterpret_cast<const void*>(cache_few_kernel<SW, RG, G>), FewLayout::kDynSmem, once);
  if (rc != CALIBATT_OK) return rc;
  cache_few_kernel<SW, RG, G><<<plan.ctas, few_threads(G), FewLayout::kDynSmem, stream>>>(mk, mv, p, plan.whole, ws);
  return cudaGetLastError() == cudaSuccess ? CALIBATT_OK : CALIBATT_ERR_CUDA;
}

template <bool SW>
int launch_few_rows(const CUtensorMap& mk, const CUtensorMap& mv, const CacheAttnParams& p, const SharePlan& plan,
                    float* ws, cudaStream_t stream) {
  if (plan.rows <= 1) return launch_few<SW, 1, 1>(mk, mv, p, plan, ws, stream);
  if (plan.rows <= 4) return launch_few<SW, 4, 1>(mk, mv, p, plan, ws, stream);
  if (plan.rows <= 8) return launch_few<SW, 4, 2>(mk, mv, p, plan, ws, stream);
  return launch_few<SW, 8, 2>(mk, mv, p, plan, ws, stream);
}

}  // namespace

int launch_cache_attn_few(const CacheAttnParams& p, const SharePlan& plan, void* ws, cudaStream_t stream) {
  CUtensorMap mk, mv;
  int rc = make_page_map(&mk, p.k8, p);
  if (rc == CALIBATT_OK) rc = make_page_map(&mv, p.v8, p);
  if (rc != CALIBATT_OK) return rc;
  float* part = static_cast<float*>(ws);
  rc = p.wait_limit_ns < kShortWaitNs ? launch_few_rows<true>(mk, mv, p, plan, part, stream)
                                      : launch_few_rows<false>(mk, mv, p, plan, part, stream);
  return rc != CALIBATT_OK || plan.whole ? rc : launch_cache_join(p, plan, part, kFewRows, stream);
}

}  // namespace calibatt
