// Attention over the paged 8-bit cache for few query rows (up to 16 that share
// a key head: one token of up to 16 query heads, a few tokens of a head).
//
// Bound by reading the cache once. Its pages are one list, stream by stream,
// key head by key head, cut into equal shares: two CTAs per SM, whatever the
// streams' lengths are (they are read on the device), so no SM waits for a
// long stream. A CTA (4 warps) walks its share; each warp takes 32 of a page's
// 128 keys, brings their K and V (8 KB) by TMA into a ring of its own, two
// pages ahead, and keeps its own running softmax: the warps meet only when a
// (stream, key head) or the share ends, and are joined there. (With a fifth
// warp as the producer the registers of three warps would share one of the
// SM's four partitions: 168 a thread instead of 255, and the rest spilled.)
// A stretch that is not all of its stream's pages leaves maximum, sum and
// unnormalised output in the workspace, and cache_few_join_kernel joins them.
//
// Products are mma.sync with the 16 rows as M. Fragments are read from shared
// memory 16 bytes at a time: the order of the contracted channels, and of the
// output channels, is free as long as both operands agree, so it is chosen to
// make a lane's share 16 consecutive bytes of a row.
//
// K and V are fp16 operands: every e4m3 value is an fp16 value. A row of Q is
// brought to fp16 by a power of two that puts its largest value into [1, 2)
// (rounding only what is below 2^-14 of it, by 2^-25 at most); that power, the
// page's key scale and the softmax scale multiply the fp32 score. The output
// stays in units of a reference value scale and relative to a running maximum
// that may be up to 2^8 stale, so most pages add their products to it and
// touch it in no other way (VRef below); P is fp16.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "cache.cuh"
#include "calibatt.h"
#include "kernels.h"
#include "ptx.cuh"
#include "sched.cuh"
#include "softmax.cuh"

namespace calibatt {
namespace {

constexpr int kFewWarps = 4;
constexpr int kFewThreads = 32 * kFewWarps;
constexpr int kFewStages = 2;
constexpr int kSliceKeys = kPage / kFewWarps;
constexpr int kSliceBytes = kSliceKeys * 128;
constexpr int kFewPartFloats = kFewRows * 128 + 2 * kFewRows;  // a partial result: O, then maximum and sum per row

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

// Normalises and stores a row's four channels of a lane; no key seen: 0 and -inf.
__device__ __forceinline__ void store_row(const CacheAttnParams& p, int64_t at, int lane, float mx, float sum,
                                          const float4& o) {
  const bool some = sum != 0.f;
  const float inv = some ? 1.f / sum : 0.f;
  uint2 w = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (!some) w = make_uint2(0, 0);
  *reinterpret_cast<uint2*>(p.o + at * 128 + lane * 4) = w;
  if (p.lse && lane == 0) p.lse[at] = some ? (mx + log2f(sum)) * kLn2 : -INFINITY;
}

struct FewShared {
  uint64_t full[kFewWarps][kFewStages];
  int abort;
  float m[kFewWarps][kFewRows], l[kFewWarps][kFewRows];
  alignas(16) float o[kFewWarps][kFewRows][132];  // padded: lanes of a quad write 32 channels apart
};
constexpr int kFewRingBytes = kFewWarps * kFewStages * 2 * kSliceBytes;
constexpr int kFewDynSmem = kFewRingBytes + static_cast<int>(sizeof(FewShared)) + 1024;

// 2D tiled load of one box into shared memory, completing on `bar`.
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y)
      : "memory");
}

// Pages of stream b that its last new token sees (at least one, so that rows
// which see nothing are written), 0 for a stream without new tokens.
__device__ __forceinline__ int stream_pages(const CacheAttnParams& p, const Stream& st) {
  if (st.bad || st.n_new == 0 || st.n_new > p.max_new || st.n_new * p.group > kFewRows) return 0;
  return max(1, (visible(st.len - 1, st.len, p.unit) + kPage - 1) / kPage);
}

// The list of all (stream, key head, page) triples.
struct PageList {
  // its length; every lane of the warp gets it
  static __device__ int64_t total(const CacheAttnParams& p, int lane) {
    int64_t sum = 0;
    for (int b = lane; b < p.batch; b += 32)
      sum += stream_pages(p, stream_of(p.tok_start, p.kv_len, b, p.n, p.table_stride));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum * p.heads_kv;
  }
  // the stream of entry w, and the entry that its pages begin at
  static __device__ int find(const CacheAttnParams& p, int64_t w, int lane, int64_t& begin) {
    begin = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      int64_t mine = 0;
      if (b0 + lane < p.batch)
        mine = static_cast<int64_t>(p.heads_kv) *
               stream_pages(p, stream_of(p.tok_start, p.kv_len, b0 + lane, p.n, p.table_stride));
      int64_t end = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, end, o);
        if (lane >= o) end += y;
      }
      const unsigned behind = __ballot_sync(0xffffffffu, begin + end > w);
      if (behind) {
        const int at = __ffs(behind) - 1;
        begin += __shfl_sync(0xffffffffu, end - mine, at);
        return b0 + at;
      }
      begin += __shfl_sync(0xffffffffu, end, 31);
    }
    return p.batch;
  }
};

// First entry of CTA c's share of `total` entries.
__device__ __forceinline__ int64_t share_begin(int64_t total, int c, int ctas) { return total * c / ctas; }

// A CTA's walk: consecutive pages pg .. pg + count - 1 of one stream and head.
struct Stretch {
  int b, head, pg, count, pages;
  Stream st;
};

struct Walk {
  int64_t w, end;
  int b, head, pg, pages;
  Stream st;

  __device__ __forceinline__ void load_stream(const CacheAttnParams& p) {
    st = stream_of(p.tok_start, p.kv_len, b, p.n, p.table_stride);
    pages = stream_pages(p, st);
  }
  __device__ void start(const CacheAttnParams& p, bool whole, int lane) {
    if (whole) {
      b = blockIdx.x / p.heads_kv;
      head = blockIdx.x % p.heads_kv;
      pg = 0;
      load_stream(p);
      w = 0;
      end = pages;
      return;
    }
    const int64_t total = PageList::total(p, lane);
    w = share_begin(total, blockIdx.x, gridDim.x);
    end = share_begin(total, blockIdx.x + 1, gridDim.x);
    if (w >= end) return;
    int64_t begin;
    b = PageList::find(p, w, lane, begin);
    load_stream(p);
    head = static_cast<int>((w - begin) / pages);
    pg = static_cast<int>((w - begin) % pages);
  }
  __device__ bool next(const CacheAttnParams& p, Stretch& s) {
    if (w >= end) return false;
    s.b = b;
    s.head = head;
    s.pg = pg;
    s.pages = pages;
    s.st = st;
    s.count = static_cast<int>(min(static_cast<int64_t>(pages - pg), end - w));
    w += s.count;
    if (w < end) {
      pg = 0;
      if (++head == p.heads_kv) {
        head = 0;
        do {
          ++b;
          load_stream(p);
        } while (pages == 0);
      }
    }
    return true;
  }
};

template <bool SW>
__global__ void __launch_bounds__(kFewThreads, 2)
    cache_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ CacheAttnParams p, bool whole, float* part) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* ring = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  FewShared& sh = *reinterpret_cast<FewShared*>(ring + kFewRingBytes);
  volatile int* abort_flag = &sh.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kFewWarps * kFewStages; ++i) mbar_init(&sh.full[0][0] + i, 1);
    sh.abort = 0;
    fence_barrier_init();
  }
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // streams that do not fit are reported once
  if (blockIdx.x == 0 && warp == 0)
    for (int b = lane; b < p.batch; b += 32) {
      const Stream st = stream_of(p.tok_start, p.kv_len, b, p.n, p.table_stride);
      if (st.bad || st.n_new > p.max_new || st.n_new * static_cast<int64_t>(p.group) > kFewRows)
        record_error(p.status, CALIBATT_ERR_CSR);
    }

  Walk walk, ahead;
  walk.start(p, whole, lane);
  ahead = walk;

  // the warp's loads, kFewStages pages ahead of its products
  uint8_t* slices = ring + warp * kFewStages * 2 * kSliceBytes;
  uint64_t* full = sh.full[warp];
  Stretch to;
  int to_page = 0, to_ids = -1, to_next = -1, issued = 0;
  auto page_id = [&](const Stretch& s, int i) {
    return i < s.count && (s.pg + i) * kPage + warp * kSliceKeys < s.st.len
               ? __ldg(p.table + static_cast<int64_t>(s.b) * p.table_stride + s.pg + i)
               : -1;
  };
  bool more = ahead.next(p, to);
  if (more) to_next = page_id(to, lane);
  auto issue = [&]() {
    if (!more) return;
    if ((to_page & 31) == 0) {
      to_ids = to_next;
      to_next = page_id(to, to_page + 32 + lane);
    }
    const int id = __shfl_sync(0xffffffffu, to_ids, to_page & 31);
    if (lane == 0) {
      uint64_t* bar = full + issued % kFewStages;
      if (id >= 0 && id < p.n_pages) {
        uint8_t* dst = slices + (issued % kFewStages) * 2 * kSliceBytes;
        const int y = (id * p.heads_kv + to.head) * kPage + warp * kSliceKeys;
        mbar_arrive_expect_tx(bar, 2 * kSliceBytes);
        tma_load_2d(dst, &tm_k, bar, 0, y);
        tma_load_2d(dst + kSliceBytes, &tm_v, bar, 0, y);
      } else {
        mbar_arrive(bar);  // nothing to read: the products skip the page as well
      }
    }
    ++issued;
    if (++to_page == to.count) {
      to_page = 0;
      more = ahead.next(p, to);
      if (more) to_next = page_id(to, lane);
    }
  };
  for (int i = 0; i < kFewStages; ++i) issue();

  const int g = lane >> 2, t = lane & 3;
  int used = 0, seg = 0;
  Stretch s;
  bool ok = true;  // warp-uniform
  while (walk.next(p, s)) {
    const int rows = s.st.n_new * p.group;
    // pages' scales, one per lane, 32 pages at a time
    const int32_t* table = p.table + static_cast<int64_t>(s.b) * p.table_stride;
    int ids = -1, ids_next = -1;
    float kss = 0.f, vss = 0.f, kss_next = 0.f, vss_next = 0.f;
    auto fetch = [&](int i) {
      ids_next = i < s.count && s.st.len > (s.pg + i) * kPage ? __ldg(table + s.pg + i) : -1;
      if (ids_next >= p.n_pages) ids_next = -1;
      if (ids_next < 0) {
        if (i < s.count && s.st.len > (s.pg + i) * kPage) record_error(p.status, CALIBATT_ERR_CSR);
        ids_next = -1;
        return;
      }
      const int64_t at = static_cast<int64_t>(ids_next) * p.heads_kv + s.head;
      kss_next = __ldg(p.k_scale + at);
      vss_next = __ldg(p.v_scale + at);
    };
    fetch(lane);
    // rows g and g + 8: token r / group, query head head * group + r % group
    int limit[2];
    float c[2];
    uint32_t qa[8][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = min(g + 8 * i, rows - 1);
      const int tok = r / p.group, h = s.head * p.group + r % p.group;
      limit[i] = g + 8 * i < rows ? visible(s.st.len - s.st.n_new + tok, s.st.len, p.unit) : 0;
      float x[32];
      float amax = load_q_row(p.q + (static_cast<int64_t>(h) * p.n + s.st.t0 + tok) * 128, t, x);
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
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    VRef vref;
    float acc[16][4];
#pragma unroll
    for (int j = 0; j < 16; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;

    for (int pi = 0; pi < s.count; ++pi) {
      if ((pi & 31) == 0) {
        ids = ids_next;
        kss = kss_next;
        vss = vss_next;
        fetch(pi + 32 + lane);
      }
      const int id = __shfl_sync(0xffffffffu, ids, pi & 31);
      const float ks = __shfl_sync(0xffffffffu, kss, pi & 31), vs = __shfl_sync(0xffffffffu, vss, pi & 31);
      const int stage = used % kFewStages;
      if (ok)
        ok = __all_sync(0xffffffffu, mbar_wait<SW>(full + stage, (used / kFewStages) & 1, abort_flag, p.status,
                                                   p.wait_limit_ns));
      const int key0 = (s.pg + pi) * kPage + warp * kSliceKeys;
      if (ok && id >= 0 && key0 < s.st.len) {
        const uint8_t* kp = slices + stage * 2 * kSliceBytes;
        const uint8_t* vp = kp + kSliceBytes;
        // 16-byte chunk j of row r is at chunk j ^ (r & 7) (128-byte swizzle)
        // S = Q K^T
        float sc[4][4];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          const uint8_t* row = kp + (nt * 8 + g) * 128;
          const uint4 kw[2] = {*reinterpret_cast<const uint4*>(row + ((t ^ g) << 4)),
                               *reinterpret_cast<const uint4*>(row + (((4 + t) ^ g) << 4))};
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[nt][i] = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t w = word_of(kw[k >> 2], k & 3);
            mma_f16(sc[nt], qa[k], e4m3x2_to_half2(w & 0xffffu), e4m3x2_to_half2(w >> 16));
          }
        }
        uint4 vw[2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = k * 16 + 2 * t + (i & 1) + (i >> 1) * 8;
            vw[k][i] = *reinterpret_cast<const uint4*>(vp + r * 128 + ((g ^ (r & 7)) << 4));
          }
        const bool all = __all_sync(0xffffffffu, key0 + 32 <= limit[0] && key0 + 32 <= limit[1]);
        if (!all) {
#pragma unroll
          for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (key0 + nt * 8 + 2 * t + (i & 1) >= limit[i >> 1]) sc[nt][i] = -INFINITY;
          // slots that no token has reached may hold anything. A product
          // takes every key for every row, and 0 * NaN is NaN: a NaN value
          // of a key that some rows do not see is taken out of the product
          // and put into the rows that see it.
          uint32_t nan = 0;
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (key0 + k * 16 + 2 * t + (i & 1) + (i >> 1) * 8 >= s.st.len) vw[k][i] = make_uint4(0, 0, 0, 0);
              nan |= take_nan(vw[k][i].x) | take_nan(vw[k][i].y);
              nan |= take_nan(vw[k][i].z) | take_nan(vw[k][i].w);
            }
          if (__any_sync(0xffffffffu, nan != 0)) {
            for (int key = 0; key < 32 && key0 + key < s.st.len; ++key) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint8_t* row = vp + key * 128 + (((2 * t + e) ^ (key & 7)) << 4);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  if ((row[j] & 0x7f) == 0x7f) {
                    if (key0 + key < limit[0]) acc[j][e] = NAN;
                    if (key0 + key < limit[1]) acc[j][2 + e] = NAN;
                  }
              }
            }
          }
        }
        // online softmax of the warp's 32 keys. The running maximum is the
        // quad's (all lanes of a row agree) and moves only if it grew by more
        // than 2^8, or to a first value.
        const float o_ratio = vref.page(vs);
        float ck[2], page_max[2];
        bool need = o_ratio != 1.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          ck[i] = score_factor(c[i], ks);
          float mx = fmaxf(max3f(sc[0][2 * i], sc[0][2 * i + 1], sc[1][2 * i]),
                           max3f(sc[1][2 * i + 1], sc[2][2 * i], sc[2][2 * i + 1]));
          mx = max3f(mx, sc[3][2 * i], sc[3][2 * i + 1]);
          page_max[i] = mx;
          // a maximum of -inf is replaced by whatever is seen first
          need |= mx * ck[i] > m[i] + kStaleMax;
          need |= fabsf(mx * ck[i]) > kBigScore && mx != -INFINITY;
        }
        float add[2] = {vref.log - (m[0] == -INFINITY ? 0.f : m[0]), vref.log - (m[1] == -INFINITY ? 0.f : m[1])};
        if (__any_sync(0xffffffffu, need)) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float mx = page_max[i];
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float now = fmaxf(m[i], mx * ck[i]);
            const float use = now == -INFINITY ? 0.f : now;
            const float alpha = ex2_approx(m[i] - use);
            m[i] = now;
            l[i] *= alpha;
            const float by = alpha * o_ratio;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              acc[j][2 * i] *= by;
              acc[j][2 * i + 1] *= by;
            }
            // relative to the page's own largest score: scores of 2^24 and
            // more would leave the rounding of mx * ck in the exponent
            const float mx0 = mx == -INFINITY ? 0.f : mx;
            add[i] = (mx == -INFINITY ? 0.f : mx * ck[i] - use) + vref.log;
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
              sc[nt][2 * i] -= mx0;
              sc[nt][2 * i + 1] -= mx0;
            }
          }
        }
        uint32_t pa[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float sum = 0.f;
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            const float e0 = ex2_approx(__fmaf_rn(sc[nt][2 * i], ck[i], add[i]));
            const float e1 = ex2_approx(__fmaf_rn(sc[nt][2 * i + 1], ck[i], add[i]));
            sum += e0 + e1;
            pa[nt >> 1][(nt & 1) * 2 + i] = pack_half2(e0, e1);
          }
          l[i] = __fmaf_rn(sum, vref.inv, l[i]);
        }
        // O += P V, four output tiles at a time
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t pair[2][2][2][2];  // k16 step, operand half, pair of channels, packed fp16 of two keys
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const uint32_t x = word_of(vw[k][2 * hf], w), y = word_of(vw[k][2 * hf + 1], w);
              const uint32_t lo = __byte_perm(x, y, 0x5140), hi = __byte_perm(x, y, 0x7362);
              pair[k][hf][0][0] = e4m3x2_to_half2(lo & 0xffffu);
              pair[k][hf][0][1] = e4m3x2_to_half2(lo >> 16);
              pair[k][hf][1][0] = e4m3x2_to_half2(hi & 0xffffu);
              pair[k][hf][1][1] = e4m3x2_to_half2(hi >> 16);
            }
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              mma_f16(acc[w * 4 + j], pa[k], pair[k][0][j >> 1][j & 1], pair[k][1][j >> 1][j & 1]);
        }
      }
      __syncwarp();
      if (ok) {
        ++used;
        issue();
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    }
    // join the four warps: lane t of a quad holds channels 32t .. 32t+31
    named_bar_sync(1, 32 * kFewWarps);  // the last stretch's rows have been read
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (t == 0) {
        sh.m[warp][g + 8 * i] = m[i];
        sh.l[warp][g + 8 * i] = l[i];
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int j = 0; j < 16; ++j) sh.o[warp][g + 8 * i][32 * t + 16 * e + j] = acc[j][2 * i + e] * vref.unit();
    }
    named_bar_sync(1, 32 * kFewWarps);
    const bool complete = s.count == s.pages;
    float* out = part + (2 * static_cast<int64_t>(blockIdx.x) + (seg > 0)) * kFewPartFloats;
    for (int r = warp; r < rows && *abort_flag == 0; r += kFewWarps) {
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) mx = fmaxf(mx, sh.m[w][r]);
      const float use = mx == -INFINITY ? 0.f : mx;
      float sum = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) {
        const float f = ex2_approx(sh.m[w][r] - use);
        const float4 x = *reinterpret_cast<const float4*>(&sh.o[w][r][lane * 4]);
        sum += sh.l[w][r] * f;
        o.x += x.x * f;
        o.y += x.y * f;
        o.z += x.z * f;
        o.w += x.w * f;
      }
      if (complete) {
        const int64_t at =
            static_cast<int64_t>(s.head * p.group + r % p.group) * p.n + s.st.t0 + r / p.group;
        store_row(p, at, lane, mx, sum, o);
      } else {
        *reinterpret_cast<float4*>(out + r * 128 + lane * 4) = o;
        if (lane == 0) *reinterpret_cast<float2*>(out + kFewRows * 128 + 2 * r) = make_float2(mx, sum);
      }
    }
    ++seg;
  }
  // no copy may still be landing when the CTA leaves
  for (; used < issued; ++used) {
    volatile int never = 0;
    mbar_wait(full + used % kFewStages, (used / kFewStages) & 1, &never, p.status);
  }
}

// Joins the stretches of one (stream, key head): the CTAs whose shares meet
// its pages, in order. A warp per row.
__global__ void __launch_bounds__(128)
    cache_few_join_kernel(const __grid_constant__ CacheAttnParams p, int ctas, const float* part) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
  if (pages == 0) return;
  total *= p.heads_kv;
  const int64_t u0 = before * p.heads_kv + static_cast<int64_t>(head) * pages, u1 = u0 + pages;
  // the last CTA whose share begins at or before u0
  int c = static_cast<int>(u0 * ctas / total);
  while (c + 1 < ctas && share_begin(total, c + 1, ctas) <= u0) ++c;
  while (c > 0 && share_begin(total, c, ctas) > u0) --c;
  if (share_begin(total, c + 1, ctas) >= u1) return;  // one CTA had all of them and wrote the result
  const int rows = st.n_new * p.group;
  for (int r = warp; r < rows; r += 4) {
    float mx = -INFINITY, sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    int64_t w0;
    for (int i = c; i < ctas && (w0 = share_begin(total, i, ctas)) < u1; ++i) {
      if (w0 == share_begin(total, i + 1, ctas)) continue;  // an empty share
      // a CTA's first stretch is in its first slot, its last in the second
      const float* at = part + (2 * static_cast<int64_t>(i) + (w0 < u0)) * kFewPartFloats;
      const float2 ml = *reinterpret_cast<const float2*>(at + kFewRows * 128 + 2 * r);
      const float4 x = *reinterpret_cast<const float4*>(at + r * 128 + lane * 4);
      const float now = fmaxf(mx, ml.x);
      const float use = now == -INFINITY ? 0.f : now;
      const float f0 = ex2_approx(mx - use), f1 = ex2_approx(ml.x - use);
      sum = sum * f0 + ml.y * f1;
      o.x = o.x * f0 + x.x * f1;
      o.y = o.y * f0 + x.y * f1;
      o.z = o.z * f0 + x.z * f1;
      o.w = o.w * f0 + x.w * f1;
      mx = now;
    }
    store_row(p, static_cast<int64_t>(head * p.group + r % p.group) * p.n + st.t0 + r / p.group, lane, mx, sum, o);
  }
}

// 128-byte rows of the cache's pages, boxes of a warp's share of a page with the 128-byte swizzle.
int make_page_map(CUtensorMap* map, const void* base, int64_t rows) {
  EncodeTiledFn enc = get_encode();
  if (!enc) return CALIBATT_ERR_CUDA;
  cuuint64_t dims[2] = {128, static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {128};
  cuuint32_t box[2] = {128, kSliceKeys};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? CALIBATT_OK : CALIBATT_ERR_CUDA;
}

template <bool SW>
int launch_few(const CUtensorMap& mk, const CUtensorMap& mv, const CacheAttnParams& p, const FewPlan& plan, float* ws,
               cudaStream_t stream) {
  static PerDeviceOnce once;
  const int rc =
      set_max_smem_once(reinterpret_cast<const void*>(cache_few_kernel<SW>), kFewDynSmem, once);
  if (rc != CALIBATT_OK) return rc;
  cache_few_kernel<SW><<<plan.ctas, kFewThreads, kFewDynSmem, stream>>>(mk, mv, p, plan.whole, ws);
  return cudaGetLastError() == cudaSuccess ? CALIBATT_OK : CALIBATT_ERR_CUDA;
}

}  // namespace

FewPlan few_plan(int batch, int heads_kv, int64_t pages, int sms) {
  const int64_t units = static_cast<int64_t>(batch) * heads_kv;
  FewPlan f;
  // up to 4 pages the join costs more than the split saves
  f.whole = pages <= 4;
  f.ctas = static_cast<int>(f.whole ? units : std::min<int64_t>(2ll * sms, units * ((pages + 1) / 2)));
  return f;
}

size_t few_workspace_bytes(const FewPlan& plan) {
  return plan.whole ? 0 : 2 * static_cast<size_t>(plan.ctas) * kFewPartFloats * sizeof(float);
}

int launch_cache_attn_few(const CacheAttnParams& p, const FewPlan& plan, void* ws, cudaStream_t stream) {
  CUtensorMap mk, mv;
  const int64_t rows = static_cast<int64_t>(p.n_pages) * p.heads_kv * kPage;
  if (rows > INT32_MAX) return CALIBATT_ERR_UNSUPPORTED;
  // an empty pool is never read: the maps need an address all the same
  int rc = make_page_map(&mk, rows ? static_cast<const void*>(p.k8) : p.q, rows ? rows : kPage);
  if (rc == CALIBATT_OK) rc = make_page_map(&mv, rows ? static_cast<const void*>(p.v8) : p.q, rows ? rows : kPage);
  if (rc != CALIBATT_OK) return rc;
  float* part = static_cast<float*>(ws);
  rc = p.wait_limit_ns < kShortWaitNs ? launch_few<true>(mk, mv, p, plan, part, stream)
                                      : launch_few<false>(mk, mv, p, plan, part, stream);
  if (rc != CALIBATT_OK || plan.whole) return rc;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.heads_kv, p.batch);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  // resident while the pages are still read: it waits in the kernel
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_few_join_kernel, p, plan.ctas, static_cast<const float*>(part)) == cudaSuccess
             ? CALIBATT_OK
             : CALIBATT_ERR_CUDA;
}

}  // namespace calibatt
