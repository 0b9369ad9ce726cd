// Attention over the paged 8-bit cache for many query rows (more than 16 that
// share a key head), on the sm_100a tensor core.
//
// The work is one list, stream by stream, key head by key head, row tile by
// row tile, page by page, cut into shares of equal cost for one CTA per SM
// whatever the streams' lengths are (they are read on the device): no SM waits
// for a long stream or a last wave. A segment of a share that is not all pages
// of its tile leaves maximum, sum and unnormalised output in the workspace,
// and cache_tile_join_kernel joins them.
//
// CTA (512 threads, persistent):
//   warps 0-3, 4-7   softmax of slot 0 and slot 1 (thread = query row = TMEM lane)
//   warps 8-11       converters: e4m3 tiles to fp16 operand tiles in a
//                    shared-memory ring (128-byte swizzle)
//   warp  12         MMA issuer (one thread): S = Q K^T and O += P V
//   warp  13         TMA producer of the e4m3 tiles (kAlt)
//   warp  14         scheduler: walks the share and hands out its segments
//   warp  15         idle
// The fourth warpgroup's registers go to the softmax warpgroups.
// A slot is 128 query rows. With more than 128 rows a CTA takes 256: each
// converted tile feeds both slots, so the conversion (on the same issue slots
// as the softmax) is paid once per two tensor-core tiles. With at most 128
// (kAlt) the slots hold the same rows and take every other page, and are
// joined at a segment's end: the chain S -> softmax -> P V of one slot then
// runs beside the other's.
// With 256 rows the pages mostly come from L2 and the converters load them
// straight into registers, two tiles ahead, beside two Q tiles and 5 operand
// tiles. With 128 the kernel waits for the cache's bytes: there, without the
// second Q tile, the e4m3 tiles come by TMA, 4 ahead (65 % of the time).
//
// K and V become fp16 without their scales: fp16 holds every e4m3 value, and
// the conversion is one instruction per two values (with the scale in it, as
// bf16, it took five and the converters, not the tensor core, set the pace).
// Q is brought to fp16 by a power of two per row; that and the key scale
// multiply the fp32 score. P is fp16; O is kept in units of a reference value
// scale (VRef), so a page's value scale costs nothing either.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "cache.cuh"
#include "calibatt.h"
#include "kernels.h"
#include "ptx.cuh"
#include "sched.cuh"
#include "softmax.cuh"

namespace calibatt {
namespace {

constexpr int kTileThreads = 512;
// registers per thread after the split; their sum must fit in the launch
// allotment of 128 x 512 (checked against the compiled count before a launch)
constexpr int kTileSoftmaxRegs = 192;
constexpr int kTileConvertRegs = 88;
constexpr int kTileControlRegs = 40;
constexpr int kTileRegs = 256 * kTileSoftmaxRegs + 128 * kTileConvertRegs + 128 * kTileControlRegs;
static_assert(kTileRegs <= 128 * kTileThreads, "register split");
constexpr float kStaleMax = 8.0f;      // log2 units: move the running max only if it grows by more
constexpr float kBigScore = 65536.0f;  // log2 units: beyond it the rounding of the row max counts
constexpr int kRawBytes = kPage * 128;
constexpr int kRaw = 4;                // e4m3 tiles in flight (kAlt)
constexpr int kSegs = 2;               // segments handed out ahead
constexpr int kNanSlots = 8;           // converters are never that many segments ahead of the softmax

// Consecutive pages pg0 .. pg0 + np - 1 of a row tile; np = 0 ends the share.
struct Segment {
  int b, head, t0, n_new, len;
  int r0, r1;     // rows of the tile
  int least;      // keys that every row sees
  int pg0, np;
  int pages;      // of the tile
  int number;     // of the segment in its share
};

template <bool kAlt>
struct TileLayout {
  static constexpr int kRing = kAlt ? 4 : 5;
  static constexpr int kQOff = 0;
  static constexpr int kRawOff = kTile;  // kAlt only, in the place of the second Q tile and a ring stage
  static constexpr int kRingOff = kAlt ? kRawOff + kRaw * kRawBytes : 2 * kTile;
  static constexpr int kBarOff = kRingOff + kRing * kTile;
};

struct TileBarriers {
  uint64_t ring_full[5], ring_empty[5];
  uint64_t raw_full[kRaw], raw_empty[kRaw];
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t q_full[2];
  uint64_t s_full[2];
  uint64_t p_full[2][2];  // per slot, per half of the page's keys
  uint64_t o_full[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
  int go[2];                // kAlt: whether the softmax warps got segment k (k even, odd)
  int raw_bad[kRaw];        // the tile's page is outside the pool: nothing was loaded
  int nan_seen[kNanSlots];  // 1 + number of the segment in which a NaN value was taken out of a page
  float2 slot_ml[128];      // kAlt: slot 1's maximum and sum
  Segment seg[kSegs];
};

template <bool kAlt>
constexpr int tile_smem() {
  return TileLayout<kAlt>::kBarOff + static_cast<int>(sizeof(TileBarriers)) + 1024;
}
static_assert(tile_smem<false>() <= 232448 && tile_smem<true>() <= 232448, "shared memory budget");

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

// ------------------------------------------------------------------ the list of work
template <bool kAlt>
struct Tiles {
  static constexpr int kRows = kAlt ? 128 : 256;

  static __device__ __forceinline__ int count(const CacheAttnParams& p, const Stream& st) {
    if (st.bad || st.n_new > p.max_new) return 0;
    return (st.n_new * p.group + kRows - 1) / kRows;
  }
  // Pages of tile t: those that its last row sees, and one at least, so that
  // rows which see nothing are written.
  static __device__ __forceinline__ int pages(const CacheAttnParams& p, const Stream& st, int t) {
    const int last = min(st.n_new * p.group, (t + 1) * kRows) - 1;
    return max(1, (visible(st.len - st.n_new + last / p.group, st.len, p.unit) + kPage - 1) / kPage);
  }
  // Cost of a page: a tile of which only slot 0 has rows takes about 3/4 of
  // the time. With `whole`, a tile is one piece that costs 1.
  static __device__ __forceinline__ int weight(const Stream& st, const CacheAttnParams& p, int t) {
    return kAlt || min(st.n_new * p.group, (t + 1) * kRows) - t * kRows > 128 ? 4 : 3;
  }
  static __device__ __forceinline__ int64_t cost(const CacheAttnParams& p, const Stream& st, int t, bool whole) {
    return whole ? 1 : static_cast<int64_t>(pages(p, st, t)) * weight(st, p, t);
  }
  // Cost of one key head of a stream: all its tiles.
  static __device__ int64_t head_cost(const CacheAttnParams& p, const Stream& st, bool whole) {
    const int n = count(p, st);
    if (n == 0) return 0;
    if (whole) return n;
    if (p.unit == 0) return (n - 1) * cost(p, st, 0, false) + cost(p, st, n - 1, false);
    int64_t sum = 0;
    for (int t = 0; t < n; ++t) sum += cost(p, st, t, false);
    return sum;
  }
  static __device__ __forceinline__ int64_t warp_sum(int64_t x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
  }
  // Cost of streams 0 .. end - 1, for every lane of the warp.
  static __device__ int64_t total(const CacheAttnParams& p, int end, bool whole, int lane) {
    int64_t sum = 0;
    for (int b = lane; b < end; b += 32)
      sum += head_cost(p, stream_of(p.tok_start, p.kv_len, b, p.n, p.table_stride), whole);
    return warp_sum(sum) * p.heads_kv;
  }
  // The stream in which cost w falls, and the cost that it begins at.
  static __device__ int find(const CacheAttnParams& p, int64_t w, bool whole, int lane, int64_t& begin) {
    begin = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      int64_t mine = 0;
      if (b0 + lane < p.batch)
        mine = p.heads_kv *
               head_cost(p, stream_of(p.tok_start, p.kv_len, b0 + lane, p.n, p.table_stride), whole);
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

// Pages of a tile that begins at cost u0 which lie before cost w of the list:
// every share takes the pages from its beginning's to its end's.
__device__ __forceinline__ int pages_before(int64_t w, int64_t u0, int pages, int weight, bool whole) {
  if (w <= u0) return 0;
  if (whole) return pages;
  const int64_t n = (w - u0 + weight - 1) / weight;
  return n < pages ? static_cast<int>(n) : pages;
}

template <bool SW, bool kAlt>
__global__ void __launch_bounds__(kTileThreads, 1)
    cache_tile_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ CacheAttnParams p, bool whole, float* part) {
  using L = TileLayout<kAlt>;
  using T = Tiles<kAlt>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const uint32_t sbase = smem_u32(smem);
  TileBarriers& bar = *reinterpret_cast<TileBarriers*>(smem + L::kBarOff);
  volatile int* abort_flag = &bar.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kRing; ++i) {
      mbar_init(&bar.ring_full[i], 128);
      mbar_init(&bar.ring_empty[i], 1);
    }
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(&bar.raw_full[i], 1);
      mbar_init(&bar.raw_empty[i], 4);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&bar.seg_full[i], 1);
      mbar_init(&bar.seg_empty[i], kAlt ? 14 : 13);  // softmax, converter and issuer warps, and the producer
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar.q_full[s], 128);
      mbar_init(&bar.s_full[s], 1);
      mbar_init(&bar.p_full[s][0], 128);
      mbar_init(&bar.p_full[s][1], 128);
      mbar_init(&bar.o_full[s], 1);
    }
    mbar_init(&bar.mma_done, 1);
    bar.abort = 0;
    for (int i = 0; i < kNanSlots; ++i) bar.nan_seen[i] = 0;
    fence_barrier_init();
  }
  if (warp == 12) tmem_alloc(&bar.tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem_base;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // Waits for segment k: false at the share's end or after a failed wait. A
  // warp reads the segment where it lies, to spare registers, and gives its
  // place back when it is done with it.
  auto has_segment = [&](int k) -> bool {
    return mbar_wait<SW>(&bar.seg_full[k % kSegs], (k / kSegs) & 1, abort_flag, p.status, p.wait_limit_ns) &&
           bar.seg[k % kSegs].np > 0;
  };

  if (warp >= 8 && warp < 12) {
    // ---------------------------------------------------------- converters
    warpgroup_regs_dec<kTileConvertRegs>();
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    auto wait_warp = [&](uint64_t* bb, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait<SW>(bb, parity, abort_flag, p.status, p.wait_limit_ns));
    };
    // Cleans a V tile of a page that some row does not see whole: a product
    // takes every key for every row, and 0 * NaN is NaN. Slots behind the last
    // token become zero, and so does a NaN, which the rows that see it get
    // back at the end.
    auto clean = [&](const Segment& seg, int key0, int row, bool bad, uint4 (&w)[8]) {
      uint32_t nan = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int key = key0 + (e >> 1) * 32 + row;
        uint32_t* x = reinterpret_cast<uint32_t*>(&w[e]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (bad || key >= seg.len) x[k] = 0;
          nan |= take_nan(x[k]);
        }
      }
      if (nan) *const_cast<volatile int*>(&bar.nan_seen[seg.number % kNanSlots]) = seg.number + 1;
    };
    auto store = [&](int row, int quarter, const uint4 (&w)[8]) -> bool {
      if (!wait_warp(&bar.ring_empty[stage], phase ^ 1)) return false;
      const uint32_t dst = sbase + L::kRingOff + stage * kTile + row * 128;
#pragma unroll
      for (int e = 0; e < 8; ++e) store_half(dst + (e & 1) * kHalf + (e >> 1) * (32 * 128), row, 2 * quarter, w[e]);
      fence_proxy_async();
      mbar_arrive(&bar.ring_full[stage]);
      if (++stage == L::kRing) {
        stage = 0;
        phase ^= 1;
      }
      return true;
    };
    uint32_t raw_stage = 0, raw_phase = 0;
    for (int k = 0; ok && __all_sync(0xffffffffu, has_segment(k)); ++k) {
      const Segment& seg = bar.seg[k % kSegs];
      const int np = seg.np;
      if constexpr (kAlt) {
        // Eight lanes are four 16-byte chunks of two rows r and r ^ 5 of a
        // group of eight: with the swizzle their loads and both their stores
        // then fall into eight different groups of banks.
        const int pair = lane >> 3, quarter = lane & 3;
        const int row = (warp - 8) * 8 + ((lane & 4) ? pair ^ 5 : pair);
        for (int t = 0; t < 2 * np && ok; ++t) {
          bool is_v;
          int i;
          ring_tile<true>(t, np, is_v, i);
          if (!(ok = wait_warp(&bar.raw_full[raw_stage], raw_phase))) break;
          const uint8_t* src = smem + L::kRawOff + raw_stage * kRawBytes + row * 128;
          uint4 w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            w[e] = *reinterpret_cast<const uint4*>(src + (e >> 1) * (32 * 128) +
                                                   ((((e & 1) * 4 + quarter) ^ (row & 7)) << 4));
          const int key0 = (seg.pg0 + i) * kPage;
          const bool bad = bar.raw_bad[raw_stage] != 0;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.raw_empty[raw_stage]);
          if (++raw_stage == kRaw) {
            raw_stage = 0;
            raw_phase ^= 1;
          }
          if (is_v && (bad || key0 + kPage > seg.least)) clean(seg, key0, row, bad, w);
          ok = store(row, quarter, w);
        }
      } else {
        // Eight lanes are four chunks of an even and an odd row: their stores
        // fall into eight different groups of banks.
        const int row = (warp - 8) * 8 + (lane >> 2), quarter = lane & 3;
        PageWindow<false> win(p, seg.b, seg.head, seg.pg0, np, seg.len);
        win.fetch(lane, p.status);
        int id_now = -1;  // page of the latest K tile; its V tile is the next one
        uint4 buf[2][8];
        auto load = [&](int t, uint4 (&w)[8]) {
          const bool is_v = t & 1;
          const int i = t >> 1;
          if (!is_v) {
            if ((i & 31) == 0) win.advance(i, lane, p.status);
            id_now = __shfl_sync(0xffffffffu, win.id, i & 31);
          }
          if (id_now < 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = make_uint4(0, 0, 0, 0);
            return;
          }
          const uint8_t* src = (is_v ? p.v8 : p.k8) +
                               (static_cast<int64_t>(id_now) * p.heads_kv + win.head) * kRawBytes + row * 128 +
                               quarter * 16;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            w[e] = __ldg(reinterpret_cast<const uint4*>(src + (e >> 1) * (32 * 128) + (e & 1) * 64));
        };
        load(0, buf[0]);
        load(1, buf[1]);
        for (int i = 0; i < np && ok; ++i) {
          if (!(ok = store(row, quarter, buf[0]))) break;
          if (i + 1 < np) load(2 * i + 2, buf[0]);
          const int key0 = (seg.pg0 + i) * kPage;
          if (key0 + kPage > seg.least) clean(seg, key0, row, false, buf[1]);
          if (!(ok = store(row, quarter, buf[1]))) break;
          if (i + 1 < np) load(2 * i + 3, buf[1]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.seg_empty[k % kSegs]);
    }
  } else if (warp >= 12) {
    warpgroup_regs_dec<kTileControlRegs>();
    if (warp == 14) {
      // -------------------------------------------------------- scheduler
      if (blockIdx.x == 0)  // streams that do not fit are reported once
        for (int b = lane; b < p.batch; b += 32) {
          const Stream st = stream_of(p.tok_start, p.kv_len, b, p.n, p.table_stride);
          if (st.bad || st.n_new > p.max_new) record_error(p.status, CALIBATT_ERR_CSR);
        }
      const int64_t total = T::total(p, p.batch, whole, lane);
      const int64_t w0 = total * blockIdx.x / gridDim.x, w1 = total * (blockIdx.x + 1) / gridDim.x;
      int k = 0;
      bool ok = true;
      auto publish = [&](const Segment& seg) {
        if (lane == 0) {
          ok = mbar_wait<SW>(&bar.seg_empty[k % kSegs], ((k / kSegs) & 1) ^ 1, abort_flag, p.status, p.wait_limit_ns);
          if (ok) {
            bar.seg[k % kSegs] = seg;
            mbar_arrive(&bar.seg_full[k % kSegs]);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        ++k;
      };
      Segment seg;
      if (w0 < w1) {
        int64_t u0;
        int b = T::find(p, w0, whole, lane, u0);
        Stream st = stream_of(p.tok_start, p.kv_len, b, p.n, p.table_stride);
        const int64_t per_head = T::head_cost(p, st, whole);
        int head = static_cast<int>((w0 - u0) / per_head), t = 0;
        u0 += head * per_head;
        for (int64_t c; u0 + (c = T::cost(p, st, t, whole)) <= w0; ++t) u0 += c;
        while (ok && u0 < w1) {
          const int pages = T::pages(p, st, t), weight = T::weight(st, p, t);
          const int first = pages_before(w0, u0, pages, weight, whole);
          const int last = pages_before(w1, u0, pages, weight, whole);
          if (last > first) {
            seg.b = b;
            seg.head = head;
            seg.t0 = st.t0;
            seg.n_new = st.n_new;
            seg.len = st.len;
            seg.r0 = t * T::kRows;
            seg.r1 = min(st.n_new * p.group, seg.r0 + T::kRows);
            seg.least = visible(st.len - st.n_new + seg.r0 / p.group, st.len, p.unit);
            seg.pg0 = first;
            seg.np = last - first;
            seg.pages = pages;
            seg.number = k;
            publish(seg);
          }
          u0 += T::cost(p, st, t, whole);
          if (u0 >= w1) break;
          if (++t == T::count(p, st)) {
            t = 0;
            if (++head == p.heads_kv) {
              head = 0;
              do {
                ++b;
                st = stream_of(p.tok_start, p.kv_len, b, p.n, p.table_stride);
              } while (T::count(p, st) == 0);
            }
          }
        }
      }
      seg.np = 0;
      if (ok) publish(seg);
    } else if (kAlt && warp == 13) {
      // -------------------------------------------------------- TMA producer
      uint32_t stage = 0, phase = 0;
      int used = 0;
      bool ok = true;
      for (int k = 0; ok && __all_sync(0xffffffffu, has_segment(k)); ++k) {
        const Segment& seg = bar.seg[k % kSegs];
        PageWindow<false> win(p, seg.b, seg.head, seg.pg0, seg.np, seg.len);
        win.fetch(lane, p.status);
        // pages are met in order by K; V follows at most one page behind
        int id_now = -1, id_before = -1, k_at = 0;
        for (int t = 0; t < 2 * seg.np && ok; ++t) {
          bool is_v;
          int i, id;
          ring_tile<true>(t, seg.np, is_v, i);
          if (!is_v) {
            if ((i & 31) == 0) win.advance(i, lane, p.status);
            id_before = id_now;
            id_now = id = __shfl_sync(0xffffffffu, win.id, i & 31);
            k_at = i;
          } else {
            id = k_at == i ? id_now : id_before;
          }
          if (lane == 0) {
            ok = mbar_wait<SW>(&bar.raw_empty[stage], phase ^ 1, abort_flag, p.status, p.wait_limit_ns);
            if (ok) {
              bar.raw_bad[stage] = id < 0;
              if (id >= 0) {
                mbar_arrive_expect_tx(&bar.raw_full[stage], kRawBytes);
                tma_load_2d(smem + L::kRawOff + stage * kRawBytes, is_v ? &tm_v : &tm_k, &bar.raw_full[stage], 0,
                            (id * p.heads_kv + seg.head) * kPage);
              } else {
                mbar_arrive(&bar.raw_full[stage]);
              }
              ++used;
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (++stage == kRaw) {
            stage = 0;
            phase ^= 1;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.seg_empty[k % kSegs]);
      }
      // no copy may still be landing when the CTA leaves
      if (lane == 0)
        for (int i = used > kRaw ? used - kRaw : 0; i < used; ++i) {
          volatile int never = 0;
          mbar_wait(&bar.raw_full[i % kRaw], (i / kRaw) & 1, &never, p.status);
        }
    } else if (warp == 12 && lane == 0) {
      // -------------------------------------------------------- MMA issuer
      uint32_t stage = 0, phase = 0;
      uint32_t n_q[2] = {0, 0}, n_p[2] = {0, 0};
      const uint64_t qdesc0 = desc_k_base(sbase + L::kQOff);
      const uint64_t kdesc0 = desc_k_base(sbase + L::kRingOff);
      const uint64_t vdesc0 = desc_v_base(sbase + L::kRingOff);
      auto wait = [&](uint64_t* bb, uint32_t parity) {
        return mbar_wait<SW>(bb, parity, abort_flag, p.status, p.wait_limit_ns);
      };
      auto ring_wait = [&]() -> bool {
        if (!wait(&bar.ring_full[stage], phase)) return false;
        tc_fence_after();
        return true;
      };
      auto advance = [&]() {
        if (++stage == L::kRing) {
          stage = 0;
          phase ^= 1;
        }
      };
      auto ring_next = [&]() {
        mma_commit(&bar.ring_empty[stage]);
        advance();
      };
      auto issue_s = [&](int s) {
        const uint64_t qd = qdesc0 + (kAlt ? 0 : s) * (kTile >> 4), kd = kdesc0 + stage * (kTile >> 4);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_ss(tmem + s * 128, qd + desc_k_step(ks), kd + desc_k_step(ks), kIdescQK, ks > 0);
        mma_commit(&bar.s_full[s]);
      };
      // the first half of P's keys is multiplied while the second is computed
      auto issue_pv = [&](int s, bool first) -> bool {
        const uint32_t parity = n_p[s]++ & 1;
        if (!wait(&bar.p_full[s][0], parity)) return false;
        if (!ring_wait()) return false;
        const uint64_t vd = vdesc0 + stage * (kTile >> 4);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_ts(tmem + 256 + s * 128, tmem + s * 128 + ks * 8, vd + desc_v_step(ks), kIdescPVh,
                 (!first || ks > 0) ? 1u : 0u);
        if (!wait(&bar.p_full[s][1], parity)) return false;
        tc_fence_after();
#pragma unroll
        for (int ks = 4; ks < 8; ++ks)
          mma_ts(tmem + 256 + s * 128, tmem + s * 128 + ks * 8, vd + desc_v_step(ks), kIdescPVh, 1u);
        return true;
      };
      bool go = true;
      for (int k = 0; go && has_segment(k); ++k) {
        const Segment& seg = bar.seg[k % kSegs];
        const int np = seg.np;
        const bool second = kAlt ? np > 1 : seg.r1 - seg.r0 > 128;
        mbar_arrive(&bar.seg_empty[k % kSegs]);
        if (!(go = wait(&bar.q_full[0], n_q[0]++ & 1))) break;
        if constexpr (kAlt) {
          for (int i = 0; i < 2 && i < np && go; ++i) {
            if (!(go = ring_wait())) break;
            issue_s(i);
            ring_next();
          }
          for (int i = 0; i < np && go; ++i) {
            const int s = i & 1;
            if (!(go = issue_pv(s, i < 2))) break;
            ring_next();
            if (i + 2 < np) {
              if (!(go = ring_wait())) break;
              issue_s(s);
              ring_next();
            } else {
              mma_commit(&bar.o_full[s]);
            }
          }
        } else {
          const int ns = second ? 2 : 1;
          if (second && !(go = wait(&bar.q_full[1], n_q[1]++ & 1))) break;
          if (!(go = ring_wait())) break;
          for (int s = 0; s < ns; ++s) issue_s(s);
          ring_next();
          for (int i = 0; i < np && go; ++i) {
            // stage holds V of page i; K of the next page is one stage on
            for (int s = 0; s < ns && go; ++s) {
              if (!(go = issue_pv(s, i == 0))) break;
              const uint32_t v_stage = stage, v_phase = phase;
              if (i + 1 < np) {
                if (s == ns - 1)
                  ring_next();
                else
                  advance();
                if (!(go = ring_wait())) break;
                issue_s(s);
                if (s == ns - 1) {
                  ring_next();
                } else {
                  stage = v_stage;
                  phase = v_phase;
                }
              } else {
                mma_commit(&bar.o_full[s]);
                if (s == ns - 1) ring_next();
              }
            }
          }
        }
      }
      // every issued MMA has finished before tensor memory is released
      mma_commit(&bar.mma_done);
      volatile int never = 0;
      mbar_wait(&bar.mma_done, 0, &never, p.status);
    }
  } else {
    // ---------------------------------------------------------- softmax
    warpgroup_regs_inc<kTileSoftmaxRegs>();
    const int s = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t sc = tmem + lane_off + s * 128, oc = tmem + lane_off + 256 + s * 128;
    uint32_t n_s = 0, n_o[2] = {0, 0};
    // after a failed wait a segment is finished without waiting or touching
    // tensor memory, so that the warps still meet at its barriers
    bool ok = true;  // warp-uniform
    auto wait_warp = [&](uint64_t* bb, uint32_t parity) -> bool {
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait<SW>(bb, parity, abort_flag, p.status, p.wait_limit_ns));
      return ok;
    };
    for (int k = 0;; ++k) {
      if constexpr (kAlt) {
        // the two slots meet at barriers inside a segment: one warp asks for all
        if (warp == 0) {
          const bool more = __all_sync(0xffffffffu, ok && has_segment(k));
          if (lane == 0) bar.go[k & 1] = more;
        }
        named_bar_sync(2, 256);
        if (bar.go[k & 1] == 0) break;
      } else {
        if (!ok || !__all_sync(0xffffffffu, has_segment(k))) break;
      }
      const Segment& seg = bar.seg[k % kSegs];
      const int np = seg.np;
      const bool second = kAlt ? np > 1 : seg.r1 - seg.r0 > 128;  // slot 1 has work
      const bool active = s == 0 || second;
      const int r = seg.r0 + (kAlt ? 0 : s * 128) + row;
      const bool row_valid = r < seg.r1;
      const int tok = row_valid ? r / p.group : 0;
      const int64_t at = static_cast<int64_t>(seg.head * p.group + (row_valid ? r % p.group : 0)) * p.n + seg.t0 + tok;
      // a padded row sees all keys: it is computed and not stored
      const int limit = row_valid ? visible(seg.len - seg.n_new + tok, seg.len, p.unit) : seg.len;
      float m_run = -INFINITY, l_run = 0.f;
      VRef<6, -6> vref;  // P below 2^8 (stale maximum) * 2^6 * 2, fp16; 2^-24 * 2^6 * 2^-6 is its smallest value
      if (active) {
        // the row of Q to shared memory, as fp16 times a power of two (kAlt:
        // slot 0 does it for both)
        const uint4* src = reinterpret_cast<const uint4*>(p.q + at * 128);
        float amax = 0.f;
        uint4 w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          w[j] = row_valid ? __ldg(src + j) : make_uint4(0, 0, 0, 0);
          const uint32_t x[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            amax = max3f(amax, fabsf(__uint_as_float(x[e] << 16)), fabsf(__uint_as_float(x[e] & 0xffff0000u)));
        }
        const float shrink = row_shrink(amax, 0);
        const float c_row = p.scale_log2 / shrink;
        if (!kAlt || s == 0) {
          const uint32_t dst = sbase + L::kQOff + s * kTile + row * 128;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint32_t x[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              h[e] = pack_half2(__uint_as_float(x[e] << 16) * shrink, __uint_as_float(x[e] & 0xffff0000u) * shrink);
            st_shared16(dst + (j >> 3) * kHalf + (((j & 7) ^ (row & 7)) << 4), h[0], h[1], h[2], h[3]);
          }
          fence_proxy_async();
          mbar_arrive(&bar.q_full[s]);
        }
        PageWindow<true> win(p, seg.b, seg.head, seg.pg0, np, seg.len);
        win.fetch(lane, p.status);
        bool started = false;  // O holds a product of this segment
        for (int i = kAlt ? s : 0; i < np; i += kAlt ? 2 : 1) {
          if ((i & 31) < (kAlt ? 2 : 1)) win.advance(i & ~31, lane, p.status);
          const int id = __shfl_sync(0xffffffffu, win.id, i & 31);
          const float ck = score_factor(c_row, __shfl_sync(0xffffffffu, win.ks, i & 31));
          const float o_ratio = vref.page(__shfl_sync(0xffffffffu, win.vs, i & 31));
          if (!wait_warp(&bar.s_full[s], n_s & 1)) break;
          ++n_s;
          tc_fence_after();
          const int key0 = (seg.pg0 + i) * kPage;
          const int cut = id < 0 ? 0 : min(limit - key0, kPage);  // keys of the page that the row sees
          float sv[2][64];
          tmem_ld64_wait(sc, sv[0]);
          tmem_ld64_wait(sc + 64, sv[1]);
          if (__any_sync(0xffffffffu, cut < kPage)) {
#pragma unroll
            for (int e = 0; e < 128; ++e)
              if (e >= cut) sv[e >> 6][e & 63] = -INFINITY;
          }
          const float mx = fmaxf(row_max64(sv[0]), row_max64(sv[1]));
          const float page_max = mx * ck;
          const float m_new = fmaxf(m_run, page_max);
          // keep a stale running max unless it grew by more than the threshold
          const bool need = m_run == -INFINITY || m_new > m_run + kStaleMax;
          const float m_prev = m_run;
          if (need) m_run = m_new;
          const float m_use = m_run == -INFINITY ? 0.f : m_run;
          const float alpha = need ? ex2_approx(m_prev - m_use) : 1.f;
          // exponent s * ck - m; for very large scores relative to the page's
          // own maximum first, whose rounding would otherwise stay in it
          float mul = ck, add = vref.log - m_use;
          if (__any_sync(0xffffffffu, fabsf(m_use) > kBigScore)) {
            const float mx0 = mx == -INFINITY ? 0.f : mx;
#pragma unroll
            for (int e = 0; e < 128; ++e) sv[e >> 6][e & 63] = (sv[e >> 6][e & 63] - mx0) * ck;
            mul = 1.f;
            add = page_max - m_use + vref.log;
          }
          // O is rescaled before P is handed on. Its product with the page
          // before is complete: the commit that signalled S tracks every
          // earlier MMA.
          if (started && (o_ratio != 1.f || __any_sync(0xffffffffu, need))) {
            const float by = alpha * o_ratio;
#pragma unroll 1
            for (int cc = 0; cc < 8; ++cc) {
              uint32_t o[16];
              tmem_ld16_wait(oc + cc * 16, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * by);
              tmem_st16(oc + cc * 16, o);
            }
          }
          started = true;
          const float2 c2 = make_float2(mul, mul), n2 = make_float2(add, add);
          float2 a4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t pk[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float2 x = exp2_mufu2(ffma2(make_float2(sv[h][2 * e], sv[h][2 * e + 1]), c2, n2));
              a4[e & 3] = fadd2(a4[e & 3], x);
              pk[e] = pack_half2(x.x, x.y);
            }
            // P (fp16, two keys per column) over the first 64 columns of S
            tmem_st32(sc + h * 32, pk);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&bar.p_full[s][h]);
          }
          const float2 s01 = fadd2(a4[0], a4[1]), s23 = fadd2(a4[2], a4[3]);
          l_run = l_run * alpha + ((s01.x + s01.y) + (s23.x + s23.y)) * vref.inv;
        }
      }
      // the segment's products are complete; kAlt: the other slot's too, for
      // the exchange below uses Q's tile
      if (active) wait_warp(&bar.o_full[s], n_o[s] & 1);
      if (active) ++n_o[s];
      if (kAlt && second) {
        wait_warp(&bar.o_full[s ^ 1], n_o[s ^ 1] & 1);
        ++n_o[s ^ 1];
      } else if (kAlt && s == 1) {
        ++n_o[0];  // slot 0's alone
      }
      tc_fence_after();
      const bool done = ok && *abort_flag == 0;
      float f0 = vref.unit(), f1 = 0.f;
      // kAlt: slot 1 hands its rows to slot 0 through Q's tile,
      // [channel][row], 64 channels at a time
      float* joined = reinterpret_cast<float*>(smem + L::kQOff);
      if (kAlt && second) {
        if (s == 1) bar.slot_ml[row] = make_float2(m_run, l_run);
        named_bar_sync(1, 256);
        if (s == 0) {
          const float2 o = bar.slot_ml[row];
          const float mx = fmaxf(m_run, o.x);
          const float use = mx == -INFINITY ? 0.f : mx;
          const float g0 = ex2_approx(m_run - use);
          f1 = ex2_approx(o.x - use);
          l_run = l_run * g0 + o.y * f1;
          f0 *= g0;
          m_run = mx;
        }
      }
      const bool some = l_run != 0.f;
      const float inv = some ? 1.f / l_run : 0.f;
      const bool complete = np == seg.pages;
      // partial results: the first segment of a share begins inside its tile,
      // the last one at its first page
      float* out = part + (2 * static_cast<int64_t>(blockIdx.x) + (seg.pg0 > 0 ? 0 : 1)) * tile_part_floats(T::kRows);
      const int part_row = r - seg.r0;
      const bool write = done && row_valid && (kAlt ? s == 0 : active);
      if (write) {
        if (!complete)
          *reinterpret_cast<float2*>(out + T::kRows * 128 + 2 * part_row) = make_float2(m_run, some ? l_run : 0.f);
        else if (p.lse)
          p.lse[at] = some ? (m_run + log2f(l_run)) * kLn2 : -INFINITY;
      }
      const bool patch =
          *const_cast<volatile int*>(&bar.nan_seen[seg.number % kNanSlots]) == seg.number + 1;
#pragma unroll 1
      for (int cc = 0; cc < 4; ++cc) {
        uint32_t o[32];
        if (kAlt && second && (cc & 1) == 0) {
          if (cc > 0) named_bar_sync(1, 256);  // slot 0 has read the first half
          if (s == 1 && done) {
            const float unit = vref.unit();
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              tmem_ld32_wait(oc + (cc + hh) * 32, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) joined[(hh * 32 + e) * 128 + row] = __uint_as_float(o[e]) * unit;
            }
          }
          named_bar_sync(1, 256);
        }
        if (!done || (kAlt ? s == 1 : !active)) continue;
        tmem_ld32_wait(oc + cc * 32, o);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          float x = __uint_as_float(o[e]) * f0;
          if (kAlt && second) x += joined[((cc & 1) * 32 + e) * 128 + row] * f1;
          o[e] = __float_as_uint(x);
        }
        if (patch && row_valid) {
          // NaN values that were taken out of pages that not every row sees whole
          const int32_t* table = p.table + static_cast<int64_t>(seg.b) * p.table_stride;
          uint32_t bad = 0;
          for (int key = max(seg.least / kPage, seg.pg0) * kPage; key < min(limit, (seg.pg0 + np) * kPage); ++key) {
            const int id = __ldg(table + key / kPage);
            if (id < 0 || id >= p.n_pages) continue;
            const uint8_t* v = p.v8 + ((static_cast<int64_t>(id) * p.heads_kv + seg.head) * kPage + key % kPage) * 128;
            for (int e = 0; e < 32; ++e)
              if ((v[cc * 32 + e] & 0x7f) == 0x7f) bad |= 1u << e;
          }
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (bad >> e & 1) o[e] = 0x7fffffffu;
        }
        if (!row_valid) continue;
        if (!complete) {
          uint4* dst = reinterpret_cast<uint4*>(out + part_row * 128 + cc * 32);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dst[e] = some ? make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]) : make_uint4(0, 0, 0, 0);
        } else {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            pk[e] = some ? pack_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv) : 0u;
          store_row_chunk(p.o + at * 128 + cc * 32, pk);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.seg_empty[k % kSegs]);
      if (kAlt && second) named_bar_sync(1, 256);  // Q's tile may be written again
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) {
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the segments of one tile: the CTAs whose shares meet its pages. A warp
// per row.
constexpr int kJoinRows = 8;
template <bool kAlt>
__global__ void __launch_bounds__(256)
    cache_tile_join_kernel(const __grid_constant__ CacheAttnParams p, int ctas, const float* part) {
  using T = Tiles<kAlt>;
  constexpr int kBlocks = T::kRows / kJoinRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x / kBlocks, row0 = blockIdx.x % kBlocks * kJoinRows;
  const int head = blockIdx.y, b = blockIdx.z;
  const Stream st = stream_of(p.tok_start, p.kv_len, b, p.n, p.table_stride);
  const int rows = st.n_new * p.group;
  const bool mine = t < T::count(p, st) && t * T::kRows + row0 < rows;
  int64_t u0 = 0, total = 0;
  int pages = 0, weight = 1;
  if (mine) {
    u0 = T::total(p, b, false, lane);
    total = T::total(p, p.batch, false, lane);
    int64_t before = 0;
    for (int i = lane; i < t; i += 32) before += T::cost(p, st, i, false);
    u0 += T::warp_sum(before) + head * T::head_cost(p, st, false);
    pages = T::pages(p, st, t);
    weight = T::weight(st, p, t);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!mine) return;
  const int64_t u1 = u0 + static_cast<int64_t>(pages) * weight;
  // the last CTA whose share begins at or before u0
  int c = static_cast<int>(u0 * ctas / total);
  while (c + 1 < ctas && total * (c + 1) / ctas <= u0) ++c;
  while (c > 0 && total * c / ctas > u0) --c;
  if (pages_before(total * (c + 1) / ctas, u0, pages, weight, false) == pages) return;  // one CTA had all of them
  const int last = static_cast<int>(std::min<int64_t>(ctas, (u1 * ctas + total - 1) / total + 1));
  for (int rr = row0 + warp; rr < row0 + kJoinRows && t * T::kRows + rr < rows; rr += 8) {
    const int r = t * T::kRows + rr;
    join_row(
        p, static_cast<int64_t>(head * p.group + r % p.group) * p.n + st.t0 + r / p.group, lane, c, last,
        [&](int i) -> const float* {
          const int64_t w0 = total * i / ctas;
          const int first = pages_before(w0, u0, pages, weight, false);
          if (first == pages_before(total * (i + 1) / ctas, u0, pages, weight, false)) return nullptr;
          return part + (2 * static_cast<int64_t>(i) + (first > 0 ? 0 : 1)) * tile_part_floats(T::kRows);
        },
        rr, T::kRows);
  }
}

template <bool SW, bool kAlt>
int launch(const CUtensorMap& mk, const CUtensorMap& mv, const CacheAttnParams& p, const TilePlan& plan, float* part,
           cudaStream_t stream) {
  static PerDeviceOnce once;
  const int rc =
      set_max_smem_once(reinterpret_cast<const void*>(cache_tile_kernel<SW, kAlt>), tile_smem<kAlt>(), once);
  if (rc != CALIBATT_OK) return rc;
  // the register split needs the allotment it was sized for
  static std::once_flag regs_once;
  static int launch_regs = 0;
  std::call_once(regs_once, [] {
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, cache_tile_kernel<SW, kAlt>) == cudaSuccess) launch_regs = fa.numRegs;
  });
  if (launch_regs * kTileThreads < kTileRegs) return CALIBATT_ERR_CUDA;
  cache_tile_kernel<SW, kAlt><<<plan.ctas, kTileThreads, tile_smem<kAlt>(), stream>>>(mk, mv, p, plan.whole, part);
  if (cudaGetLastError() != cudaSuccess) return CALIBATT_ERR_CUDA;
  if (plan.whole) return CALIBATT_OK;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(plan.tiles) * (Tiles<kAlt>::kRows / kJoinRows), p.heads_kv, p.batch);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  // resident while the pages are still read: it waits in the kernel
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_tile_join_kernel<kAlt>, p, plan.ctas, static_cast<const float*>(part)) ==
                 cudaSuccess
             ? CALIBATT_OK
             : CALIBATT_ERR_CUDA;
}

}  // namespace

TilePlan tile_plan(int batch, int heads_kv, int64_t rows, int64_t pages, int sms) {
  TilePlan t;
  t.alternate = rows <= 128;
  const int tile = t.alternate ? 128 : 256;
  t.tiles = static_cast<int>((rows + tile - 1) / tile);
  const int64_t units = static_cast<int64_t>(batch) * heads_kv * t.tiles;
  // up to 4 pages the join costs more than the split saves, and a share has
  // at least two pages
  t.whole = pages <= 4;
  t.ctas = static_cast<int>(std::min<int64_t>(sms, t.whole ? units : units * ((pages + 1) / 2)));
  return t;
}

size_t tile_workspace_bytes(const TilePlan& plan) {
  if (plan.whole) return 0;
  return 2 * static_cast<size_t>(plan.ctas) * tile_part_floats(plan.alternate ? 128 : 256) * sizeof(float);
}

int launch_cache_attn_tiles(const CacheAttnParams& p, const TilePlan& plan, void* ws, cudaStream_t stream) {
  CUtensorMap mk, mv;
  int rc = make_page_map(&mk, p.k8, p);
  if (rc == CALIBATT_OK) rc = make_page_map(&mv, p.v8, p);
  if (rc != CALIBATT_OK) return rc;
  float* part = static_cast<float*>(ws);
  const bool short_waits = p.wait_limit_ns < kShortWaitNs;
  if (plan.alternate)
    return short_waits ? launch<true, true>(mk, mv, p, plan, part, stream)
                       : launch<false, true>(mk, mv, p, plan, part, stream);
  return short_waits ? launch<true, false>(mk, mv, p, plan, part, stream)
                     : launch<false, false>(mk, mv, p, plan, part, stream);
}

}  // namespace calibatt
