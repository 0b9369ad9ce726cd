// Attention over the paged 8-bit cache for 17 to 128 query rows that share a
// key head, on the sm_100a tensor core.
//
// Like with fewer rows the cache's pages are one list, stream by stream, key
// head by key head, cut into equal shares whatever the streams' lengths are,
// one CTA per SM. A stretch of a share that is not all of its stream's pages
// leaves maximum, sum and unnormalised output in the workspace, and
// cache_join_kernel joins them.
//
// CTA (512 threads, persistent), one tile of 128 / KS query rows, KS times over:
//   warps 0-3, 4-7   softmax of slot 0 and slot 1 (thread = TMEM lane = query
//                    row and its KS-th of a page's keys)
//   warps 8-11       converters: e4m3 tiles to fp16 operand tiles in a
//                    4-stage ring (128-byte swizzle on both sides)
//   warp  12         MMA issuer (one thread): S = Q K^T and O += P V
//   warp  13         TMA producer of the e4m3 tiles, 4 ahead
//   warp  14         scheduler: walks the share and hands out its stretches
//   warp  15         idle
// The two slots hold the same rows and take every other page, and are joined
// at a stretch's end: the chain S -> softmax -> P V of one slot runs beside the
// other's. The tensor core multiplies 128 rows whatever is in them, so up to 64
// (32) rows stand in the tile 2 (4) times, and each copy takes the softmax of a
// half (quarter) of the keys, with zeros for the others in P: all warps work on
// a chain that is 2 (4) times as short. Numbers are held as in cache_tile.cu: fp16 operands without scales,
// O in units of a reference value scale.
// Bound, by this count, by shared memory: a page's 32 KB land there, are read and written as
// 64 KB by the converters, and 96 KB are read as operands (Q's tile anew for
// each page): 224 KB at 128 bytes a cycle are 1790 cycles, of the ~1850 that a
// page takes with 25 rows. Measured: 16 streams of 20000 tokens, 40 query heads
// on 8, 5 new tokens each in 132 us, half of the DRAM rate (150 us without the
// copies; 148 us with K as an 8-bit operand and Q in three parts, which are 12
// products instead of 8; 132 us with a second warpgroup of converters).
// The register split keeps the issuer's loop in registers; a spill there is
// read back through an L1 that the tiles have flushed (measured at 40
// registers: ~350 cycles per MMA). ptxas spills 24 bytes with one copy of the
// rows, none with two and four.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "cache.cuh"
#include "cache_list.cuh"
#include "calibatt.h"
#include "kernels.h"
#include "ptx.cuh"
#include "sched.cuh"
#include "softmax.cuh"

namespace calibatt {
namespace {

constexpr int kMidThreads = 512;
// registers per thread after the split; their sum must fit in the launch
// allotment of 128 x 512 (checked against the compiled count before a launch)
constexpr int kMidSoftmaxRegs = 192;
constexpr int kMidConvertRegs = 64;
constexpr int kMidControlRegs = 64;
constexpr int kMidRegs = 256 * kMidSoftmaxRegs + 128 * kMidConvertRegs + 128 * kMidControlRegs;
static_assert(kMidRegs <= 128 * kMidThreads, "register split");
constexpr float kStaleMax = 8.0f;      // log2 units: move the running max only if it grows by more
constexpr float kBigScore = 65536.0f;  // log2 units: beyond it the rounding of the row max counts
constexpr int kRawBytes = kPage * 128;
constexpr int kRing = 4;               // fp16 tiles
constexpr int kRaw = 4;                // e4m3 tiles in flight
constexpr int kSegs = 2;               // stretches handed out ahead
constexpr int kNanSlots = 4;           // converters are never that many stretches ahead of the softmax

// What a warp needs of a stretch; np = 0 ends the share.
struct Segment {
  int b, head, t0, n_new, len;
  int rows;
  int least;      // keys that every row sees
  int pg0, np;
  int pages;      // of the stream
  int number;     // of the stretch in its share
  int seconds;    // stretches of several pages before it
};

struct MidLayout {
  static constexpr int kQOff = 0;
  static constexpr int kRawOff = kTile;
  static constexpr int kRingOff = kRawOff + kRaw * kRawBytes;
  static constexpr int kBarOff = kRingOff + kRing * kTile;
};

struct MidBarriers {
  uint64_t ring_full[kRing], ring_empty[kRing];
  uint64_t raw_full[kRaw], raw_empty[kRaw];
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t q_full;
  uint64_t s_full[2];
  uint64_t p_full[2][2];  // per slot, per half of the page's keys
  uint64_t o_full[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
  int go[2];                // whether the softmax warps got stretch k (k even, odd)
  int raw_bad[kRaw];        // the tile's page is outside the pool: nothing was loaded
  int nan_seen[kNanSlots];  // 1 + number of the stretch in which a NaN value was taken out of a page
  Segment seg[kSegs];
};

constexpr int kMidSmem = MidLayout::kBarOff + static_cast<int>(sizeof(MidBarriers)) + 1024;
static_assert(kMidSmem <= 232448, "shared memory budget");

__device__ __forceinline__ void tmem_ld_scores(uint32_t at, float (&s)[32]) {
  tmem_ld32_wait(at, reinterpret_cast<uint32_t(&)[32]>(s));
}
__device__ __forceinline__ void tmem_ld_scores(uint32_t at, float (&s)[64]) { tmem_ld64_wait(at, s); }
__device__ __forceinline__ void tmem_ld_scores(uint32_t at, float (&s)[128]) {
  tmem_ld64_wait(at, reinterpret_cast<float(&)[64]>(s[0]));
  tmem_ld64_wait(at + 64, reinterpret_cast<float(&)[64]>(s[64]));
}

template <bool SW, int KS>
__global__ void __launch_bounds__(kMidThreads, 1)
    cache_mid_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ CacheAttnParams p, bool whole, float* part) {
  using L = MidLayout;
  constexpr int kRows = 128 / KS;   // rows of Q's tile, which holds them KS times
  constexpr int kKeys = kPage / KS;  // of a page, for the rows of one copy
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const uint32_t sbase = smem_u32(smem);
  MidBarriers& bar = *reinterpret_cast<MidBarriers*>(smem + L::kBarOff);
  volatile int* abort_flag = &bar.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&bar.ring_full[i], 128);
      mbar_init(&bar.ring_empty[i], 1);
    }
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(&bar.raw_full[i], 1);
      mbar_init(&bar.raw_empty[i], 4);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&bar.seg_full[i], 1);
      mbar_init(&bar.seg_empty[i], 14);  // softmax and converter warps, issuer, producer
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar.s_full[s], 1);
      mbar_init(&bar.p_full[s][0], 128);
      mbar_init(&bar.p_full[s][1], 128);
      mbar_init(&bar.o_full[s], 1);
    }
    mbar_init(&bar.q_full, 128);
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
    warpgroup_regs_dec<kMidConvertRegs>();
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
      if (++stage == kRing) {
        stage = 0;
        phase ^= 1;
      }
      return true;
    };
    uint32_t raw_stage = 0, raw_phase = 0;
    for (int k = 0; ok && __all_sync(0xffffffffu, has_segment(k)); ++k) {
      const Segment& seg = bar.seg[k % kSegs];
      const int np = seg.np;
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
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.seg_empty[k % kSegs]);
    }
  } else if (warp >= 12) {
    warpgroup_regs_dec<kMidControlRegs>();
    if (warp == 14) {
      // -------------------------------------------------------- scheduler
      if (blockIdx.x == 0)  // streams that do not fit are reported once
        for (int b = lane; b < p.batch; b += 32) {
          const Stream st = stream_of(p.tok_start, p.kv_len, b, p.n, p.table_stride);
          if (!stream_fits(p, st)) record_error(p.status, CALIBATT_ERR_CSR);
        }
      int k = 0, seconds = 0;
      bool ok = true;
      Walk walk;
      walk.start(p, whole, lane);
      Stretch s;
      for (bool more = true; more && ok; ++k) {
        more = walk.next(p, s);
        if (lane == 0) {
          ok = mbar_wait<SW>(&bar.seg_empty[k % kSegs], ((k / kSegs) & 1) ^ 1, abort_flag, p.status, p.wait_limit_ns);
          if (ok) {
            Segment& seg = bar.seg[k % kSegs];
            seg.np = 0;
            if (more) {
              seg.b = s.b;
              seg.head = s.head;
              seg.t0 = s.st.t0;
              seg.n_new = s.st.n_new;
              seg.len = s.st.len;
              seg.rows = s.st.n_new * p.group;
              seg.least = visible(s.st.len - s.st.n_new, s.st.len, p.unit);
              seg.pg0 = s.pg;
              seg.np = s.count;
              seg.pages = s.pages;
              seg.number = k;
              seg.seconds = seconds;
            }
            mbar_arrive(&bar.seg_full[k % kSegs]);
          }
        }
        if (more && s.count > 1) ++seconds;
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
    } else if (warp == 13) {
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
      uint32_t n_q = 0, n_p[2] = {0, 0};
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
        if (++stage == kRing) {
          stage = 0;
          phase ^= 1;
        }
      };
      auto ring_next = [&]() {
        mma_commit(&bar.ring_empty[stage]);
        advance();
      };
      auto issue_s = [&](int s) {
        const uint64_t qd = qdesc0, kd = kdesc0 + stage * (kTile >> 4);
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
        const int np = bar.seg[k % kSegs].np;
        mbar_arrive(&bar.seg_empty[k % kSegs]);
        if (!(go = wait(&bar.q_full, n_q++ & 1))) break;
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
      }
      // every issued MMA has finished before tensor memory is released
      mma_commit(&bar.mma_done);
      volatile int never = 0;
      mbar_wait(&bar.mma_done, 0, &never, p.status);
    }
  } else {
    // ---------------------------------------------------------- softmax
    warpgroup_regs_inc<kMidSoftmaxRegs>();
    const int s = warp >> 2;
    const int tm_row = (warp & 3) * 32 + lane;  // of Q's tile = TMEM lane
    const int row = tm_row % kRows, copy = tm_row / kRows;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t sc = tmem + lane_off + s * 128, oc = tmem + lane_off + 256 + s * 128;
    uint32_t n_s = 0;
    // after a failed wait a segment is finished without waiting or touching
    // tensor memory, so that the warps still meet at its barriers
    bool ok = true;  // warp-uniform
    auto wait_warp = [&](uint64_t* bb, uint32_t parity) -> bool {
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait<SW>(bb, parity, abort_flag, p.status, p.wait_limit_ns));
      return ok;
    };
    for (int k = 0;; ++k) {
      // the two slots meet at barriers inside a stretch: one warp asks for all
      if (warp == 0) {
        const bool more = __all_sync(0xffffffffu, ok && has_segment(k));
        if (lane == 0) bar.go[k & 1] = more;
      }
      named_bar_sync(2, 256);
      if (bar.go[k & 1] == 0) break;
      const Segment& seg = bar.seg[k % kSegs];
      const int np = seg.np;
      const bool second = np > 1;  // slot 1 has work
      const bool active = s == 0 || second;
      // A warp without rows leaves its part of S and P as it is: only its own
      // rows of O depend on it.
      const bool row_valid = row < seg.rows;
      const bool idle = !__any_sync(0xffffffffu, row_valid);
      const int tok = row_valid ? row / p.group : 0;
      const int64_t at =
          static_cast<int64_t>(seg.head * p.group + (row_valid ? row % p.group : 0)) * p.n + seg.t0 + tok;
      // a padded row sees all keys: it is computed and not stored
      const int limit = row_valid ? visible(seg.len - seg.n_new + tok, seg.len, p.unit) : seg.len;
      float m_run = -INFINITY, l_run = 0.f;
      VRef<6, -6> vref;  // P below 2^8 (stale maximum) * 2^6 * 2, fp16; 2^-24 * 2^6 * 2^-6 is its smallest value
      if (active) {
        // the row of Q to shared memory, as fp16 times a power of two (by slot
        // 0 for both)
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
        if (s == 0) {
          const uint32_t dst = sbase + L::kQOff + tm_row * 128;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint32_t x[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              h[e] = pack_half2(__uint_as_float(x[e] << 16) * shrink, __uint_as_float(x[e] & 0xffff0000u) * shrink);
            st_shared16(dst + (j >> 3) * kHalf + (((j & 7) ^ (tm_row & 7)) << 4), h[0], h[1], h[2], h[3]);
          }
          fence_proxy_async();
          mbar_arrive(&bar.q_full);
        }
        PageWindow<true> win(p, seg.b, seg.head, seg.pg0, np, seg.len);
        win.fetch(lane, p.status);
        bool started = false;  // O holds a product of this segment
        for (int i = s; i < np; i += 2) {
          if ((i & 31) < 2) win.advance(i & ~31, lane, p.status);
          const int id = __shfl_sync(0xffffffffu, win.id, i & 31);
          const float ck = score_factor(c_row, __shfl_sync(0xffffffffu, win.ks, i & 31));
          const float o_ratio = vref.page(__shfl_sync(0xffffffffu, win.vs, i & 31));
          if (!wait_warp(&bar.s_full[s], n_s & 1)) break;
          ++n_s;
          if (idle) {
            mbar_arrive(&bar.p_full[s][0]);
            mbar_arrive(&bar.p_full[s][1]);
            continue;
          }
          tc_fence_after();
          const int key0 = (seg.pg0 + i) * kPage;
          // keys that the row sees, of the page's that are its copy's
          const int cut = id < 0 ? 0 : min(limit - key0 - copy * kKeys, kKeys);
          float sv[kKeys];
          tmem_ld_scores(sc + copy * kKeys, sv);
          if (__any_sync(0xffffffffu, cut < kKeys)) {
#pragma unroll
            for (int e = 0; e < kKeys; ++e)
              if (e >= cut) sv[e] = -INFINITY;
          }
          const float mx = row_max_of(sv);
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
            for (int e = 0; e < kKeys; ++e) sv[e] = (sv[e] - mx0) * ck;
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
          // P (fp16, two keys per column) over the first 64 columns of S: in
          // two halves, or with zeros for the other copies' keys
          if constexpr (KS > 1) {
            const uint32_t zero[16] = {};
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (c / (4 / KS) != copy) tmem_st16(sc + c * 16, zero);
          }
          constexpr int kPart = kKeys < 64 ? kKeys : 64;
#pragma unroll
          for (int h = 0; h < kKeys / kPart; ++h) {
            uint32_t pk[kPart / 2];
#pragma unroll
            for (int e = 0; e < kPart / 2; ++e) {
              const float2 x = exp2_mufu2(ffma2(make_float2(sv[h * kPart + 2 * e], sv[h * kPart + 2 * e + 1]), c2, n2));
              a4[e & 3] = fadd2(a4[e & 3], x);
              pk[e] = pack_half2(x.x, x.y);
            }
            if constexpr (KS == 4)
              tmem_st16(sc + copy * 16, pk);
            else
              tmem_st32(sc + (copy + h) * 32, pk);
            tmem_wait_st();
            tc_fence_before();
            if constexpr (KS == 1) {
              mbar_arrive(&bar.p_full[s][h]);
            } else {
              mbar_arrive(&bar.p_full[s][0]);
              mbar_arrive(&bar.p_full[s][1]);
            }
          }
          const float2 s01 = fadd2(a4[0], a4[1]), s23 = fadd2(a4[2], a4[3]);
          l_run = l_run * alpha + ((s01.x + s01.y) + (s23.x + s23.y)) * vref.inv;
        }
      }
      // The stretch's products are complete, of both slots that have some: the
      // exchange below uses Q's tile. A slot without pages waits for the other
      // one all the same, which is still writing Q there or multiplying it.
      wait_warp(&bar.o_full[0], k & 1);  // slot 0 has a page of every stretch
      if (second) wait_warp(&bar.o_full[1], seg.seconds & 1);
      tc_fence_after();
      const bool done = ok && *abort_flag == 0;
      m_run += vref.raise();
      l_run *= vref.damp();
      // A row's shares of the stretch, two slots by KS copies, are added up
      // through Q's tile, 32 channels at a time and 16 / KS of them by each of
      // the threads that hold a share: [share][channel][row].
      float* joined = reinterpret_cast<float*>(smem + L::kQOff);
      const int share = s * KS + copy, n_shares = second ? 2 * KS : KS;
      float2* ml = reinterpret_cast<float2*>(joined);  // maxima and sums first
      ml[share * kRows + row] = make_float2(m_run, l_run);
      named_bar_sync(1, 256);
      float mx = -INFINITY, l = 0.f;
      for (int i = 0; i < n_shares; ++i) mx = fmaxf(mx, ml[i * kRows + row].x);
      const float use = mx == -INFINITY ? 0.f : mx;
      for (int i = 0; i < n_shares; ++i) {
        const float2 x = ml[i * kRows + row];
        l += x.y * ex2_approx(x.x - use);
      }
      const float factor = ex2_approx(m_run - use) * vref.unit();
      const bool some = l != 0.f;
      const float inv = some ? 1.f / l : 0.f;
      const bool complete = np == seg.pages;
      float* out = part_of(part, blockIdx.x, seg.pg0 > 0, kMidRows);
      if (done && row_valid && share == 0) {
        if (!complete)
          *reinterpret_cast<float2*>(out + kMidRows * 128 + 2 * row) = make_float2(mx, some ? l : 0.f);
        else if (p.lse)
          p.lse[at] = some ? (mx + log2f(l)) * kLn2 : -INFINITY;
      }
      const bool patch =
          *const_cast<volatile int*>(&bar.nan_seen[seg.number % kNanSlots]) == seg.number + 1;
      constexpr int kCh = 16 / KS;
#pragma unroll 1
      for (int cc = 0; cc < 4; ++cc) {
        named_bar_sync(1, 256);  // what was there has been read
        if (done && active && !idle) {
          uint32_t o[32];
          tmem_ld32_wait(oc + cc * 32, o);
#pragma unroll
          for (int e = 0; e < 32; ++e) joined[(share * 32 + e) * kRows + row] = __uint_as_float(o[e]) * factor;
        }
        named_bar_sync(1, 256);
        if (!done || !row_valid) continue;
        const int ch = cc * 32 + share * kCh;  // the thread's channels
        float x[kCh];
#pragma unroll
        for (int e = 0; e < kCh; ++e) x[e] = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * KS; ++i) {
          if (i >= n_shares) break;
#pragma unroll
          for (int e = 0; e < kCh; ++e) x[e] += joined[(i * 32 + share * kCh + e) * kRows + row];
        }
        if (patch) {
          // NaN values that were taken out of pages that not every row sees whole
          const int32_t* table = p.table + static_cast<int64_t>(seg.b) * p.table_stride;
          uint32_t bad = 0;
          for (int key = max(seg.least / kPage, seg.pg0) * kPage; key < min(limit, (seg.pg0 + np) * kPage); ++key) {
            const int id = __ldg(table + key / kPage);
            if (id < 0 || id >= p.n_pages) continue;
            const uint8_t* v = p.v8 + ((static_cast<int64_t>(id) * p.heads_kv + seg.head) * kPage + key % kPage) * 128;
            for (int e = 0; e < kCh; ++e)
              if ((v[ch + e] & 0x7f) == 0x7f) bad |= 1u << e;
          }
#pragma unroll
          for (int e = 0; e < kCh; ++e)
            if (bad >> e & 1) x[e] = __int_as_float(0x7fffffff);
        }
        if (!complete) {
          float4* dst = reinterpret_cast<float4*>(out + row * 128 + ch);
#pragma unroll
          for (int e = 0; e < kCh / 4; ++e)
            dst[e] = some ? make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3])
                          : make_float4(0.f, 0.f, 0.f, 0.f);
        } else {
          uint2* dst = reinterpret_cast<uint2*>(p.o + at * 128 + ch);
#pragma unroll
          for (int e = 0; e < kCh / 4; ++e)
            dst[e] = some ? make_uint2(pack_bf16x2(x[4 * e] * inv, x[4 * e + 1] * inv),
                                       pack_bf16x2(x[4 * e + 2] * inv, x[4 * e + 3] * inv))
                          : make_uint2(0, 0);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.seg_empty[k % kSegs]);
      named_bar_sync(1, 256);  // Q's tile may be written again
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

template <bool SW, int KS>
int launch(const CUtensorMap& mk, const CUtensorMap& mv, const CacheAttnParams& p, const SharePlan& plan, float* part,
           cudaStream_t stream) {
  static PerDeviceOnce once;
  const int rc = set_max_smem_once(reinterpret_cast<const void*>(cache_mid_kernel<SW, KS>), kMidSmem, once);
  if (rc != CALIBATT_OK) return rc;
  // the register split needs the allotment it was sized for
  static std::once_flag regs_once;
  static int launch_regs = 0;
  std::call_once(regs_once, [] {
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, cache_mid_kernel<SW, KS>) == cudaSuccess) launch_regs = fa.numRegs;
  });
  if (launch_regs * kMidThreads < kMidRegs) return CALIBATT_ERR_CUDA;
  cache_mid_kernel<SW, KS><<<plan.ctas, kMidThreads, kMidSmem, stream>>>(mk, mv, p, plan.whole, part);
  return cudaGetLastError() == cudaSuccess ? CALIBATT_OK : CALIBATT_ERR_CUDA;
}

}  // namespace

int launch_cache_attn_mid(const CacheAttnParams& p, const SharePlan& plan, void* ws, cudaStream_t stream) {
  CUtensorMap mk, mv;
  int rc = make_page_map(&mk, p.k8, p);
  if (rc == CALIBATT_OK) rc = make_page_map(&mv, p.v8, p);
  if (rc != CALIBATT_OK) return rc;
  float* part = static_cast<float*>(ws);
  const bool sw = p.wait_limit_ns < kShortWaitNs;
  if (p.max_rows <= 32)
    rc = sw ? launch<true, 4>(mk, mv, p, plan, part, stream) : launch<false, 4>(mk, mv, p, plan, part, stream);
  else if (p.max_rows <= 64)
    rc = sw ? launch<true, 2>(mk, mv, p, plan, part, stream) : launch<false, 2>(mk, mv, p, plan, part, stream);
  else
    rc = sw ? launch<true, 1>(mk, mv, p, plan, part, stream) : launch<false, 1>(mk, mv, p, plan, part, stream);
  return rc != CALIBATT_OK || plan.whole ? rc : launch_cache_join(p, plan, part, kMidRows, stream);
}

}  // namespace calibatt
