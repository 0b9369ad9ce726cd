// Attention over the paged 8-bit cache for many query rows (more than 128 that
// share a key head), on the sm_100a tensor core.
//
// CTA (512 threads, one per SM; one row tile, key head and split of the pages):
//   warps 0-3, 4-7   softmax of slot 0 and slot 1 (thread = query row = TMEM lane)
//   warps 8-11       converters: read a page's e4m3 tile from global memory two
//                    tiles ahead, write it as a 16-bit operand tile into a
//                    5-stage shared-memory ring (128-byte swizzle)
//   warp  12         MMA issuer (one thread): S = Q K^T and O += P V
//   warps 13-15      idle (they complete the fourth warpgroup, whose registers
//                    go to the softmax warpgroups)
// A slot is 128 query rows: each converted tile feeds both, so the conversion
// (on the same issue slots as the softmax) is paid once per two tensor-core
// tiles.
//
// K and V become fp16 without their scales: fp16 holds every e4m3 value, and
// the conversion is one instruction per two values (with the scale in it, as
// bf16, it took five and the converters, not the tensor core, set the pace).
// Q is brought to fp16 by a power of two per row; that and the key scale
// multiply the fp32 score. P is fp16; O is kept in units of a reference value
// scale (VRef), so a page's value scale costs nothing either.
//
// Bound by the chain S -> softmax -> P V of a slot and, with all SMs at work, by
// the power limit. Measured on B200: a 480p frame (1560 tokens of 40 heads over
// 32760) in 1075 to 1120 us, 0.57 of the rate of a library matrix product (7
// tiles a head, the last of 24 rows; 0.61 counting the rows that are computed
// for nothing); three streams of four frames, causal by frames, in 460 us,
// 0.53. Slower: exponentials on the FMA pipe (1/8 to 3/8 of them: 2 to 13 %),
// one hand-over of P instead of two (5 %) or four (2.5 %), e4m3 tiles by TMA
// (15 %), 176/96/64 registers (15 %; with this split ptxas spills 4 bytes), a
// persistent grid with equal shares (its bookkeeping spilled the issuer's
// registers: 3 times as slow).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
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

constexpr int kTileThreads = 512;
// registers per thread after the split; their sum must fit in the launch
// allotment of 128 x 512 (checked against the compiled count before a launch)
constexpr int kTileSoftmaxRegs = 192;
constexpr int kTileConvertRegs = 88;
constexpr int kTileControlRegs = 40;
constexpr int kTileRegs = 256 * kTileSoftmaxRegs + 128 * kTileConvertRegs + 128 * kTileControlRegs;
static_assert(kTileRegs <= 128 * kTileThreads, "register split");
constexpr int kTileRing = 5;
constexpr float kStaleMax = 8.0f;      // log2 units: move the running max only if it grows by more
constexpr float kBigScore = 65536.0f;  // log2 units: beyond it the rounding of the row max counts

struct TileBarriers {
  uint64_t ring_full[kTileRing];
  uint64_t ring_empty[kTileRing];
  uint64_t q_full[2];
  uint64_t s_full[2];
  uint64_t p_full[2][2];  // per slot, per half of the page's keys
  uint64_t o_full[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
  int nan_seen;       // a NaN value was taken out of a page that some rows do not see whole
};

struct TileLayout {
  static constexpr int kQOff = 0;
  static constexpr int kRingOff = 2 * kTile;
  static constexpr int kBarOff = kRingOff + kTileRing * kTile;
  static constexpr int kBytes = kBarOff + static_cast<int>(sizeof(TileBarriers));
  static constexpr int kDynSmem = kBytes + 1024;
};
static_assert(TileLayout::kDynSmem <= 232448, "shared memory budget");

// Tiles are taken rank by rank for a chunk of (stream, key head) pairs. Under a
// causal mask the tiles with most keys have the lowest ranks, so the last ones
// to start are short (3 x 16 heads, 6240 tokens by frames of 1560: 491 -> 455
// us against head by head).
struct TileUnit {
  int b, head, rank;
};
__device__ __forceinline__ TileUnit tile_unit(const CacheAttnParams& p, const TilePlan& plan, int unit) {
  const int per_chunk = plan.chunk * plan.tiles;
  const int pair0 = unit / per_chunk * plan.chunk, pairs = min(plan.chunk, p.batch * p.heads_kv - pair0);
  const int pair = pair0 + unit % per_chunk % pairs;
  return {pair / p.heads_kv, pair % p.heads_kv, unit % per_chunk / pairs};
}
__device__ __forceinline__ int tile_first_row(const CacheAttnParams& p, const TileUnit& u, int tiles) {
  return (p.unit > 0 ? tiles - 1 - u.rank : u.rank) * kTileRows;
}

template <bool SW>
__global__ void __launch_bounds__(kTileThreads, 1)
    cache_tile_kernel(const __grid_constant__ CacheAttnParams p, const TilePlan plan, float* part) {
  using L = TileLayout;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const uint32_t sbase = smem_u32(smem);
  TileBarriers& bar = *reinterpret_cast<TileBarriers*>(smem + L::kBarOff);
  volatile int* abort_flag = &bar.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ------------------------------------------------------------ the CTA's work
  const int behind = static_cast<int>(blockIdx.x) - plan.whole;
  const int splits = behind < 0 ? 1 : plan.splits, split = behind < 0 ? 0 : behind % splits;
  const TileUnit u = tile_unit(p, plan, plan.whole + (behind < 0 ? behind : behind / splits));
  const int b = u.b, head = u.head;
  const Stream st = stream_of(p.tok_start, p.kv_len, b, p.n, p.table_stride);
  if (st.bad || st.n_new > p.max_new) {
    if (threadIdx.x == 0) record_error(p.status, CALIBATT_ERR_CSR);
    return;
  }
  const int rows = st.n_new * p.group;
  const int tiles = (rows + kTileRows - 1) / kTileRows;
  if (u.rank >= tiles) return;
  const int r0 = tile_first_row(p, u, tiles);
  const int r1 = min(rows, r0 + kTileRows);
  const int first_pos = st.len - st.n_new;  // position of the first new token
  const int least = visible(first_pos + r0 / p.group, st.len, p.unit);        // keys that every row sees
  const int most = visible(first_pos + (r1 - 1) / p.group, st.len, p.unit);   // keys that any row sees
  const int pages = (most + kPage - 1) / kPage;
  const int per = (pages + splits - 1) / splits;
  const int pg0 = min(pages, split * per);
  const int np = min(pages, pg0 + per) - pg0;
  const bool second = r1 - r0 > 128;  // slot 1 has work
  const int32_t* table = p.table + static_cast<int64_t>(b) * p.table_stride + pg0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kTileRing; ++i) {
      mbar_init(&bar.ring_full[i], 128);
      mbar_init(&bar.ring_empty[i], 1);
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
    bar.nan_seen = 0;
    fence_barrier_init();
  }
  if (warp == 12) tmem_alloc(&bar.tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem_base;

  if (warp >= 8 && warp < 12) {
    // ---------------------------------------------------------- converters
    warpgroup_regs_dec<kTileConvertRegs>();
    bool ok = true;
    // lanes of a store phase: two rows (one even, one odd) of four quarters
    // of a 64-channel half, so their 16-byte chunks fall into eight banks groups
    const int row = (warp - 8) * 8 + (lane >> 2), quarter = lane & 3;
    PageWindow<false> win(p, b, head, pg0, np, st.len);
    win.fetch(lane, p.status);
    // pages are met in order by K; V follows at most one page behind
    int id_now = -1, id_before = -1, k_at = 0;
    const int nt = 2 * np;
    uint4 buf[2][8];
    auto load = [&](int t, uint4 (&w)[8]) {
      bool is_v;
      int i, id;
      ring_tile<false>(t, np, is_v, i);
      if (!is_v) {
        if ((i & 31) == 0) win.advance(i, lane, p.status);
        id_before = id_now;
        id_now = id = __shfl_sync(0xffffffffu, win.id, i & 31);
        k_at = i;
      } else {
        id = k_at == i ? id_now : id_before;
      }
      if (id < 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = make_uint4(0, 0, 0, 0);
        return;
      }
      const uint8_t* src = (is_v ? p.v8 : p.k8) + (static_cast<int64_t>(id) * p.heads_kv + head) * (kPage * 128) +
                           row * 128 + quarter * 16;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        w[e] = __ldg(reinterpret_cast<const uint4*>(src + (e >> 1) * (32 * 128) + (e & 1) * 64));
    };
    uint32_t stage = 0, phase = 0;
    auto convert = [&](int t, uint4 (&w)[8]) -> bool {
      bool is_v;
      int i;
      ring_tile<false>(t, np, is_v, i);
      const int key0 = (pg0 + i) * kPage;
      if (is_v && key0 + kPage > least) {
        // a page that some row does not see whole: a product takes every key
        // for every row, and 0 * NaN is NaN. Slots behind the last token
        // become zero, and so does a NaN, which the rows that see it get back
        // at the end.
        uint32_t nan = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int key = key0 + (e >> 1) * 32 + row;
          uint32_t* x = reinterpret_cast<uint32_t*>(&w[e]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (key >= st.len) x[k] = 0;
            nan |= take_nan(x[k]);
          }
        }
        if (nan) *const_cast<volatile int*>(&bar.nan_seen) = 1;
      }
      if (!mbar_wait<SW>(&bar.ring_empty[stage], phase ^ 1, abort_flag, p.status, p.wait_limit_ns)) return false;
      const uint32_t dst = sbase + L::kRingOff + stage * kTile + row * 128;
#pragma unroll
      for (int e = 0; e < 8; ++e) store_half(dst + (e & 1) * kHalf + (e >> 1) * (32 * 128), row, 2 * quarter, w[e]);
      fence_proxy_async();
      mbar_arrive(&bar.ring_full[stage]);
      if (++stage == kTileRing) {
        stage = 0;
        phase ^= 1;
      }
      return true;
    };
    // the wait's outcome is made the warp's, for the shuffles that follow
    if (nt > 0) load(0, buf[0]);
    if (nt > 1) load(1, buf[1]);
    for (int t = 0; t < nt && ok; t += 2) {
      ok = __all_sync(0xffffffffu, convert(t, buf[0]));
      if (t + 2 < nt) load(t + 2, buf[0]);
      if (t + 1 < nt && ok) {
        ok = __all_sync(0xffffffffu, convert(t + 1, buf[1]));
        if (t + 3 < nt) load(t + 3, buf[1]);
      }
    }
  } else if (warp >= 12) {
    warpgroup_regs_dec<kTileControlRegs>();
    if (warp == 12 && lane == 0 && np > 0) {
      // -------------------------------------------------------- MMA issuer
      uint32_t stage = 0, phase = 0;
      const uint64_t qdesc0 = desc_k_base(sbase + L::kQOff);
      const uint64_t kdesc0 = desc_k_base(sbase + L::kRingOff);
      const uint64_t vdesc0 = desc_v_base(sbase + L::kRingOff);
      auto ring_wait = [&]() -> bool {
        if (!mbar_wait<SW>(&bar.ring_full[stage], phase, abort_flag, p.status, p.wait_limit_ns)) return false;
        tc_fence_after();
        return true;
      };
      auto ring_next = [&]() {
        mma_commit(&bar.ring_empty[stage]);
        if (++stage == kTileRing) {
          stage = 0;
          phase ^= 1;
        }
      };
      auto issue_s = [&](int s) {
        const uint64_t qd = qdesc0 + s * (kTile >> 4), kd = kdesc0 + stage * (kTile >> 4);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_ss(tmem + s * 128, qd + desc_k_step(ks), kd + desc_k_step(ks), kIdescQK, ks > 0);
        mma_commit(&bar.s_full[s]);
      };
      // the first half of P's keys is multiplied while the second is computed
      auto issue_pv = [&](int s, bool first, uint32_t parity) -> bool {
        if (!mbar_wait<SW>(&bar.p_full[s][0], parity, abort_flag, p.status, p.wait_limit_ns)) return false;
        if (!ring_wait()) return false;
        const uint64_t vd = vdesc0 + stage * (kTile >> 4);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_ts(tmem + 256 + s * 128, tmem + s * 128 + ks * 8, vd + desc_v_step(ks), kIdescPVh,
                 (!first || ks > 0) ? 1u : 0u);
        if (!mbar_wait<SW>(&bar.p_full[s][1], parity, abort_flag, p.status, p.wait_limit_ns)) return false;
        tc_fence_after();
#pragma unroll
        for (int ks = 4; ks < 8; ++ks)
          mma_ts(tmem + 256 + s * 128, tmem + s * 128 + ks * 8, vd + desc_v_step(ks), kIdescPVh, 1u);
        return true;
      };
      bool go = mbar_wait<SW>(&bar.q_full[0], 0, abort_flag, p.status, p.wait_limit_ns);
      const int ns = second ? 2 : 1;
      if (go && second) go = mbar_wait<SW>(&bar.q_full[1], 0, abort_flag, p.status, p.wait_limit_ns);
      if (go && (go = ring_wait())) {
        for (int s = 0; s < ns; ++s) issue_s(s);
        ring_next();
      }
      for (int i = 0; i < np && go; ++i) {
        // stage holds V of page i; K of the next page is one stage on
        for (int s = 0; s < ns && go; ++s) {
          if (!(go = issue_pv(s, i == 0, i & 1))) break;
          const uint32_t v_stage = stage, v_phase = phase;
          if (i + 1 < np) {
            if (s == ns - 1) {
              ring_next();
            } else if (++stage == kTileRing) {
              stage = 0;
              phase ^= 1;
            }
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
    float m_run = -INFINITY, l_run = 0.f;
    VRef<6, -6> vref;  // P below 2^8 (stale maximum) * 2^6 * 2, fp16; 2^-24 * 2^6 * 2^-6 is its smallest value

    bool ok = true;  // warp-uniform
    const int s = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int r = r0 + s * 128 + row;
    const bool row_valid = r < r1;
    // a warp without rows leaves its part of S and P as it is: only its own
    // rows of O depend on it
    const bool idle = !__any_sync(0xffffffffu, row_valid);
    const int tok = row_valid ? r / p.group : 0;
    const int64_t at = static_cast<int64_t>(head * p.group + (row_valid ? r % p.group : 0)) * p.n + st.t0 + tok;
    // a padded row sees all keys: it is computed and not stored
    const int limit = row_valid ? visible(first_pos + tok, st.len, p.unit) : st.len;
    float c_row = p.scale_log2;
    if (np > 0 && (s == 0 || second)) {
      // the row of Q to shared memory, as fp16 times a power of two
      uint4 w[16];
      const uint4* src = reinterpret_cast<const uint4*>(p.q + at * 128);
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        w[j] = row_valid ? __ldg(src + j) : make_uint4(0, 0, 0, 0);
        const uint32_t x[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          amax = max3f(amax, fabsf(__uint_as_float(x[e] << 16)), fabsf(__uint_as_float(x[e] & 0xffff0000u)));
      }
      const float shrink = row_shrink(amax, 0);
      c_row = p.scale_log2 / shrink;
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
    auto wait_warp = [&](uint64_t* bb, uint32_t parity) -> bool {
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait<SW>(bb, parity, abort_flag, p.status, p.wait_limit_ns));
      return ok;
    };
    const bool active = s == 0 || second;
    if (active && np > 0) {
      PageWindow<true> win(p, b, head, pg0, np, st.len);
      win.fetch(lane, p.status);
      for (int i = 0; i < np; ++i) {
        if ((i & 31) == 0) win.advance(i, lane, p.status);
        const int id = __shfl_sync(0xffffffffu, win.id, i & 31);
        const float ck = score_factor(c_row, __shfl_sync(0xffffffffu, win.ks, i & 31));
        const float o_ratio = vref.page(__shfl_sync(0xffffffffu, win.vs, i & 31));
        if (!wait_warp(&bar.s_full[s], i & 1)) break;
        if (idle) {
          mbar_arrive(&bar.p_full[s][0]);
          mbar_arrive(&bar.p_full[s][1]);
          continue;
        }
        tc_fence_after();
        const int key0 = (pg0 + i) * kPage;
        const int cut = id < 0 ? 0 : min(limit - key0, kPage);  // keys of the page that the row sees
        const uint32_t sc = tmem + lane_off + s * 128;
        float sv[2][64];
        tmem_ld64_wait(sc, sv[0]);
        tmem_ld64_wait(sc + 64, sv[1]);
        if (__any_sync(0xffffffffu, cut < kPage)) {
#pragma unroll
          for (int e = 0; e < 128; ++e)
            if (e >= cut) sv[e >> 6][e & 63] = -INFINITY;
        }
        const float mx = fmaxf(row_max_of(sv[0]), row_max_of(sv[1]));
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
        if (i > 0 && (o_ratio != 1.f || __any_sync(0xffffffffu, need))) {
          const float by = alpha * o_ratio;
#pragma unroll 1
          for (int cc = 0; cc < 8; ++cc) {
            uint32_t o[16];
            tmem_ld16_wait(tmem + lane_off + 256 + s * 128 + cc * 16, o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * by);
            tmem_st16(tmem + lane_off + 256 + s * 128 + cc * 16, o);
          }
        }
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
      wait_warp(&bar.o_full[s], 0);
      tc_fence_after();
    }

    // ---------------------------------------------------------- results
    const bool done = ok && *abort_flag == 0;
    const float unit = vref.unit();
    m_run += vref.raise();
    l_run *= vref.damp();
    if (done && active) {
      const bool some = np > 0 && l_run != 0.f;
      const float inv = some ? 1.f / l_run : 0.f;
      float* out = part + static_cast<int64_t>(behind) * part_floats(kTileRows);  // with splits
      if (row_valid) {
        if (splits > 1)
          *reinterpret_cast<float2*>(out + kTileRows * 128 + 2 * (s * 128 + row)) = make_float2(m_run, some ? l_run : 0.f);
        else if (p.lse)
          p.lse[at] = some ? (m_run + log2f(l_run)) * kLn2 : -INFINITY;
      }
      const bool patch = *const_cast<volatile int*>(&bar.nan_seen) != 0;
#pragma unroll 1
      for (int cc = 0; cc < 4; ++cc) {
        uint32_t o[32];
        if (np > 0) {
          tmem_ld32_wait(tmem + lane_off + 256 + s * 128 + cc * 32, o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * unit);
        if (patch && row_valid) {
          // NaN values that were taken out of pages that not every row sees whole
          uint32_t bad = 0;
          for (int key = max(least / kPage, pg0) * kPage; key < min(limit, (pg0 + np) * kPage); ++key) {
            const int id = __ldg(table + key / kPage - pg0);
            if (id < 0 || id >= p.n_pages) continue;
            const uint8_t* v = p.v8 + ((static_cast<int64_t>(id) * p.heads_kv + head) * kPage + key % kPage) * 128;
            for (int e = 0; e < 32; ++e)
              if ((v[cc * 32 + e] & 0x7f) == 0x7f) bad |= 1u << e;
          }
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (bad >> e & 1) o[e] = 0x7fffffffu;
        }
        if (!row_valid) continue;
        if (splits > 1) {
          uint4* dst = reinterpret_cast<uint4*>(out + (s * 128 + row) * 128 + cc * 32);
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

// Joins the splits of the rows: a warp per row.
constexpr int kJoinRows = 8;
__global__ void __launch_bounds__(32 * kJoinRows)
    cache_tile_join_kernel(const __grid_constant__ CacheAttnParams p, const TilePlan plan, const float* part) {
  const int lane = threadIdx.x & 31;
  const int nth = blockIdx.x / (kTileRows / kJoinRows);  // of the split tiles
  const int row = blockIdx.x % (kTileRows / kJoinRows) * kJoinRows + (threadIdx.x >> 5);
  const TileUnit u = tile_unit(p, plan, plan.whole + nth);
  const Stream st = stream_of(p.tok_start, p.kv_len, u.b, p.n, p.table_stride);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (st.bad || st.n_new > p.max_new) return;
  const int rows = st.n_new * p.group, tiles = (rows + kTileRows - 1) / kTileRows;
  if (u.rank >= tiles) return;
  const int r = tile_first_row(p, u, tiles) + row;
  if (r >= rows) return;
  join_row(
      p, static_cast<int64_t>(u.head * p.group + r % p.group) * p.n + st.t0 + r / p.group, lane, 0, plan.splits,
      [&](int i) { return part + (static_cast<int64_t>(nth) * plan.splits + i) * part_floats(kTileRows); }, row,
      kTileRows);
}

template <bool SW>
int launch(const CacheAttnParams& p, const TilePlan& plan, float* part, cudaStream_t stream) {
  static PerDeviceOnce once;
  const int rc = set_max_smem_once(reinterpret_cast<const void*>(cache_tile_kernel<SW>), TileLayout::kDynSmem, once);
  if (rc != CALIBATT_OK) return rc;
  // the register split needs the allotment it was sized for
  static std::once_flag regs_once;
  static int launch_regs = 0;
  std::call_once(regs_once, [] {
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, cache_tile_kernel<SW>) == cudaSuccess) launch_regs = fa.numRegs;
  });
  if (launch_regs * kTileThreads < kTileRegs) return CALIBATT_ERR_CUDA;
  const int64_t ctas = plan.whole + static_cast<int64_t>(plan.units - plan.whole) * plan.splits;
  cache_tile_kernel<SW><<<static_cast<unsigned>(ctas), kTileThreads, TileLayout::kDynSmem, stream>>>(p, plan, part);
  return cudaGetLastError() == cudaSuccess ? CALIBATT_OK : CALIBATT_ERR_CUDA;
}

}  // namespace

int launch_cache_attn_tiles(const CacheAttnParams& p, const TilePlan& plan, void* ws, cudaStream_t stream) {
  float* part = static_cast<float*>(ws);
  const int rc = p.wait_limit_ns < kShortWaitNs ? launch<true>(p, plan, part, stream)
                                                : launch<false>(p, plan, part, stream);
  if (rc != CALIBATT_OK || plan.whole == plan.units) return rc;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(plan.units - plan.whole) * (kTileRows / kJoinRows));
  cfg.blockDim = dim3(32 * kJoinRows);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_tile_join_kernel, p, plan, static_cast<const float*>(part)) ==
                 cudaSuccess
             ? CALIBATT_OK
             : CALIBATT_ERR_CUDA;
}

}  // namespace calibatt
