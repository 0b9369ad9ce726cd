// The work of the cache attention kernels with one row tile per key head: all
// (stream, key head, page) triples as one list, cut into equal shares for a
// fixed number of CTAs. The streams' lengths are read on the device.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "cache.cuh"

namespace calibatt {

// Whether the kernels can take the stream: its lists fit, and its rows.
__device__ __forceinline__ bool stream_fits(const CacheAttnParams& p, const Stream& st) {
  return !st.bad && st.n_new <= p.max_new && static_cast<int64_t>(st.n_new) * p.group <= p.max_rows;
}

// Pages of a stream that its last new token sees (at least one, so that rows
// which see nothing are written), 0 for a stream without new tokens.
__device__ __forceinline__ int stream_pages(const CacheAttnParams& p, const Stream& st) {
  if (st.n_new == 0 || !stream_fits(p, st)) return 0;
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

// A stretch that is not all of its stream's pages: a CTA has two at most, its
// first, which begins inside the stream's pages, and its last, which begins
// with them. Per row 128 outputs, then maximum (log2 units) and sum of all rows.
__host__ __device__ constexpr int part_floats(int rows) { return rows * 130; }
__device__ __forceinline__ float* part_of(float* part, int cta, bool inside, int rows) {
  return part + (2 * static_cast<int64_t>(cta) + (inside ? 0 : 1)) * part_floats(rows);
}

}  // namespace calibatt
