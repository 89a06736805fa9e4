// How paged decode attention splits a ragged batch over a fixed grid.
//
// The work is a line of key tiles: sequence by sequence, within a sequence
// head item by head item (one key head with up to a fixed number of its query
// heads), within an item tile by tile.  CTA c of n takes tiles
// [c W / n, (c + 1) W / n): every CTA reads the same number of keys, however
// ragged the lengths, and the lengths stay on the device, so a captured
// launch follows them from replay to replay.  A CTA's range is a run of
// segments; only its first can continue an item begun by an earlier CTA and
// only its last can leave one unfinished, so two slots per CTA hold every
// partial result (slot 0: an item continued from an earlier CTA, slot 1: an
// item begun here and continued later) and a join over the CTAs finishes
// them.
#pragma once

#include "nt_common.cuh"

namespace nt {

// An item costs more than its tiles (query rows, merge, output): it counts as
// `extra` tiles more, in front of its first.  A CTA whose share ends among
// those takes nothing of the item.
struct PagedPlan {
  int64_t warp_sum[32];
  int64_t total, lo, hi;   // units of the call, this CTA's range
  int64_t start;           // first unit of sequence b0, which holds lo
  int b0;
};

__device__ __forceinline__ int paged_length(const int32_t* lengths, int b, int64_t cap, unsigned int* status) {
  const int n = lengths[b];
  if (n < 0 || n > cap) {
    flag_device(status, kDevCheck);
    return n < 0 ? 0 : (int)cap;
  }
  return n;
}
// (unsigned: len + tile passes 2^31 for the longest)
__device__ __forceinline__ int64_t paged_tiles(int len, int tile) { return ((uint32_t)len + tile - 1) / tile; }

// Units of a sequence's items.
__device__ __forceinline__ int64_t paged_units(int len, int tile, int items, int extra) {
  return len > 0 ? (paged_tiles(len, tile) + extra) * items : 0;
}
// floor(a / b), in 32 bits where that does (a 64-bit division takes a hundred
// cycles, and every CTA waits for three of them before its first load)
__device__ __forceinline__ int64_t paged_div(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// CTAs that share the units, and the first unit of CTA c of them.
__device__ __forceinline__ int64_t paged_ctas(int64_t total, int ctas) { return max64(1, min64(ctas, total)); }
__device__ __forceinline__ int64_t paged_first(int64_t total, int64_t n, int64_t c) { return paged_div(total * c, n); }

// Every thread of the CTA calls this (nthreads a multiple of 32, at most
// 1024): each sums a strip of the sequences (for up to nthreads of them one
// coalesced load, whose latency is most of what this costs), the strips are
// scanned, and the thread whose strip holds the CTA's first unit walks to its
// sequence.
__device__ __forceinline__ void paged_plan(const int32_t* lengths, int B, int64_t cap, int items, int tile, int extra,
                                           int cta, int ctas, PagedPlan* s, unsigned int* status, int nthreads) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = nthreads >> 5;
  const int strip = (B + nthreads - 1) / nthreads;
  const int b_lo = min(B, tid * strip), b_hi = min(B, b_lo + strip);
  int64_t sum = 0;
  for (int b = b_lo; b < b_hi; ++b) sum += paged_units(paged_length(lengths, b, cap, status), tile, items, extra);
  int64_t inc = sum;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, inc, m);
    if (lane >= m) inc += o;
  }
  if (lane == 31) s->warp_sum[warp] = inc;
  __syncthreads();
  int64_t before = 0, total = 0;
  for (int w = 0; w < warps; ++w) {
    const int64_t x = s->warp_sum[w];
    if (w < warp) before += x;
    total += x;
  }
  // with fewer units than CTAs the last CTAs get none, so that no CTA without
  // work lies between two that share an item
  const int64_t n = paged_ctas(total, ctas), c = min64(cta, n), c1 = min64(cta + 1, n);
  const int64_t lo = paged_first(total, n, c);
  int64_t at = before + inc - sum;
  if (lo >= at && lo < at + sum) {
    int b = b_lo;
    if (strip > 1) {
      for (; b < b_hi; ++b) {
        const int64_t w = paged_units(paged_length(lengths, b, cap, nullptr), tile, items, extra);
        if (lo < at + w) break;
        at += w;
      }
    }
    s->b0 = b;
    s->start = at;
  }
  if (tid == 0) {
    s->total = total;
    s->lo = lo;
    s->hi = paged_first(total, n, c1);
  }
  __syncthreads();
}

// Walks a CTA's range segment by segment.  With `whole`, items are not split:
// the CTA takes those that start in its range, to their end.
struct PagedWalk {
  bool whole;
  int64_t left;           // units of the range not yet handed out
  int b, item, len;
  int len_after;          // of sequence b + 1, loaded when b was reached
  int64_t units;          // of an item of sequence b
  int64_t unit;           // of the item, where the next segment starts
  // the current segment: tiles [t0, t1) of item seg_item of sequence seg_b
  int seg_b, seg_item, seg_len;
  int64_t t0, t1;
  bool begins, ends;

  __device__ __forceinline__ void init(const PagedPlan& s, const int32_t* lengths, int B, int64_t cap,
                                       int tile_keys, int extra, bool whole_items) {
    whole = whole_items;
    left = s.hi - s.lo;
    if (left <= 0) return;
    b = s.b0;
    len = paged_length(lengths, b, cap, nullptr);
    len_after = b + 1 < B ? paged_length(lengths, b + 1, cap, nullptr) : 0;
    units = paged_tiles(len, tile_keys) + extra;
    const int64_t off = s.lo - s.start;
    item = (int)paged_div(off, units);
    unit = off - item * units;
    if (whole && unit > 0) {
      left -= units - unit;
      unit = 0;
      ++item;
    }
  }
  __device__ __forceinline__ bool next(const int32_t* lengths, int B, int64_t cap, int items, int tile_keys,
                                       int extra) {
    do {
      if (left <= 0) return false;
      if (item == items) {
        item = 0;
        do {                              // the range holds a further unit, so a longer sequence follows
          if (++b >= B) return false;
          len = len_after;
          len_after = b + 1 < B ? paged_length(lengths, b + 1, cap, nullptr) : 0;
        } while (len == 0);
        units = paged_tiles(len, tile_keys) + extra;
      }
      const int64_t end = whole ? units : min64(units, unit + left);
      seg_b = b;
      seg_item = item;
      seg_len = len;
      t0 = max64(0, unit - extra);
      t1 = end - extra;
      begins = t0 == 0;
      ends = end == units;
      left -= end - unit;
      unit = 0;
      ++item;
    } while (t1 <= t0);                   // nothing but the item's extra units
    return true;
  }
  // CTAs that take tiles of the current segment's item, for a segment that
  // begins its item and does not end it (so the range ends inside it): the
  // item ends at unit e of the call, and CTA c starts in front of e when
  // floor(total c / n) < e.
  __device__ __forceinline__ int parts(const PagedPlan& s, int extra, int cta, int ctas) const {
    const int64_t n = paged_ctas(s.total, ctas), e = s.hi + units - (t1 + extra);
    return (int)paged_div(e * n + s.total - 1, s.total) - cta;
  }
};

// Whether a call keeps its items whole: when the longest the tables allow is
// so short that one CTA reads it in about the time the join's launch costs
// (16 contexts of 300 keys, 8 key heads of 128: 10.0 us whole, 12.6 split; one
// of 1,000 with two heads of 64, the worst case: 8.4 and 6.9).
constexpr int64_t kPagedWholeBytes = 256 * 1024;
inline bool paged_whole_items(const PagedAttnProblem& p, int elem) {
  return (int64_t)p.max_pages * p.pool.page_size * p.d * 2 * elem <= kPagedWholeBytes;
}

// The partials in the workspace: per CTA the item that it begins and leaves
// unfinished (b * items + item, -1 none) and how many CTAs share that item;
// then per slot a (max, sum) pair for each query head of an item, the max in
// base-2 logarithms, and the heads' d unnormalised fp32 outputs.  Slot 2 c of
// CTA c holds an item begun by an earlier CTA, slot 2 c + 1 one begun there.
struct PagedPartials {
  int64_t* id;
  float* ml;
  float* o;
};
__host__ __device__ __forceinline__ PagedPartials paged_partials(void* ws, int ctas, int heads) {
  PagedPartials p;                    // each part a multiple of 16 bytes
  p.id = static_cast<int64_t*>(ws);
  p.ml = reinterpret_cast<float*>(p.id + 2 * (int64_t)ctas);
  p.o = p.ml + 2 * (int64_t)ctas * heads * 2;
  return p;
}

// Joins the items that the split left unfinished; `heads` is the most query
// heads an item takes (the partials hold min(heads, G)).
cudaError_t launch_paged_join(nt_dtype dt, const PagedAttnProblem& p, int ctas, int items, int heads, cudaStream_t s);

}  // namespace nt
