// How attention of drafted tokens over a paged cache splits a ragged batch
// over a fixed grid, and which keys a drafted token sees.
//
// The work is a line of key tiles: sequence by sequence, within a sequence
// item by item (a key head, up to `heads` of its query heads, and a group of
// the sequence's new tokens), within an item tile by tile.  As for one new
// token per sequence (paged_plan.cuh), CTA c of n takes units
// [c W / n, (c + 1) W / n) of the line, so that every CTA reads the same
// number of keys however ragged the batch is, and lengths and offsets stay on
// the device.  Here the items of a sequence are as many as its tokens need.
#pragma once

#include "paged_plan.cuh"

namespace nt {

// The batch as the kernels see it.  Rows of an item are its tokens' query
// heads, token by token.
struct DraftBatch {
  const int32_t* cu;        // [B + 1] offsets of the new tokens
  const int32_t* lengths;   // [B] positions, the new tokens' among them
  const int32_t* table;
  const int64_t* bits;      // [T, words]: the new tokens that a token sees, or NULL: itself and those before it
  int B, max_new, words;
  int64_t T, cap;           // packed tokens; positions a table holds
  int max_pages, page_size, n_pages;
  int H, G, Hkv;
  int heads, hgroups;       // query heads of an item, and groups of them to a key head
  int tokens;               // of an item
  unsigned int* status;
};

// A sequence's positions and new tokens; nothing (flagged) where its numbers
// do not fit together.
struct DraftSeq {
  int len, n, first;        // first: its first token in the packed batch
};
__device__ __forceinline__ DraftSeq draft_seq(const DraftBatch& a, int b, unsigned int* status) {
  DraftSeq s;
  s.first = a.cu[b];
  const int hi = a.cu[b + 1];
  s.len = a.lengths[b];
  const bool bad = s.first < 0 || hi < s.first || hi > a.T || (int64_t)hi - s.first > a.max_new ||
                   s.len < hi - s.first || s.len > a.cap;
  if (bad) flag_device(status, kDevCheck);
  s.n = bad ? 0 : hi - s.first;
  return s;
}
__device__ __forceinline__ int draft_items(const DraftBatch& a, int n) {
  return a.Hkv * a.hgroups * ((n + a.tokens - 1) / a.tokens);
}
__device__ __forceinline__ int64_t draft_units(const DraftBatch& a, const DraftSeq& s, int tile, int extra) {
  return s.n > 0 ? (paged_tiles(s.len, tile) + extra) * draft_items(a, s.n) : 0;
}

// Every thread of the CTA calls this (nthreads a multiple of 32, at most
// 1024); as paged_plan.
__device__ __forceinline__ void draft_plan(const DraftBatch& a, int tile, int extra, int cta, int ctas, PagedPlan* s,
                                           int nthreads) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = nthreads >> 5;
  const int strip = (a.B + nthreads - 1) / nthreads;
  const int b_lo = (int)min64(a.B, (int64_t)tid * strip), b_hi = (int)min64(a.B, (int64_t)b_lo + strip);
  int64_t sum = 0;
  for (int b = b_lo; b < b_hi; ++b) sum += draft_units(a, draft_seq(a, b, a.status), tile, extra);
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
  const int64_t n = paged_ctas(total, ctas), c = min64(cta, n), c1 = min64(cta + 1, n);
  const int64_t lo = paged_first(total, n, c);
  int64_t at = before + inc - sum;
  if (lo >= at && lo < at + sum) {
    int b = b_lo;
    if (strip > 1) {
      for (; b < b_hi; ++b) {
        const int64_t w = draft_units(a, draft_seq(a, b, nullptr), tile, extra);
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

// Walks a CTA's range segment by segment; as PagedWalk.
struct DraftWalk {
  bool whole;
  int64_t left;           // units of the range not yet handed out
  int b, item, items;
  DraftSeq cur;
  int64_t units;          // of an item of sequence b
  int64_t unit;           // of the item, where the next segment starts
  // the current segment: tiles [t0, t1) of item seg_item of sequence b's
  DraftSeq seq;
  int seg_b, seg_item, seg_items;
  int64_t t0, t1;
  bool begins, ends;

  __device__ __forceinline__ void init(const DraftBatch& a, const PagedPlan& s, int tile, int extra, bool whole_items) {
    whole = whole_items;
    left = s.hi - s.lo;
    if (left <= 0) return;
    b = s.b0;
    cur = draft_seq(a, b, nullptr);
    items = draft_items(a, cur.n);
    units = paged_tiles(cur.len, tile) + extra;
    const int64_t off = s.lo - s.start;
    item = (int)paged_div(off, units);
    unit = off - item * units;
    if (whole && unit > 0) {
      left -= units - unit;
      unit = 0;
      ++item;
    }
  }
  __device__ __forceinline__ bool next(const DraftBatch& a, int tile, int extra) {
    do {
      if (left <= 0) return false;
      if (item == items) {
        item = 0;
        do {                              // the range holds a further unit, so a sequence with tokens follows
          if (++b >= a.B) return false;
          cur = draft_seq(a, b, nullptr);
        } while (cur.n == 0);
        items = draft_items(a, cur.n);
        units = paged_tiles(cur.len, tile) + extra;
      }
      const int64_t end = whole ? units : min64(units, unit + left);
      seg_b = b;
      seg_item = item;
      seg_items = items;
      seq = cur;
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
  // CTAs that take tiles of the current segment's item, where it begins and does not end; as PagedWalk::parts
  __device__ __forceinline__ int parts(const PagedPlan& s, int extra, int cta, int ctas) const {
    const int64_t n = paged_ctas(s.total, ctas), e = s.hi + units - (t1 + extra);
    return (int)paged_div(e * n + s.total - 1, s.total) - cta;
  }
};

// What an item of a sequence is.
struct DraftItem {
  int kvh, h0, nh;          // key head; first of its query heads, and how many
  int i0, ni;               // first token, and how many
};
__device__ __forceinline__ DraftItem draft_item(const DraftBatch& a, int n, int item, int items) {
  const int groups = items / (a.Hkv * a.hgroups);
  const int rest = item / groups;
  DraftItem it;
  it.i0 = (item - rest * groups) * a.tokens;
  it.ni = min(a.tokens, n - it.i0);
  it.kvh = rest / a.hgroups;
  it.h0 = (rest - it.kvh * a.hgroups) * a.heads;
  it.nh = min(a.heads, a.G - it.h0);
  return it;
}

// The keys that new token i of a sequence sees among positions [x, x + 64), a
// bit each.  x may lie behind the sequence's end.
__device__ __forceinline__ uint64_t draft_sees(const DraftBatch& a, const DraftSeq& s, int i, int64_t x) {
  const int64_t left = s.len - x;
  if (left <= 0) return 0;
  const uint64_t there = left < 64 ? (1ull << left) - 1 : ~0ull;
  const int64_t j = x - (s.len - s.n);                 // the first of them as a new token
  if (j <= -64) return there;
  if (!a.bits) {
    const int64_t upto = i - j;                        // the last one seen, from x
    return upto < 0 ? 0 : upto >= 63 ? there : there & ((2ull << upto) - 1);
  }
  const int64_t* w = a.bits + ((int64_t)s.first + i) * a.words;
  if (j < 0) return there & ((1ull << -j) - 1 | (uint64_t)w[0] << -j);
  const int k = (int)(j >> 6), sh = (int)(j & 63);
  uint64_t m = k < a.words ? (uint64_t)w[k] >> sh : 0;
  if (sh && k + 1 < a.words) m |= (uint64_t)w[k + 1] << (64 - sh);
  return there & m;
}
// Whether it sees any.
__device__ __forceinline__ bool draft_sees_any(const DraftBatch& a, const DraftSeq& s, int i) {
  if (s.len > s.n || !a.bits) return true;
  for (int x = 0; x < s.n; x += 64)
    if (draft_sees(a, s, i, x)) return true;
  return false;
}

// The partials in the workspace; as PagedPartials, with `rows` rows to a slot
// and the sequence and item of what a CTA leaves unfinished beside the count of
// the CTAs that share it.
struct DraftPartials {
  int4* open;               // per CTA: sequence (-1 none), item, items, CTAs
  float* ml;
  float* o;
};
__host__ __device__ __forceinline__ DraftPartials draft_partials(void* ws, int ctas, int rows) {
  DraftPartials p;
  p.open = static_cast<int4*>(ws);
  p.ml = reinterpret_cast<float*>(p.open + ctas);
  p.o = p.ml + 2 * (int64_t)ctas * rows * 2;
  return p;
}

// Joins the items that a split into `ctas` parts left unfinished; `rows` rows
// to a partial result.
cudaError_t launch_draft_join(nt_dtype dt, const DraftBatch& a, int d, int ctas, int rows, void* workspace, void* o,
                              float* lse, cudaStream_t s);

}  // namespace nt
