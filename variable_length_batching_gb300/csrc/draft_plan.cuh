// How attention of drafted tokens over a paged cache splits a ragged batch
// over a fixed grid, and which keys a drafted token sees.
//
// The work is a line of key tiles: sequence by sequence, within a sequence
// item by item (a key head, up to `heads` of its query heads, and a group of
// the sequence's new tokens), within an item tile by tile.  As for one new
// token per sequence (paged_plan.cuh), CTA c of n takes units
// [c W / n, (c + 1) W / n) of the line, so that every CTA reads the same
// number of keys however ragged the batch is, and lengths and offsets stay on
// the device.  Here the items of a sequence are as many as its tokens need; and
// where an item may have two row tiles over its keys, a tile of a sequence that
// needs both counts 5 and one of another 2, and belongs to the CTA that has its
// first unit (16 contexts, trees of 20 to 64 tokens, d = 128: 2.3 us against 0.8; 62
// contexts of 2,000 with one token beside two pieces of 256: 222 us all alike, 150
// with 5 and 3, 122 so).
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
  int light;                // tokens of one row tile, or 0: an item has but one
  bool few;                 // few enough sequences and units for a warp to plan
  unsigned int* status;
};

// A sequence's positions and new tokens; nothing (flagged) where its numbers
// do not fit together.
struct DraftSeq {
  int len, n, first;        // first: its first token in the packed batch
};
__device__ __forceinline__ DraftSeq draft_seq(const DraftBatch& a, int first, int hi, int len, unsigned int* status) {
  DraftSeq s;
  s.first = first;
  s.len = len;
  const bool bad = first < 0 || hi < first || hi > a.T || (int64_t)hi - first > a.max_new || len < hi - first ||
                   len > a.cap;
  if (bad) flag_device(status, kDevCheck);
  s.n = bad ? 0 : hi - first;
  return s;
}
__device__ __forceinline__ DraftSeq draft_seq(const DraftBatch& a, int b, unsigned int* status) {
  return draft_seq(a, a.cu[b], a.cu[b + 1], a.lengths[b], status);
}
// Items of a sequence, and the most of any.
inline int draft_items_most(const DraftBatch& a) {
  return a.Hkv * a.hgroups * ((a.max_new + a.tokens - 1) / a.tokens);
}
__device__ __forceinline__ int draft_items(const DraftBatch& a, int n) {
  return a.Hkv * a.hgroups * (n <= a.tokens ? 1 : (n + a.tokens - 1) / a.tokens);
}
constexpr int kHeavy = 5, kLight = 2;
__host__ __device__ __forceinline__ int draft_weight_most(const DraftBatch& a) { return a.light ? kHeavy : 1; }
// Units of a tile of a sequence of n new tokens.
__device__ __forceinline__ int draft_weight(const DraftBatch& a, int n) {
  return !a.light ? 1 : n > a.light ? kHeavy : kLight;
}
__device__ __forceinline__ int64_t draft_units(const DraftBatch& a, const DraftSeq& s, int tile, int extra) {
  return s.n > 0 ? (paged_tiles(s.len, tile) + extra) * draft_items(a, s.n) * draft_weight(a, s.n) : 0;
}

// The units of the call dealt out to n CTAs: CTA c has per of them, one more for
// the first rem CTAs.
struct DraftPlan {
  int64_t total, per, rem;
  int64_t lo, hi;           // this CTA's
  int64_t start;            // first unit of sequence b0, which holds lo
  int n, b0;
  DraftSeq seq;             // sequence b0
  // `least` units to a CTA, so that each has the first one of a tile; with fewer the last CTAs get none.
  __device__ __forceinline__ void deal(int64_t total_, int least, int cta, int ctas) {
    total = total_;
    n = (int)min64(ctas, total);
    if (least > 1 && total > 0 && (int64_t)n * least > total) n = (int)max64(1, total / least);
    per = n ? paged_div(total, n) : 0;
    rem = total - per * n;
    lo = cta < n ? per * cta + min64(cta, rem) : total;
    hi = cta < n ? lo + per + (cta < rem) : total;
  }
  // The CTA that has unit u.
  __device__ __forceinline__ int cta_of(int64_t u) const {
    const int64_t longer = rem * (per + 1);
    return (int)(u < longer ? paged_div(u, per + 1) : rem + paged_div(u - longer, per));
  }
};
struct DraftPlanSums {
  int64_t warp_sum[32];
  int64_t start;
  int b0;
};

// By a warp alone, without a barrier: batches of at most 128 sequences whose
// units are below 2^31 (a.few).  Every lane gets the plan.
constexpr int kPlanFew = 128;
__device__ __forceinline__ DraftPlan draft_plan_warp(const DraftBatch& a, int tile, int extra, int cta, int ctas,
                                                     unsigned int* status) {
  const int lane = threadIdx.x & 31, strip = (a.B + 31) >> 5, b_lo = lane * strip;
  DraftSeq q[kPlanFew / 32];
  int u[kPlanFew / 32], sum = 0;
#pragma unroll
  for (int k = 0; k < kPlanFew / 32; ++k) {
    u[k] = 0;
    if (k < strip && b_lo + k < a.B) {
      q[k] = draft_seq(a, b_lo + k, status);
      u[k] = (int)draft_units(a, q[k], tile, extra);
    }
    sum += u[k];
  }
  int inc = sum;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, inc, m);
    if (lane >= m) inc += o;
  }
  DraftPlan p;
  p.deal(__shfl_sync(0xffffffffu, inc, 31), draft_weight_most(a), cta, ctas);
  int at = inc - sum, b = -1;
  DraftSeq s = {0, 0, 0};
  const int lo = (int)p.lo;
#pragma unroll
  for (int k = 0; k < kPlanFew / 32; ++k) {
    if (b < 0 && lo >= at && lo < at + u[k]) {
      b = b_lo + k;
      s = q[k];
    } else if (b < 0) {
      at += u[k];
    }
  }
  const unsigned int who = __ballot_sync(0xffffffffu, b >= 0);
  const int from = who ? __ffs(who) - 1 : 0;
  p.b0 = __shfl_sync(0xffffffffu, b, from);
  p.start = __shfl_sync(0xffffffffu, at, from);
  p.seq.first = __shfl_sync(0xffffffffu, s.first, from);
  p.seq.len = __shfl_sync(0xffffffffu, s.len, from);
  p.seq.n = __shfl_sync(0xffffffffu, s.n, from);
  return p;
}

// Every thread of the CTA calls this (nthreads a multiple of 32, at most
// 1024); as paged_plan.
__device__ __forceinline__ DraftPlan draft_plan_cta(const DraftBatch& a, int tile, int extra, int cta, int ctas,
                                                    DraftPlanSums* s, int nthreads) {
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
  DraftPlan p;
  p.deal(total, draft_weight_most(a), cta, ctas);
  int64_t at = before + inc - sum;
  if (p.lo >= at && p.lo < at + sum) {
    int b = b_lo;
    if (strip > 1) {
      for (; b < b_hi; ++b) {
        const int64_t w = draft_units(a, draft_seq(a, b, nullptr), tile, extra);
        if (p.lo < at + w) break;
        at += w;
      }
    }
    s->b0 = b;
    s->start = at;
  }
  __syncthreads();
  p.b0 = s->b0;
  p.start = s->start;
  if (p.lo < p.hi) p.seq = draft_seq(a, p.b0, nullptr);
  return p;
}
__device__ __forceinline__ DraftPlan draft_plan(const DraftBatch& a, int tile, int extra, int cta, int ctas,
                                                DraftPlanSums* s, int nthreads) {
  if (a.few) return draft_plan_warp(a, tile, extra, cta, ctas, threadIdx.x < 32 ? a.status : nullptr);
  return draft_plan_cta(a, tile, extra, cta, ctas, s, nthreads);
}

// What an item of a sequence is.
struct DraftItem {
  int kvh, h0, nh;          // key head; first of its query heads, and how many
  int i0, ni;               // first token, and how many
};
__device__ __forceinline__ DraftItem draft_item(const DraftBatch& a, int n, int kvh, int hgroup, int group) {
  DraftItem it;
  it.kvh = kvh;
  it.h0 = hgroup * a.heads;
  it.nh = min(a.heads, a.G - it.h0);
  it.i0 = group * a.tokens;
  it.ni = min(a.tokens, n - it.i0);
  return it;
}
__device__ __forceinline__ DraftItem draft_item(const DraftBatch& a, int n, int item, int items) {
  const int groups = items / (a.Hkv * a.hgroups), head = item / groups, kvh = head / a.hgroups;
  return draft_item(a, n, kvh, head - kvh * a.hgroups, item - head * groups);
}

// Positions that the item's tokens see at most: without a mask none behind the last of them.
__device__ __forceinline__ int draft_visible(const DraftBatch& a, const DraftSeq& s, const DraftItem& it) {
  return a.bits ? s.len : s.len - s.n + it.i0 + it.ni;
}

// Walks a CTA's range segment by segment; as PagedWalk.  An item's share of the
// line is as long as its sequence; its last segment ends where its tokens see
// nothing more.
struct DraftWalk {
  int64_t left;           // units of the range not yet handed out
  int b, item, items;
  DraftSeq cur;
  int next_lo, next_hi, next_len;         // of sequence b + 1, loaded when b was reached
  int weight;             // units of a tile of sequence b
  int units;              // of an item of sequence b
  int unit;               // of the item, where the next segment starts
  int kvh, hgroup, group, groups;         // of the item: key head, group of its query heads, group of tokens of how many
  // the current segment: tiles [t0, t1) of item `it` (seg_item) of sequence seg_b
  DraftSeq seq;
  DraftItem it;
  int seg_b, seg_item, seg_items;
  int t0, t1;
  int end, last;          // where it ends in the item, and where the item's last tile does, in units
  bool begins, ends;

  __device__ __forceinline__ void load_next(const DraftBatch& a) {
    const bool there = b + 1 < a.B;
    next_lo = there ? a.cu[b + 1] : 0;
    next_hi = there ? a.cu[b + 2] : 0;
    next_len = there ? a.lengths[b + 1] : 0;
  }
  __device__ __forceinline__ void sequence(const DraftBatch& a, int tile, int extra) {
    groups = cur.n <= a.tokens ? 1 : (cur.n + a.tokens - 1) / a.tokens;
    items = a.Hkv * a.hgroups * groups;
    weight = draft_weight(a, cur.n);
    units = ((int)paged_tiles(cur.len, tile) + extra) * weight;
  }
  __device__ __forceinline__ void step_item(const DraftBatch& a) {
    ++item;
    if (++group == groups) {
      group = 0;
      if (++hgroup == a.hgroups) {
        hgroup = 0;
        ++kvh;
      }
    }
  }
  __device__ __forceinline__ void init(const DraftBatch& a, const DraftPlan& s, int tile, int extra) {
    left = s.hi - s.lo;
    if (left <= 0) return;
    b = s.b0;
    cur = s.seq;
    load_next(a);
    sequence(a, tile, extra);
    const int64_t off = s.lo - s.start;
    item = kvh = hgroup = group = 0;
    unit = (int)off;
    if (off >= units) {
      item = (int)paged_div(off, units);
      unit = (int)(off - (int64_t)item * units);
      const int head = item / groups;
      group = item - head * groups;
      kvh = head / a.hgroups;
      hgroup = head - kvh * a.hgroups;
    }
  }
  __device__ __forceinline__ bool next(const DraftBatch& a, int tile, int extra) {
    do {
      if (left <= 0) return false;
      if (item == items) {
        do {                              // the range holds a further unit, so a sequence with tokens follows
          if (++b >= a.B) return false;
          cur = draft_seq(a, next_lo, next_hi, next_len, nullptr);
          load_next(a);
        } while (cur.n == 0);
        item = group = hgroup = kvh = 0;
        sequence(a, tile, extra);
      }
      end = (int)min64(units, unit + left);
      seg_b = b;
      seg_item = item;
      seg_items = items;
      seq = cur;
      it = draft_item(a, cur.n, kvh, hgroup, group);
      last = units;
      if (groups > 1 && !a.bits) last = ((int)paged_tiles(draft_visible(a, cur, it), tile) + extra) * weight;
      int from = unit, to = min(end, last);           // in tiles
      if (weight > 1) {
        from = (from + weight - 1) / weight;
        to = (to + weight - 1) / weight;
      }
      t0 = max(0, from - extra);
      t1 = to - extra;
      begins = t0 == 0;
      ends = to * weight >= last;
      left -= end - unit;
      unit = 0;
      step_item(a);
    } while (t1 <= t0);                   // nothing but the item's extra units
    return true;
  }
  // CTAs that take tiles of the current segment's item, where it begins and does not end (so the range ends inside it)
  __device__ __forceinline__ int parts(const DraftPlan& s, int cta) const {
    return s.cta_of(s.hi + last - weight - end) - cta + 1;
  }
};

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
// The same from the token's mask words, read before.
struct DraftMask {
  uint64_t w[kDraftMaxNew / 64];
  __device__ __forceinline__ void read(const DraftBatch& a, const DraftSeq& s, int i, bool there) {
#pragma unroll
    for (int k = 0; k < kDraftMaxNew / 64; ++k)
      w[k] = there && a.bits && k < a.words ? (uint64_t)a.bits[((int64_t)s.first + i) * a.words + k] : 0;
  }
  __device__ __forceinline__ uint64_t sees(const DraftBatch& a, const DraftSeq& s, int i, int x) const {
    const int left = s.len - x, j = x - (s.len - s.n);
    if (left <= 0) return 0;
    const uint64_t all = left < 64 ? (1ull << left) - 1 : ~0ull;
    if (j <= -64) return all;
    if (!a.bits) {
      const int upto = i - j;
      return upto < 0 ? 0 : upto >= 63 ? all : all & ((2ull << upto) - 1);
    }
    if (j < 0) return all & ((1ull << -j) - 1 | w[0] << -j);
    const int k = j >> 6, sh = j & 63;
    uint64_t m = 0;
#pragma unroll
    for (int y = 0; y < kDraftMaxNew / 64; ++y) {
      if (y == k) m |= w[y] >> sh;
      if (y == k + 1 && sh) m |= w[y] << (64 - sh);
    }
    return all & m;
  }
  __device__ __forceinline__ bool sees_any(const DraftBatch& a, const DraftSeq& s) const {
    if (s.len > s.n || !a.bits) return true;
    bool any = false;
#pragma unroll
    for (int k = 0; k < kDraftMaxNew / 64; ++k) {
      const int n = s.n - 64 * k;
      if (n > 0 && (w[k] & (n < 64 ? (1ull << n) - 1 : ~0ull))) any = true;
    }
    return any;
  }
};
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
