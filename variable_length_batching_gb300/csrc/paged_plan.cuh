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

struct PagedPlanShared {
  int64_t warp_sum[32];
  int64_t total, lo, hi;   // tiles of the call, this CTA's range
  int64_t start;           // first tile of sequence b0
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
__device__ __forceinline__ int64_t paged_tiles(int len, int tile) { return (len + tile - 1) / tile; }

// Every thread of the CTA calls this (nthreads a multiple of 32, at most
// 1024): each sums a strip of the sequences, the strips are scanned, and the
// thread whose strip holds the CTA's first tile walks to its sequence.
__device__ inline void paged_plan(const int32_t* lengths, int B, int64_t cap, int items, int tile, int cta, int ctas,
                                  PagedPlanShared* s, unsigned int* status, int nthreads) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = nthreads >> 5;
  const int strip = (B + nthreads - 1) / nthreads;
  const int b_lo = min(B, tid * strip), b_hi = min(B, b_lo + strip);
  int64_t sum = 0;
  for (int b = b_lo; b < b_hi; ++b) sum += paged_tiles(paged_length(lengths, b, cap, status), tile);
  sum *= items;
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
    if (w < warp) before += s->warp_sum[w];
    total += s->warp_sum[w];
  }
  // with fewer tiles than CTAs the last CTAs get none, so that no CTA without
  // work lies between two that share an item
  const int64_t n = max64(1, min64(ctas, total)), c = min64(cta, n), c1 = min64(cta + 1, n);
  const int64_t lo = total / n * c + total % n * c / n;
  const int64_t hi = total / n * c1 + total % n * c1 / n;
  int64_t at = before + inc - sum;
  if (lo >= at && lo < at + sum) {
    int b = b_lo;
    for (; b < b_hi; ++b) {
      const int64_t w = paged_tiles(paged_length(lengths, b, cap, nullptr), tile) * items;
      if (lo < at + w) break;
      at += w;
    }
    s->b0 = b;
    s->start = at;
  }
  if (tid == 0) {
    s->total = total;
    s->lo = lo;
    s->hi = hi;
  }
  __syncthreads();
}

// Walks a CTA's range segment by segment.
struct PagedWalk {
  int64_t left;           // tiles of the range not yet handed out
  int b, item, len;
  int64_t tiles, tile;    // tiles of sequence b; first tile of the next segment
  // the current segment
  int seg_b, seg_item, seg_len;
  int64_t t0, t1;
  bool begins, ends;

  __device__ __forceinline__ void init(const PagedPlanShared* s, const int32_t* lengths, int64_t cap, int tile_keys) {
    left = s->hi - s->lo;
    if (left <= 0) return;
    b = s->b0;
    len = paged_length(lengths, b, cap, nullptr);
    tiles = paged_tiles(len, tile_keys);
    const int64_t off = s->lo - s->start;
    item = (int)(off / tiles);
    tile = off % tiles;
  }
  __device__ __forceinline__ bool next(const int32_t* lengths, int B, int64_t cap, int items, int tile_keys) {
    if (left <= 0) return false;
    if (item == items) {
      item = 0;
      do {                              // the range holds a further tile, so a longer sequence follows
        if (++b >= B) return false;
        len = paged_length(lengths, b, cap, nullptr);
      } while (len == 0);
      tiles = paged_tiles(len, tile_keys);
    }
    seg_b = b;
    seg_item = item;
    seg_len = len;
    t0 = tile;
    t1 = min64(tiles, tile + left);
    begins = t0 == 0;
    ends = t1 == tiles;
    left -= t1 - t0;
    tile = 0;
    ++item;
    return true;
  }
};

// The partials in the workspace: per slot (two per CTA) the item it belongs
// to (b * items + item, -1 none), then a (max, sum) pair per query head of an
// item (the max in base-2 logarithms), then the heads' d unnormalised fp32
// outputs.
struct PagedPartials {
  int64_t* id;
  float* ml;
  float* o;
};
__host__ __device__ __forceinline__ PagedPartials paged_partials(void* ws, int ctas, int heads) {
  PagedPartials p;
  p.id = static_cast<int64_t*>(ws);
  p.ml = reinterpret_cast<float*>(p.id + 2 * (int64_t)ctas);
  p.o = p.ml + 2 * (int64_t)ctas * heads * 2;
  return p;
}

// Joins the items that the split left unfinished; `heads` is the most query
// heads an item takes (the partials hold min(heads, G)).
cudaError_t launch_paged_join(nt_dtype dt, const PagedAttnProblem& p, int ctas, int items, int heads, cudaStream_t s);

}  // namespace nt
