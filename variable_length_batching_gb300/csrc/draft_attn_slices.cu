// Attention of drafted tokens over a paged cache, few rows to a key head (up to
// 64 of tokens times query heads): bf16, pages of a multiple of 8 positions.
//
// Up to some 50 rows the cache's bytes are the bound even for mma.sync, which
// does 983 multiply-adds a cycle here (a key and its value take 3 d of them
// for each row: scores, and values by two parts of P).  So, as for one new token
// per sequence (paged_attn_tma.cu), the kernel is a stream of TMA loads: two
// producer warps walk the CTA's share of the batch (draft_plan.cuh) tile by
// tile into a ring of stages, and eight warps each take 16 keys of a tile and
// 16 rows with a running maximum, sum and output of their own in registers;
// no warp waits for another until the end of a segment, where their results are
// merged.  The tensor-memory kernel (draft_attn_tc.cu) has 128 rows to a tile,
// and two hand-offs between warps for every 128 keys; it takes over where more
// rows than 64 pay for that (152 contexts of 8,000 keys, 16 rows: d = 64 69 us
// there, d = 128 103).
//
// RG row groups of 16 (1, 2 or 4) share the eight warps with 8 / RG slices of
// the keys.  A row's mask words are fetched with the queries.  Values that are
// not finite are taken out of a tile that new tokens are in, and added to the
// rows that see them when results are merged (draft_attn_rows.cu says why).
#include "draft_plan.cuh"
#include "draft_worker.cuh"

namespace nt {
namespace {

using namespace draft;

constexpr int kConsumers = 8;               // warps
constexpr int kProducers = 2;               // warps, tiles alternating
constexpr int kThreads = (kConsumers + kProducers + 1) * 32;
constexpr int kWords = kDraftMaxNew / 64;
constexpr int kBadWords = 10;               // new tokens, from the 16 keys that the first of them is in

template <int D, int RG>
struct Cfg {
  static constexpr int kRows = 16 * RG;
  static constexpr int kUnits = kConsumers / RG;              // warps of one row group
  static constexpr int kTile = D == 32 ? 128 : D == 128 && RG == 4 ? 32 : 64;      // keys of a stage, 16 KB or so
  static constexpr int kSlices = kTile / 16;
  static constexpr int kGroups = kUnits > kSlices ? kUnits / kSlices : 1;          // stages worked on at once
  static constexpr int kTurns = kUnits > kSlices ? 1 : kSlices / kUnits;           // slices of a stage to a warp
  static constexpr uint32_t kRow = D * 2;
  static constexpr uint32_t kSide = kTile * kRow, kStage = 2 * kSide;
  static constexpr int kRedStride = D + 4;                    // floats: keeps the results' writes conflict-free
  static constexpr uint32_t kRed = kUnits * kRows * kRedStride * 4;
  static constexpr int kQSlots = 4 / RG > 2 ? 4 / RG : 2;     // items whose queries are in flight or in use
  static constexpr uint32_t kQBytes = kRows * kRow, kMask = kRows * kWords * 8;
  static constexpr uint32_t kFixed = kRed + kQSlots * (kQBytes + kMask) + 4096;
  // a multiple of the groups and of the producers, so that a stage is always the same warps' (paged_attn_tma.cu)
  static constexpr int kRound = kGroups > kProducers ? kGroups : kProducers;
  static constexpr int kFit = (int)((226 * 1024 - 1024 - kFixed) / kStage);
  static constexpr int kStages = (kFit < 16 ? kFit : 16) / kRound * kRound;
  static constexpr uint32_t kSmem = 1024 + kStages * kStage + kFixed;
  static constexpr int kExtra = 2;                            // an item's cost beside its tiles, in tiles
  static_assert(kStages >= 4 && kSmem <= 227 * 1024, "shared memory");
};

struct Ctl {
  uint64_t full[16], empty[16], q_full[4], q_empty[4], red_full;
  float m[kConsumers][16], l[kConsumers][16];       // of a unit's rows
  unsigned int bad[2][kBadWords + 1];               // of two segments in turn: keys, and whether any
  PagedPlan plan;
  int abort;
};
static_assert(sizeof(Ctl) <= 4096, "control block");

struct SliceArgs {
  DraftBatch a;
  const uint8_t* v;
  bf16* o;
  float* lse;
  void* workspace;
  bool whole;                     // items are not split
  int box;                        // keys per box
  float scale_log2;
};

// Keys [x, x + 16) that a row sees, from its mask words in shared memory.
__device__ __forceinline__ uint32_t sees16(const DraftBatch& a, const DraftSeq& s, int i, const unsigned long long* words,
                                           int x) {
  const int left = s.len - x, j = x - (s.len - s.n);
  const uint32_t there = left >= 16 ? 0xffffu : (1u << max(left, 0)) - 1;
  if (j <= -16) return there;
  if (!a.bits) {
    const int upto = i - j;                         // the last one seen, from x
    return upto < 0 ? 0 : upto >= 15 ? there : there & ((2u << upto) - 1);
  }
  if (j < 0) return there & ((1u << -j) - 1 | (uint32_t)(words[0] << -j));
  const int k = j >> 6, sh = j & 63;
  uint64_t m = k < a.words ? words[k] >> sh : 0;
  if (sh && k + 1 < a.words) m |= words[k + 1] << (64 - sh);
  return there & (uint32_t)m;
}

// A warp's 16 rows and their running statistics; a lane has two, g and g + 8.
template <int D, int RG>
struct Part {
  using C = Cfg<D, RG>;
  static constexpr uint32_t kBoxRow = D < 64 ? D * 2 : 128;   // bytes of a key in a box's columns
  uint32_t qa[D / 16][4];
  float m[2], l[2], o[D / 8][4];
  int g, tq;
  uint32_t hs;                     // to a box's next 64 columns
  int box;                         // a power of two

  __device__ __forceinline__ explicit Part(int box_) : box(box_) {
    const int lane = threadIdx.x & 31;
    g = lane >> 2;
    tq = lane & 3;
    hs = box * 128;
  }
  __device__ __forceinline__ uint32_t row_at(int r) const {
    return (uint32_t)(r & -box) * C::kRow + (r & (box - 1)) * kBoxRow;
  }
  __device__ __forceinline__ static int swizzle(int r) { return D < 64 ? (r >> 1) & 3 : r & 7; }
  // rows `first` to first + 15 of the item's, as TMA laid them down (those behind its last hold anything)
  __device__ __forceinline__ void load_q(uint32_t rows, int first) {
    const int lane = threadIdx.x & 31, row = first + (lane & 15);
    const uint32_t at = rows + row * kBoxRow, x = ((lane >> 4) ^ swizzle(row)) << 4;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
      ldsm4(at + (ks >> 2) * C::kRows * 128 + ((((uint32_t)ks & 3) << 5) ^ x), qa[ks]);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[i][c] = 0.f;
  }
  // Slice `slice` of the stage; `all`: every row sees every key, else the rows' masks in `see`.
  __device__ __forceinline__ void tile(uint32_t kbase, int slice, bool all, const uint32_t (&see)[2], float scale_log2) {
    const int lane = threadIdx.x & 31;
    const uint32_t vbase = kbase + C::kSide;
    const int krow = slice * 16 + ((lane >> 4) << 3) + (lane & 7), vrow = slice * 16 + (lane & 15);
    const uint32_t k_at = kbase + row_at(krow), v_at = vbase + row_at(vrow);
    const uint32_t kx = (((lane >> 3) & 1) ^ swizzle(krow)) << 4, vx = ((lane >> 4) ^ swizzle(vrow)) << 4;
    // two chains for each eight keys
    float s[2][4] = {}, s2[2][4] = {};
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t b[4];
      ldsm4(k_at + (ks >> 2) * hs + ((((uint32_t)ks & 3) << 5) ^ kx), b);
      mma16816(ks & 1 ? s2[0] : s[0], qa[ks], b[0], b[1]);
      mma16816(ks & 1 ? s2[1] : s[1], qa[ks], b[2], b[3]);
    }
    uint32_t ph[4], pl[4];
    float corr[2];
    bool moved = false;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        v[c] = (s[c >> 1][2 * r + (c & 1)] + s2[c >> 1][2 * r + (c & 1)]) * scale_log2;
        if (!all && !(see[r] >> ((c >> 1) * 8 + 2 * tq + (c & 1)) & 1)) v[c] = -INFINITY;
      }
      float mx = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m[r], mx), base = mn == -INFINITY ? 0.f : mn;
      moved |= mn > m[r];
      corr[r] = ex2_approx(m[r] - base);
      m[r] = mn;
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = ex2_approx(v[c] - base);
      l[r] = l[r] * corr[r] + (v[0] + v[1]) + (v[2] + v[3]);
      Worker<bf16, D, 8>::split(v[0], v[1], ph[r], pl[r]);
      Worker<bf16, D, 8>::split(v[2], v[3], ph[2 + r], pl[2 + r]);
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][0] *= corr[0];
        o[i][1] *= corr[0];
        o[i][2] *= corr[1];
        o[i][3] *= corr[1];
      }
    }
    // two column blocks at a time: a product does not wait for the one before it
#pragma unroll
    for (int i = 0; i < D / 16; i += 2) {
      uint32_t b[2][4];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        ldsm4_t(v_at + ((i + k) >> 2) * hs + ((((uint32_t)(i + k) & 3) << 5) ^ vx), b[k]);
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          mma16816(o[2 * (i + k)], part ? pl : ph, b[k][0], b[k][1]);
          mma16816(o[2 * (i + k) + 1], part ? pl : ph, b[k][2], b[k][3]);
        }
    }
  }
  // V of a slice as the products may read it: rows behind the last key become zeros, values that are not finite are
  // taken out (their keys in `found`).
  __device__ __forceinline__ uint32_t clean(uint8_t* stage, int slice, int left) const {
    const int lane = threadIdx.x & 31;
    uint32_t found = 0;
    for (int e = lane; e < 16 * (D / 8); e += 32) {
      const int key = e / (D / 8), ch = e % (D / 8);
      uint8_t* at = stage + C::kSide + row_at(slice * 16 + key) + (ch >> 3) * hs + (ch & 7) * 16;
      if (key >= left) *reinterpret_cast<uint4*>(at) = make_uint4(0, 0, 0, 0);
      else if (clear_bad<bf16>(at)) found |= 1u << key;
    }
    __syncwarp();
    return __reduce_or_sync(0xffffffffu, found);
  }
  // the warp's results: maxima and sums (-1: no keys, nothing to add), outputs [16][kRedStride]
  __device__ __forceinline__ void result(float* rm, float* rl, float* ro, bool active) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (tq == 0) {
        rm[g + 8 * r] = m[r];
        rl[g + 8 * r] = active ? l[r] : -1.f;
      }
      if (!active) continue;
      float* to = ro + (g + 8 * r) * C::kRedStride + 2 * tq;
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<float2*>(to + i * 8) = make_float2(o[i][2 * r], o[i][2 * r + 1]);
    }
  }
};

template <int D, int RG>
__global__ void __launch_bounds__(kThreads, 1)
draft_slices_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap, const SliceArgs p) {
  using C = Cfg<D, RG>;
  constexpr int S = C::kStages, kTile = C::kTile, kE = C::kExtra;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  uint8_t* stages = smem;
  float* red = reinterpret_cast<float*>(smem + S * C::kStage);
  uint8_t* qbuf = reinterpret_cast<uint8_t*>(red) + C::kRed;
  unsigned long long* masks = reinterpret_cast<unsigned long long*>(qbuf + C::kQSlots * C::kQBytes);
  Ctl* ctl = reinterpret_cast<Ctl*>(reinterpret_cast<uint8_t*>(masks) + C::kQSlots * C::kMask);
  const DraftBatch& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const DraftPartials part = draft_partials(p.workspace, gridDim.x, C::kRows);

  if (threadIdx.x < S) {
    mbar_init(&ctl->full[threadIdx.x], 1);
    mbar_init(&ctl->empty[threadIdx.x], C::kGroups > 1 ? C::kSlices * RG : kConsumers);
  }
  if (threadIdx.x < C::kQSlots) {
    mbar_init(&ctl->q_full[threadIdx.x], 1);
    mbar_init(&ctl->q_empty[threadIdx.x], kConsumers);
  }
  if (threadIdx.x == 0) {
    mbar_init(&ctl->red_full, kConsumers);
    for (int i = 0; i < 2; ++i)
      for (int k = 0; k <= kBadWords; ++k) ctl->bad[i][k] = 0;
    ctl->abort = 0;
  }
  if (threadIdx.x < 32) fence_mbar_init();
  if (threadIdx.x == 0) prefetch_tmap(&qmap);
  if (threadIdx.x == 32) prefetch_tmap(&kmap);
  if (threadIdx.x == 64) prefetch_tmap(&vmap);
  pdl_wait();
  pdl_trigger();
  draft_plan(a, kTile, kE, blockIdx.x, gridDim.x, &ctl->plan, kThreads);
  DraftWalk w;
  w.init(a, ctl->plan, kTile, kE, p.whole);

  if (warp == kConsumers + kProducers) {
    // ---- query rows and mask words, item by item ----------------------------------
    uint32_t segs = 0;
    while (w.next(a, kTile, kE)) {
      const DraftItem& it = w.it;
      const int slot = segs % C::kQSlots;
      if (!mbar_wait_warp(&ctl->q_empty[slot], ((segs / C::kQSlots) & 1) ^ 1, &ctl->abort, a.status)) break;
      const int64_t token = (int64_t)w.seq.first + it.i0;
      if (a.bits)
        for (int e = lane; e < it.ni * a.words; e += 32)
          masks[slot * C::kRows * kWords + e / a.words * kWords + e % a.words] = (uint64_t)a.bits[token * a.words + e];
      __syncwarp();
      if (lane == 0) {
        constexpr int kCols = D < 64 ? D : 64;
        mbar_arrive_expect_tx(&ctl->q_full[slot], a.tokens * a.heads * C::kRow);
        for (int h = 0; h < D / kCols; ++h)
          tma_load_3d(qbuf + slot * C::kQBytes + h * C::kRows * 128, &qmap, &ctl->q_full[slot], h * kCols,
                      it.kvh * a.G + it.h0, (int)token);
      }
      ++segs;
    }
    // no copy may land after the CTA is gone: not where a wait was given up, here or by another warp
    if (lane == 0)
      for (uint32_t i = segs > C::kQSlots ? segs - C::kQSlots : 0; i < segs; ++i)
        mbar_wait(&ctl->q_full[i % C::kQSlots], (i / C::kQSlots) & 1, nullptr, a.status);
    return;
  }
  if (warp >= kConsumers) {
    // ---- producers: tiles warp - kConsumers, + kProducers, ...; as paged_attn_tma.cu -----
    const uint32_t me = warp - kConsumers;
    const uint32_t rows = kTile / p.box;              // boxes down a tile
    const uint32_t rb = lane % rows, side = lane / rows;
    const bool has_box = side < 2;
    const CUtensorMap* map = side ? &vmap : &kmap;
    const uint32_t dst = side * C::kSide + rb * p.box * C::kRow;
    const int32_t* trow = nullptr;
    uint32_t pages = 0;                               // of the sequence
    const uint32_t ps = a.page_size, step_pg = kProducers * kTile / ps, step_row = kProducers * kTile % ps;
    // the table is read 32 entries at a time, and one such window ahead
    uint32_t win = 0;                                 // its first page index
    int cur = -1, nxt = -1, wb = -1;                  // entries win + lane, win + 32 + lane; sequence
    auto entry = [&](uint32_t i) { return i < pages ? trow[i] : -1; };
    uint32_t seg_it = 0, last = 0;                    // the segment's first tile in the CTA's order
    bool ok = true;
    while (ok && w.next(a, kTile, kE)) {
      int64_t t = w.t0 + ((me - seg_it) & (kProducers - 1));
      if (t < w.t1) {
        const int kvh = w.it.kvh;
        trow = a.table + (int64_t)w.seg_b * a.max_pages;
        pages = ((uint32_t)w.seq.len + ps - 1) / ps;
        const uint32_t key0 = (uint32_t)t * kTile, pg0 = key0 / ps;
        uint32_t row = key0 - pg0 * ps + rb * p.box, pg = pg0;      // of this lane's box
        while (row >= ps) {
          row -= ps;
          ++pg;
        }
        uint32_t first = pg0, first_row = key0 - pg0 * ps;          // of the tile's first key
        if (wb != w.seg_b || win != pg0) {
          wb = w.seg_b;
          win = pg0;
          cur = entry(win + lane);
          nxt = entry(win + 32 + lane);
        }
        for (; t < w.t1; t += kProducers) {
          if (first - win >= 32) {
            win += 32;
            cur = nxt;
            nxt = entry(win + 32 + lane);
          }
          const uint32_t at = pg - win;
          const int id0 = __shfl_sync(0xffffffffu, cur, at & 31), id1 = __shfl_sync(0xffffffffu, nxt, at & 31);
          const int page = at < 32 ? id0 : id1;
          const bool now = has_box && t * kTile + rb * p.box < w.seq.len;
          int z = page * a.Hkv + kvh;
          if (now && (uint32_t)page >= (uint32_t)a.n_pages) {
            flag_device(a.status, kDevCheck);
            z = a.n_pages * a.Hkv;                    // outside the map: reads as zeros
          }
          const uint32_t it = seg_it + (uint32_t)(t - w.t0);
          const int st = it % S;
          ok = mbar_wait_warp(&ctl->empty[st], ((it / S) & 1) ^ 1, &ctl->abort, a.status);
          if (!ok) break;
          const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, now));
          if (lane == 0) mbar_arrive_expect_tx(&ctl->full[st], boxes * p.box * C::kRow);
          __syncwarp();
          if (now) tma_load_4d(stages + st * C::kStage + dst, map, &ctl->full[st], 0, (int)row, 0, z);
          last = it + 1;
          pg += step_pg;
          row += step_row;
          if (row >= ps) {
            row -= ps;
            ++pg;
          }
          first += step_pg;
          first_row += step_row;
          if (first_row >= ps) {
            first_row -= ps;
            ++first;
          }
        }
      }
      seg_it += (uint32_t)(w.t1 - w.t0);
    }
    if (lane == 0)                                    // as for the query rows
      for (uint32_t i = 0; i < (uint32_t)S && i < last; ++i)
        if (((last - 1 - i) & (kProducers - 1)) == me)
          mbar_wait(&ctl->full[(last - 1 - i) % S], ((last - 1 - i) / S) & 1, nullptr, a.status);
    return;
  }

  // ---- consumers -------------------------------------------------------------
  const int rg = warp % RG, unit = warp / RG;
  const int grp = C::kGroups > 1 ? unit / C::kSlices : 0, slice0 = C::kGroups > 1 ? unit % C::kSlices : unit;
  Part<D, RG> me(p.box);
  // a row's token: floor(row / heads), exact for rows of up to 64 (an item of part of a key head's query heads has one)
  const uint32_t by_heads = (65535 + a.heads) / a.heads;
  auto token_of = [&](int row) { return a.hgroups > 1 ? 0 : (int)(row * by_heads >> 16); };
  int4 open = make_int4(-1, 0, 0, 0);
  uint32_t it = 0, segs = 0;
  bool ok = true;
  while (ok && w.next(a, kTile, kE)) {
    const DraftItem& item = w.it;
    const int rows = item.ni * item.nh, slot = segs % C::kQSlots;
    const int ctx = w.seq.len - w.seq.n, new16 = ctx & ~15;
    unsigned int* bad = ctl->bad[segs & 1];
    const unsigned long long* words = masks + slot * C::kRows * kWords;
    ok = mbar_wait_warp(&ctl->q_full[slot], (segs / C::kQSlots) & 1, &ctl->abort, a.status);
    if (!ok) break;
    const bool live = rg * 16 < rows;
    if (live) me.load_q(smem_u32(qbuf + slot * C::kQBytes), rg * 16);
    const int r0 = rg * 16 + me.g, i0 = token_of(r0), i1 = token_of(r0 + 8);
    bool active = false;
    for (int64_t t = w.t0; t < w.t1; ++t, ++it) {
      if (C::kGroups > 1 && it % C::kGroups != (uint32_t)grp) continue;
      const int st = it % S;
      ok = mbar_wait_warp(&ctl->full[st], (it / S) & 1, &ctl->abort, a.status);
      if (!ok) break;
      uint8_t* stage = stages + st * C::kStage;
      bool wrote = false;
      if (live) {
#pragma unroll 1
        for (int n = 0; n < C::kTurns; ++n) {
          const int slice = slice0 + n * C::kUnits, x = (int)t * kTile + slice * 16, left = w.seq.len - x;
          if (left <= 0) break;
          active = true;
          const bool all = x + 16 <= ctx;
          uint32_t see[2] = {0, 0};
          if (!all) {
            wrote = true;
            const uint32_t found = me.clean(stage, slice, left);
            if (found && lane == 0) {
              const int k = x - new16;
              atomicOr(&bad[k >> 5], found << (k & 31));
              bad[kBadWords] = 1;
            }
            if (r0 < rows) see[0] = sees16(a, w.seq, item.i0 + i0, words + i0 * kWords, x);
            if (r0 + 8 < rows) see[1] = sees16(a, w.seq, item.i0 + i1, words + i1 * kWords, x);
            __syncwarp();
          }
          me.tile(smem_u32(stage), slice, all, see, p.scale_log2);
        }
      }
      if (wrote) fence_async_shared();                // before the next copy into this stage
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->empty[st]);
    }
    if (!ok) break;
    // ---- merge: the units' results of every row ----------------------------------
    if (live)
      me.result(ctl->m[warp], ctl->l[warp], red + (unit * C::kRows + rg * 16) * C::kRedStride, active);
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->red_full);
    ok = mbar_wait_warp(&ctl->red_full, segs * 2 & 1, &ctl->abort, a.status);
    if (!ok) break;
    const bool whole = w.begins && w.ends, odd = bad[kBadWords] != 0;
    const int64_t pslot = (2 * (int64_t)blockIdx.x + (w.begins ? 1 : 0)) * C::kRows;
    const int c = threadIdx.x % (D / 4) * 4;          // the thread's columns
    for (int row = threadIdx.x / (D / 4); row < rows; row += kConsumers * 128 / D) {
      const int i = token_of(row);
      const float* rm = &ctl->m[row >> 4][row & 15];  // of unit u: RG warps on
      const float* rl = &ctl->l[row >> 4][row & 15];
      float f[C::kUnits], lu[C::kUnits], mm = -INFINITY;
      float4 v[C::kUnits];
#pragma unroll
      for (int u = 0; u < C::kUnits; ++u) {
        f[u] = rm[u * RG * 16];
        lu[u] = rl[u * RG * 16];
        v[u] = *reinterpret_cast<const float4*>(red + (u * C::kRows + row) * C::kRedStride + c);
        mm = fmaxf(mm, f[u]);
      }
      const float base = mm == -INFINITY ? 0.f : mm;
      float ll = 0.f;
      float4 oo = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < C::kUnits; ++u)
        if (lu[u] != -1.f) {                          // (its outputs are not there otherwise)
          const float fu = ex2_approx(f[u] - base);
          ll += fu * lu[u];
          oo.x += fu * v[u].x;
          oo.y += fu * v[u].y;
          oo.z += fu * v[u].z;
          oo.w += fu * v[u].w;
        }
      const unsigned long long* mine = words + i * kWords;
      if (odd) {
        for (int k = 0; k < kBadWords * 2; ++k) {     // 16 keys at a time
          const int x0 = new16 + k * 16;
          uint32_t todo = bad[k >> 1] >> (k & 1) * 16 & 0xffffu;
          if (todo) todo &= sees16(a, w.seq, item.i0 + i, mine, x0);
          for (; todo; todo &= todo - 1) {
            const int x = x0 + __ffs(todo) - 1, pg = x / a.page_size;
            const int id = a.table[(int64_t)w.seg_b * a.max_pages + pg];
            if ((unsigned)id >= (unsigned)a.n_pages) continue;
            const uint2 q = *reinterpret_cast<const uint2*>(
                p.v + ((((int64_t)id * a.Hkv + item.kvh) * a.page_size + (x - pg * a.page_size)) * D + c) * 2);
            oo.x += if_bad(bf16lo(q.x));
            oo.y += if_bad(bf16hi(q.x));
            oo.z += if_bad(bf16lo(q.y));
            oo.w += if_bad(bf16hi(q.y));
          }
        }
      }
      if (whole) {
        bool any = ctx > 0 || !a.bits;
        for (int x = 0; !any && x < w.seq.n; x += 16) any = sees16(a, w.seq, item.i0 + i, mine, x) != 0;
        const float inv = 1.f / ll;
        const int64_t tt = (int64_t)w.seq.first + item.i0 + i;
        const int h = item.kvh * a.G + item.h0 + row - i * item.nh;
        *reinterpret_cast<uint2*>(p.o + (tt * a.H + h) * D + c) =
            any ? make_uint2(pack_bf16x2(oo.x * inv, oo.y * inv), pack_bf16x2(oo.z * inv, oo.w * inv))
                : make_uint2(0u, 0u);
        if (p.lse && c == 0) p.lse[(int64_t)h * a.T + tt] = row_lse(mm, ll, any);
      } else {
        *reinterpret_cast<float4*>(part.o + (pslot + row) * D + c) = oo;
        if (c == 0) *reinterpret_cast<float2*>(part.ml + (pslot + row) * 2) = make_float2(mm, ll);
      }
    }
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&ctl->q_empty[slot]);
      mbar_arrive(&ctl->red_full);                    // the results may be written over
    }
    ok = mbar_wait_warp(&ctl->red_full, segs * 2 + 1 & 1, &ctl->abort, a.status);
    if (!ok) break;
    if (threadIdx.x == 0)                             // everybody has read it; the segment after the next writes it
      for (int k = 0; k <= kBadWords; ++k) bad[k] = 0;
    if (w.begins && !w.ends)
      open = make_int4(w.seg_b, w.seg_item, w.seg_items, w.parts(ctl->plan, kE, blockIdx.x, gridDim.x));
    ++segs;
  }
  if (threadIdx.x == 0) part.open[blockIdx.x] = open;
}

template <int D, int RG>
cudaError_t run(const DraftProblem& p, unsigned int* status, cudaStream_t s) {
  using C = Cfg<D, RG>;
  SliceArgs r = {};
  r.a = draft_batch(p, C::kRows, 1, status);
  r.v = static_cast<const uint8_t*>(p.pool.v);
  r.o = static_cast<bf16*>(p.o);
  r.lse = p.lse;
  r.workspace = p.workspace;
  r.whole = false;
  r.box = C::kTile < 64 ? C::kTile : 64;
  while (p.pool.page_size % r.box) r.box >>= 1;
  r.scale_log2 = p.scale * 1.4426950408889634f;
  CUtensorMap maps[3];
  // a page's rows as 128-byte parts (64 for rows of 32), so that one swizzled box holds them all
  constexpr uint32_t kCols = D < 64 ? D : 64;
  const uint64_t rows = (uint64_t)p.pool.page_size;
  const uint64_t dims[4] = {kCols, rows, D / kCols, (uint64_t)p.pool.n_pages * p.pool.H};
  const uint64_t strides[3] = {C::kRow, kCols * 2, C::kRow * rows};
  const uint32_t box[4] = {kCols, (uint32_t)r.box, D / kCols, 1};
  constexpr CUtensorMapSwizzle kSwizzle = D < 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  const uint64_t q_dims[3] = {(uint64_t)D, (uint64_t)p.H, (uint64_t)p.T};
  const uint64_t q_strides[2] = {C::kRow, (uint64_t)p.q_stride * 2};
  const uint32_t q_box[3] = {kCols, (uint32_t)r.a.heads, (uint32_t)r.a.tokens};
  if (!make_tmap(&maps[2], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kSwizzle, p.q, 3, q_dims, q_strides, q_box))
    return cudaErrorInvalidValue;
  for (int i = 0; i < 2; ++i)
    if (!make_tmap(&maps[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kSwizzle, i ? p.pool.v : p.pool.k, 4, dims, strides, box))
      return cudaErrorInvalidValue;
  const int ctas = min(sm_count(), kPagedMaxCtas);
  cudaError_t e = allow_smem_once<draft_slices_kernel<D, RG>>(C::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(draft_slices_kernel<D, RG>, dim3(ctas), dim3(kThreads), C::kSmem, s, maps[2], maps[0], maps[1], r);
  if (e != cudaSuccess || r.whole) return e;
  return launch_draft_join(NT_BF16, r.a, D, ctas, C::kRows, p.workspace, p.o, p.lse, s);
}

template <int D>
cudaError_t run_d(const DraftProblem& p, unsigned int* status, cudaStream_t s) {
  const int64_t rows = (int64_t)p.max_new * (p.H / p.pool.H);
  if (rows <= 16) return run<D, 1>(p, status, s);
  return rows <= 32 ? run<D, 2>(p, status, s) : run<D, 4>(p, status, s);
}

}  // namespace

bool draft_slices_supported(nt_dtype dt, const DraftProblem& p) {
  return dt == NT_BF16 && p.pool.page_size % 8 == 0 && p.pool.n_pages > 0;
}

cudaError_t launch_draft_slices(const DraftProblem& p, unsigned int* status, cudaStream_t s) {
  if (p.d == 32) return run_d<32>(p, status, s);
  return p.d == 64 ? run_d<64>(p, status, s) : run_d<128>(p, status, s);
}

}  // namespace nt
