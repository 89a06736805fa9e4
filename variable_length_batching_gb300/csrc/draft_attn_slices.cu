// Attention of drafted tokens over a paged cache, few rows to a key head (up to
// 64 of tokens times query heads): bf16 at d = 32 and 64, pages of a multiple of 8
// positions.
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
// and two hand-offs between warps for every 128 keys: it costs more where rows
// are few (152 contexts of 8,000 keys in a graph, d = 64, 16 rows: 69 us there, 57
// here; 32 rows 69 and 81), but has no d = 32 (16 rows 44 us here and 90 on the general
// kernel, 32 rows 65 and 104, 64 rows 107 and 108), and at d = 128 it was the faster
// one (64 contexts of up to 8,192 keys, up to 16 rows: 95 us against 122).  At d = 32
// a slice's bytes are half of those at d = 64 and its softmax is the same: some 265
// warp instructions to a slice, two consumer warps to a scheduler, which issues in 42%
// of its cycles and waits for one instruction after the other in the rest; HBM is 44%
// busy.
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

template <int D, int RG>
struct Cfg {
  static constexpr int kRows = 16 * RG;
  static constexpr int kUnits = kConsumers / RG;              // warps of one row group
  static constexpr int kTile = D == 32 ? 128 : 64;            // keys of a stage, 16 KB
  static constexpr int kSlices = kTile / 16;
  static constexpr int kGroups = kUnits > kSlices ? kUnits / kSlices : 1;          // stages worked on at once
  static constexpr int kTurns = kUnits > kSlices ? 1 : kSlices / kUnits;           // slices of a stage to a warp
  static constexpr uint32_t kRow = D * 2;
  static constexpr uint32_t kSide = kTile * kRow, kStage = 2 * kSide;
  static constexpr int kRedStride = Slice<D, 0>::kRedStride;
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
  DraftPlanSums plan;
  int abort;
};
static_assert(sizeof(Ctl) <= 4096, "control block");

struct SliceArgs {
  DraftBatch a;
  const uint8_t* v;
  bf16* o;
  float* lse;
  void* workspace;
  int box;                        // keys per box
  float scale_log2;
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
  __syncthreads();
  const DraftPlan plan = draft_plan(a, kTile, kE, blockIdx.x, gridDim.x, &ctl->plan, kThreads);
  DraftWalk w;
  w.init(a, plan, kTile, kE);

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
  Slice<D, C::kSide> me(p.box);
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
    if (live) me.load_q(smem_u32(qbuf + slot * C::kQBytes), rg * 16, C::kRows * 128);
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
      open = make_int4(w.seg_b, w.seg_item, w.seg_items, w.parts(plan, blockIdx.x));
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
  if (e != cudaSuccess) return e;
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
  return dt == NT_BF16 && p.d <= 64 && p.pool.page_size % 8 == 0 && p.pool.n_pages > 0;
}

cudaError_t launch_draft_slices(const DraftProblem& p, unsigned int* status, cudaStream_t s) {
  return p.d == 32 ? run_d<32>(p, status, s) : run_d<64>(p, status, s);
}

}  // namespace nt
