// Attention of one new token per sequence over a paged key/value cache whose
// pages hold a multiple of 8 positions.
//
// The floor is the cache's bytes: 2 len H_kv d elements read once, for G
// multiply-adds per element (G query heads to a key head), so the kernel is
// a stream of TMA loads and everything else has to hide behind it.  One CTA
// per SM holds 128 to 160 KB of key/value tiles in flight (what a latency of
// about 1 us at the SM's share of the bandwidth needs, three times over).
// Four contexts of 120,000 keys with 8 key heads of 128 take 279 us in bf16
// (104% of the measured copy rate), 64 of 16 to 8,192 keys 57 us (82%), in
// fp32 106 (87%).
//
// Two producer warps walk the CTA's share of the batch (paged_plan.cuh) tile
// by tile, alternating: one box of R = gcd(page_size, 64, tile) keys per lane
// into a ring of stages.  (A copy takes its warp about 85 cycles to issue, so
// one warp alone could not keep up with HBM for 64 keys of d = 64 in pages of
// 16: eight boxes in 700 cycles.)  A third warp copies the items' query rows.
// Eight consumer warps take 16 keys of a tile each, every warp with its own
// running maximum, sum and output.
//
// bf16 (boxes in the 128-byte swizzle; 64-byte for d = 32): a warp's part is
//   S = Q K^T      (heads x 16 keys; rows beyond the item's heads are zero)
//   P = exp2(S - max), as the sum of two bf16 (two products; HBM hides the
//                  second: the ragged batch takes 56.9 us, 56.5 with one bf16,
//                  which is off by 2^-8 of P)
//   O^T += V^T P^T (d x heads): S's accumulator layout is the B operand's, so
//                  P goes from registers to the product, and V^T comes from
//                  the tile by transposed matrix loads.
// These are mma.sync products of 16 rows: a decode item has at most 16 query
// rows where a tcgen05 tile has 64 at least, and its accumulators' round trip
// through TMEM would be longer than the whole product.  The products and
// matrix loads of a 32 KB stage take about a tenth of the time HBM takes to
// deliver it.
//
// fp32: packed multiply-adds, a key's columns in two lanes for the scores,
// four columns of the output in each lane (paged_worker.cuh).
//
// At the end of a segment the eight warps leave their results in shared
// memory for a fourth kind of warp, which merges them and writes the output
// or a partial result for the join, while the eight go on: with short
// sequences the merge is as long as the segment's tiles.
#include "paged_plan.cuh"
#include "paged_worker.cuh"

namespace nt {
namespace {

using namespace paged;

constexpr int kConsumers = 8;               // warps
constexpr int kProducers = 2;               // warps, tiles alternating
constexpr int kQSlots = 4;                  // items whose query rows are in flight or in use
constexpr int kOthers = kConsumers + kProducers + 1;       // warps beside the merge's

// HP: query heads of an item, at most, and what the registers are laid out
// for: 8 or 16 in bf16 (one or two accumulator tiles), 1, 2, 4 or 8 in fp32.
// MW: warps that merge, 0 for the eight together.
template <typename T, int D, int HP, int MW>
struct Cfg {
  static constexpr bool kBf16 = sizeof(T) == 2;
  // keys per stage, and per unit of the split: 16 KB of bf16 (32 at d = 128), 32 of fp32
  static constexpr int kTile = kBf16 ? (D == 32 ? 128 : 64) : 4096 / D;
  static constexpr int kSlices = kTile / 16;                  // warps that share a stage
  static constexpr int kGroups = kConsumers / kSlices;        // stages worked on at once
  static constexpr uint32_t kRow = D * sizeof(T);             // bytes of a key's row
  static constexpr uint32_t kSide = kTile * kRow;             // K or V of a stage
  static constexpr uint32_t kStage = 2 * kSide;
  static constexpr int kRedStride = D + 4;                    // floats: keeps the merge's writes conflict-free
  static constexpr uint32_t kRed = kConsumers * HP * kRedStride * 4;
  static constexpr int kRedBufs = HP * D <= 1024 ? 2 : 1;     // segments whose results wait for the merge
  static constexpr int kThreads = (kOthers + (MW ? MW : 1)) * 32;
  static constexpr uint32_t kQBytes = HP * kRow;
  static constexpr int kExtra = HP == 16 ? 3 : 2;             // an item's cost beside its tiles, in tiles
  static constexpr uint32_t kScratch = kConsumers * Worker<T, D, HP>::kScratch;
  static constexpr uint32_t kFixed = kRedBufs * kRed + kQSlots * kQBytes + kScratch + 4096 /* statistics, barriers, plan */;
  // A multiple of the groups and of the producers: a stage is then always the
  // same warps' and they see every phase of its barriers.  (Otherwise a warp
  // would wait on a phase whose predecessor it never waited for, which parity
  // cannot tell apart from the phase before that.)
  static constexpr int kRound = kGroups > kProducers ? kGroups : kProducers;
  static constexpr int kFit = (int)((226 * 1024 - 1024 - kFixed) / kStage);
  static constexpr int kStages = (kFit < 16 ? kFit : 16) / kRound * kRound;
  static constexpr uint32_t kSmem = 1024 + kStages * kStage + kFixed;
  static_assert(kStages >= 4 && kStages % kGroups == 0 && kStages % kProducers == 0 && kSmem <= 227 * 1024,
                "shared memory");
};

struct Ctl {
  uint64_t full[16], empty[16], q_full[kQSlots], q_empty[kQSlots], red_full[2], red_empty[2];
  float m[2][kConsumers][16], l[2][kConsumers][16];
  PagedPlan plan;
  int abort;
};
static_assert(sizeof(Ctl) <= 4096, "control block");

struct TmaArgs {
  const void* q;
  int64_t q_stride;
  const int32_t* table;
  const int32_t* lengths;
  void* o;
  float* lse;
  void* workspace;
  int B, H, G, Hkv, max_pages, page_size, n_pages;
  int items, hgroups, heads;      // head items per sequence; item slots of the partials
  bool whole;                     // items are not split
  int box;                        // keys per box: gcd(page_size, 64)
  float scale_log2;
  unsigned int* status;
};

// The merge of a segment's eight warps, and its output or partial result: the
// caller is thread `first` of `step`.
template <typename T, int D, int HP, int MW>
__device__ __forceinline__ void merge_segment(const TmaArgs& a, const PagedWalk& w, const Ctl* ctl, const float* red,
                                              int buf, int first, int step) {
  using C = Cfg<T, D, HP, MW>;
  constexpr int kHeads = HP;
  const PagedPartials part = paged_partials(a.workspace, gridDim.x, a.heads);
  const int kvh = w.seg_item / a.hgroups, h0 = (w.seg_item % a.hgroups) * kHeads;
  const int nh = min(kHeads, a.G - h0);
  const bool whole = w.begins && w.ends;
  const int64_t pslot = 2 * (int64_t)blockIdx.x + (w.begins ? 1 : 0);
  const int64_t hq = (int64_t)kvh * a.G + h0;
  const float(*sm)[16] = ctl->m[buf];
  const float(*sl)[16] = ctl->l[buf];
  // a lane's four columns of a head; two passes at a time, to overlap their reads
#pragma unroll 2
  for (int e = first; e < nh * (D / 4); e += step) {
    const int h = e / (D / 4), c = e % (D / 4) * 4;
    float f[kConsumers], mm = -INFINITY;
    float4 v[kConsumers];
#pragma unroll
    for (int x = 0; x < kConsumers; ++x) {
      f[x] = sm[x][h];
      mm = fmaxf(mm, f[x]);
      v[x] = sl[x][h] == -1.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                              : *reinterpret_cast<const float4*>(red + buf * (C::kRed / 4) +
                                                                 (x * kHeads + h) * C::kRedStride + c);
    }
    const float base = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f;
    float4 oo = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int x = 0; x < kConsumers; ++x) {
      const float lx = sl[x][h];
      const float fx = lx == -1.f ? 0.f : ex2_approx(f[x] - base);
      ll += fx * lx;
      oo.x += fx * v[x].x;
      oo.y += fx * v[x].y;
      oo.z += fx * v[x].z;
      oo.w += fx * v[x].w;
    }
    if (whole) {
      const float inv = 1.f / ll;
      T* out = static_cast<T*>(a.o) + ((int64_t)w.seg_b * a.H + hq + h) * D + c;
      if constexpr (C::kBf16)
        *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(oo.x * inv, oo.y * inv),
                                                    pack_bf16x2(oo.z * inv, oo.w * inv));
      else
        *reinterpret_cast<float4*>(out) = make_float4(oo.x * inv, oo.y * inv, oo.z * inv, oo.w * inv);
      if (a.lse && c == 0) a.lse[(hq + h) * a.B + w.seg_b] = (mm + log2f(ll)) * 0.6931471805599453f;
    } else {
      *reinterpret_cast<float4*>(part.o + (pslot * a.heads + h) * D + c) = oo;
      if (c == 0) {
        part.ml[(pslot * a.heads + h) * 2] = mm;
        part.ml[(pslot * a.heads + h) * 2 + 1] = ll;
      }
    }
  }
}

template <typename T, int D, int HP, int MW>
__global__ void __launch_bounds__((Cfg<T, D, HP, MW>::kThreads), 1)
paged_attn_tma_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const TmaArgs a) {
  using C = Cfg<T, D, HP, MW>;
  constexpr int kHeads = HP, S = C::kStages, kTile = C::kTile;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  uint8_t* stages = smem;
  float* red = reinterpret_cast<float*>(smem + S * C::kStage);
  uint8_t* qbuf = reinterpret_cast<uint8_t*>(red) + C::kRedBufs * C::kRed;
  uint8_t* scratch = qbuf + kQSlots * C::kQBytes;
  Ctl* ctl = reinterpret_cast<Ctl*>(scratch + C::kScratch);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t cap = min64((int64_t)a.max_pages * a.page_size, 0x7fffffff);
  const PagedPartials part = paged_partials(a.workspace, gridDim.x, a.heads);

  // a lane to each barrier
  if (threadIdx.x < S) {
    mbar_init(&ctl->full[threadIdx.x], 1);
    mbar_init(&ctl->empty[threadIdx.x], C::kSlices);
  }
  if (threadIdx.x < kQSlots) {
    mbar_init(&ctl->q_full[threadIdx.x], 1);
    mbar_init(&ctl->q_empty[threadIdx.x], kConsumers);
  }
  if (threadIdx.x < C::kRedBufs) {
    mbar_init(&ctl->red_full[threadIdx.x], kConsumers);
    mbar_init(&ctl->red_empty[threadIdx.x], MW ? MW : kConsumers);
  }
  if (threadIdx.x == 0) ctl->abort = 0;
  if (threadIdx.x < 32) fence_mbar_init();
  if (threadIdx.x == 32) prefetch_tmap(&kmap);
  if (threadIdx.x == 64) prefetch_tmap(&vmap);
  pdl_wait();
  pdl_trigger();
  paged_plan(a.lengths, a.B, cap, a.items, kTile, C::kExtra, blockIdx.x, gridDim.x, &ctl->plan, a.status, C::kThreads);
  PagedWalk w;
  w.init(ctl->plan, a.lengths, a.B, cap, kTile, C::kExtra, a.whole);

  if (warp == kOthers - 1) {
    // ---- query rows, item by item ------------------------------------------
    uint32_t segs = 0;
    while (w.next(a.lengths, a.B, cap, a.items, kTile, C::kExtra)) {
      const int slot = segs % kQSlots;
      if (!mbar_wait_warp(&ctl->q_empty[slot], ((segs / kQSlots) & 1) ^ 1, &ctl->abort, a.status)) break;
      const int kvh = w.seg_item / a.hgroups, h0 = (w.seg_item % a.hgroups) * kHeads;
      const uint32_t bytes = min(kHeads, a.G - h0) * C::kRow;
      if (lane == 0) {
        mbar_arrive_expect_tx(&ctl->q_full[slot], bytes);
        bulk_load(qbuf + slot * C::kQBytes,
                  static_cast<const T*>(a.q) + w.seg_b * a.q_stride + (int64_t)(kvh * a.G + h0) * D, bytes,
                  &ctl->q_full[slot]);
      }
      ++segs;
    }
    // no copy may land after the CTA is gone: not where a wait was given up, here or by another warp
    if (lane == 0)
      for (uint32_t i = segs > kQSlots ? segs - kQSlots : 0; i < segs; ++i)
        mbar_wait(&ctl->q_full[i % kQSlots], (i / kQSlots) & 1, nullptr, a.status);
    return;
  }
  if (warp >= kOthers) {
    // ---- merge: the consumers' results of a segment ------------------------------
    uint32_t segs = 0;
    int64_t open_id = -1, open_parts = 0;             // the item left unfinished
    while (w.next(a.lengths, a.B, cap, a.items, kTile, C::kExtra)) {
      if (MW > 0) {
        const int buf = segs % C::kRedBufs;
        if (!mbar_wait_warp(&ctl->red_full[buf], (segs / C::kRedBufs) & 1, &ctl->abort, a.status)) break;
        merge_segment<T, D, HP, MW>(a, w, ctl, red, buf, threadIdx.x - kOthers * 32, MW * 32);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->red_empty[buf]);
        ++segs;
      }
      if (w.begins && !w.ends) {
        open_id = (int64_t)w.seg_b * a.items + w.seg_item;
        open_parts = w.parts(ctl->plan, C::kExtra, blockIdx.x, gridDim.x);
      }
    }
    if (threadIdx.x == kOthers * 32) {
      part.id[2 * blockIdx.x] = open_id;
      part.id[2 * blockIdx.x + 1] = open_parts;
    }
    return;
  }
  if (warp >= kConsumers) {
    // ---- producers: tiles warp - kConsumers, + kProducers, ... ----------------
    const uint32_t me = warp - kConsumers;
    const uint32_t rows = kTile / a.box;              // boxes down a tile
    const uint32_t rb = lane % rows, side = lane / rows;
    const bool has_box = side < 2;
    const CUtensorMap* map = side ? &vmap : &kmap;
    const uint32_t dst = side * C::kSide + rb * a.box * C::kRow;
    const int32_t* trow = nullptr;
    uint32_t pages = 0;                               // of the sequence
    const uint32_t ps = a.page_size, step_pg = kProducers * kTile / ps, step_row = kProducers * kTile % ps;
    // The block table is read 32 entries at a time, a lane each, and one such
    // window ahead, so that a lookup is a shuffle.  The window stays when the
    // next segment starts on the same pages: the sequence's next head.
    uint32_t win = 0;                                 // its first page index
    int cur = -1, nxt = -1, wb = -1;                  // entries win + lane, win + 32 + lane; sequence
    auto entry = [&](uint32_t i) { return i < pages ? trow[i] : -1; };
    uint32_t seg_it = 0, last = 0;                    // the segment's first tile in the CTA's order
    bool ok = true;
    while (ok && w.next(a.lengths, a.B, cap, a.items, kTile, C::kExtra)) {
      int64_t t = w.t0 + ((me - seg_it) & (kProducers - 1));
      if (t < w.t1) {
        const int kvh = w.seg_item / a.hgroups;
        trow = a.table + (int64_t)w.seg_b * a.max_pages;
        pages = ((uint32_t)w.seg_len + ps - 1) / ps;
        const uint32_t key0 = (uint32_t)t * kTile, pg0 = key0 / ps;
        uint32_t row = key0 - pg0 * ps + rb * a.box, pg = pg0;      // of this lane's box
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
          const bool now = has_box && t * kTile + rb * a.box < w.seg_len;
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
          if (lane == 0) mbar_arrive_expect_tx(&ctl->full[st], boxes * a.box * C::kRow);
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
  // sequences with no key: zeros
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    if (paged_length(a.lengths, b, cap, nullptr) != 0) continue;
    for (int e = threadIdx.x; e < a.H * D; e += kConsumers * 32)
      static_cast<T*>(a.o)[(int64_t)b * a.H * D + e] = from_f32<T>(0.f);
    if (a.lse)
      for (int h = threadIdx.x; h < a.H; h += kConsumers * 32) a.lse[(int64_t)h * a.B + b] = -INFINITY;
  }
  const int grp = warp / C::kSlices, slice = warp % C::kSlices;
  using W = Worker<T, D, HP>;
  W me(a.box, slice, scratch + warp * W::kScratch);
  uint32_t it = 0, segs = 0;
  bool ok = true;
  while (ok && w.next(a.lengths, a.B, cap, a.items, kTile, C::kExtra)) {
    const int nh = min(kHeads, a.G - (w.seg_item % a.hgroups) * kHeads);
    const int slot = segs % kQSlots, buf = segs % C::kRedBufs;
    ok = mbar_wait_warp(&ctl->q_full[slot], (segs / kQSlots) & 1, &ctl->abort, a.status);
    if (!ok) break;
    me.load_q(qbuf + slot * C::kQBytes, nh);
    __syncwarp();
    if (!W::kKeepsQ && lane == 0) mbar_arrive(&ctl->q_empty[slot]);
    bool active = false;
    for (int64_t t = w.t0; t < w.t1; ++t, ++it) {
      if (it % C::kGroups != (uint32_t)grp) continue;
      const int st = it % S;
      ok = mbar_wait_warp(&ctl->full[st], (it / S) & 1, &ctl->abort, a.status);
      if (!ok) break;
      const int left = (int)min64(w.seg_len - t * kTile - slice * 16, 16);     // keys of this slice
      if (left > 0) {
        active = true;
        me.tile(stages + st * C::kStage, C::kSide, left, a.scale_log2);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->empty[st]);
    }
    if (!ok) break;
    if (W::kKeepsQ && lane == 0) mbar_arrive(&ctl->q_empty[slot]);
    ok = mbar_wait_warp(&ctl->red_empty[buf], ((segs / C::kRedBufs) & 1) ^ 1, &ctl->abort, a.status);
    if (!ok) break;
    me.result(ctl->m[buf][warp], ctl->l[buf][warp], red + buf * (C::kRed / 4) + warp * kHeads * C::kRedStride, nh,
              active);
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->red_full[buf]);
    if (MW == 0) {
      ok = mbar_wait_warp(&ctl->red_full[buf], (segs / C::kRedBufs) & 1, &ctl->abort, a.status);
      if (!ok) break;
      merge_segment<T, D, HP, MW>(a, w, ctl, red, buf, threadIdx.x, kConsumers * 32);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->red_empty[buf]);
    }
    ++segs;
  }
}

template <typename T, int D, int HP, int MW>
cudaError_t run(const PagedAttnProblem& p, unsigned int* status, cudaStream_t s) {
  using C = Cfg<T, D, HP, MW>;
  TmaArgs a;
  a.q = p.q;
  a.q_stride = p.q_stride;
  a.table = p.table;
  a.lengths = p.lengths;
  a.o = p.o;
  a.lse = p.lse;
  a.workspace = p.workspace;
  a.B = p.B;
  a.H = p.H;
  a.G = p.H / p.pool.H;
  a.Hkv = p.pool.H;
  a.max_pages = p.max_pages;
  a.page_size = p.pool.page_size;
  a.n_pages = p.pool.n_pages;
  a.hgroups = (a.G + HP - 1) / HP;
  a.items = a.Hkv * a.hgroups;
  a.heads = min(HP, a.G);
  a.whole = paged_whole_items(p, sizeof(T));
  a.box = min(64, C::kTile);
  while (a.page_size % a.box) a.box >>= 1;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  a.status = status;
  CUtensorMap maps[2];
  // a page's rows as 128-byte parts (64 for bf16 rows of 32), so that one swizzled box holds them all
  constexpr uint32_t kCols = C::kRow < 128 ? D : 128 / sizeof(T);
  const uint64_t rows = (uint64_t)a.page_size;
  const uint64_t dims[4] = {kCols, rows, D / kCols, (uint64_t)a.n_pages * a.Hkv};
  const uint64_t strides[3] = {C::kRow, kCols * sizeof(T), C::kRow * rows};
  const uint32_t box[4] = {kCols, (uint32_t)a.box, D / kCols, 1};
  constexpr CUtensorMapSwizzle kSwizzle = C::kRow < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  for (int i = 0; i < 2; ++i)
    if (!make_tmap(&maps[i], C::kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, kSwizzle,
                   i ? p.pool.v : p.pool.k, 4, dims, strides, box))
      return cudaErrorInvalidValue;
  const int ctas = min(sm_count(), kPagedMaxCtas);
  cudaError_t e = allow_smem_once<paged_attn_tma_kernel<T, D, HP, MW>>(C::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(paged_attn_tma_kernel<T, D, HP, MW>, dim3(ctas), dim3(C::kThreads), C::kSmem, s, maps[0], maps[1], a);
  if (e != cudaSuccess || a.whole) return e;
  return launch_paged_join(C::kBf16 ? NT_BF16 : NT_F32, p, ctas, a.items, HP, s);
}

template <int D>
cudaError_t run_d(nt_dtype dt, const PagedAttnProblem& p, unsigned int* status, cudaStream_t s) {
  const int G = p.H / p.pool.H;
  // The merge: one warp of its own; two for more than four heads (the ragged
  // batch of 64 with 8 heads to a key head of 128: 65.7 us with one, 60.1 with
  // two; with four heads 57.3 and 57.4, and many short contexts lose 4%, as the
  // registers have to do for 13 warps); the eight together for more than eight
  // (16 heads: 78 us where one alone took 104; the probabilities' second
  // product adds 2 to 5% to these).
  if (dt == NT_BF16) {
    if (G <= 4) return run<bf16, D, 8, 1>(p, status, s);
    return G <= 8 ? run<bf16, D, 8, 2>(p, status, s) : run<bf16, D, 16, 0>(p, status, s);
  }
  if (G == 1) return run<float, D, 1, 1>(p, status, s);
  if (G == 2) return run<float, D, 2, 1>(p, status, s);
  if (G <= 4) return run<float, D, 4, 1>(p, status, s);
  return run<float, D, 8, 1>(p, status, s);
}

}  // namespace

// An item costs an SM 0.5 us and 1.4 ns for each of its outputs.  Items kept
// whole: about 5 us and, for every round of them on the SMs, that and 0.75 us
// a 32 KB of keys and values.  Split: 8 us (the plan, the ragged end, the
// join; 11 with 16 heads), their cost, and 6.1 TB/s.
double paged_attn_tma_us(nt_dtype dt, const PagedAttnProblem& p) {
  if (p.pool.page_size % 8 || p.pool.n_pages == 0) return INFINITY;
  const int es = dt == NT_BF16 ? 2 : 4, G = p.H / p.pool.H, HP = dt == NT_BF16 && G > 8 ? 16 : 8;
  const double rounds = (double)paged_items(p, HP) / sm_count(), own = 0.5 + 0.0014 * min(G, HP) * p.d;
  const double keys = (double)paged_cap(p) * p.d * es * 2, mean = paged_mean_part(p);
  if (paged_whole_items(p, es))
    return (p.d == 128 ? 4.8 : 4.3) + own + 0.75 * keys / 32768 +
           fmax(0, rounds - 1) * (own + 0.75 * keys / 32768 * mean);
  return (HP == 16 ? 11 : p.d == 128 ? 8.5 : 8) + rounds * own + (double)p.B * p.pool.H * keys * mean / 6.1e6;
}

cudaError_t launch_paged_attn_tma(nt_dtype dt, const PagedAttnProblem& p, unsigned int* status, cudaStream_t s) {
  if (p.d == 32) return run_d<32>(dt, p, status, s);
  if (p.d == 64) return run_d<64>(dt, p, status, s);
  return run_d<128>(dt, p, status, s);
}

}  // namespace nt
