// Attention of drafted tokens over a paged cache on the tcgen05 tensor cores:
// bf16, head width 64 or 128, pages of a multiple of 8 positions, up to 128
// query heads to a key head.
//
// With G query heads to a key head and n new tokens of a sequence, a key and
// its value are 4 d bytes for 4 d n G operations: memory is the bound up to
// some 280 rows (n G), the products above.  So an item takes up to 128 rows
// (R = 1) or 256 (R = 2, two row tiles over the same keys), and its keys go by
// in tiles of 128, each fetched by TMA page by page into rings of shared memory
// and read there by the tensor cores for all rows at once.  The batch's tiles
// are dealt out evenly to one CTA per SM (draft_plan.cuh); items cut between
// CTAs are joined by a second kernel.
//
// A step is one row tile against one key tile:
//   S = Q K^T           (128 x 128; one of kBufs buffers in TMEM)
//   P = 2^(scale S - m) as the sum of two bf16, written over S
//   O += P V            (two products, P from TMEM; O stays in TMEM)
// Warps: 0 to 7 softmax, 8 issues the products, 9 and 10 fetch keys and
// values, 11 queries.  A row's 128 scores belong to two threads (warps w and
// w + 4), 64 each, which tell one another their maxima; a thread keeps its
// scores in registers from S to P.  The products of step s + 1 run under the
// softmax of step s, and the fetches under both.  The running maximum m moves
// only when a tile's exceeds it by 8 (a factor of 256, which fp32 sums and the
// bf16 parts of P bear), so O is rescaled on few tiles.
//
// Two bf16 for P: one would be off by 2^-8 of P, which shows in the output.
// The upper part is cut from P (1 - 2^-10), so that both parts are positive:
// an infinite value in the cache then gives the infinity that P times it is.
//
// Tiles behind the context (new tokens, the last key) are the only ones with a
// mask, and with rows of V that a product may not read as they are: those
// behind the last key hold anything and become zeros; values that are not
// finite are taken out, and added in the end to the rows that see them.
#include "draft_plan.cuh"
#include "draft_worker.cuh"

namespace nt {
namespace {

using namespace tc;

constexpr int kKeys = 128, kRows = 128;
constexpr int kSoftmax = 8;                         // warps
constexpr int kThreads = 12 * 32;
constexpr uint32_t kTmemCols = 512;

template <int D, int R>
struct Cfg {
  static constexpr uint32_t kHalf = kKeys * 128;                   // 64 columns of a tile
  static constexpr uint32_t kTile = kHalf * (D / 64);              // keys or values of a stage; a row tile of Q
  static constexpr int kQBufs = D == 128 && R == 2 ? 1 : 2;        // items whose queries are in flight or in use
  static constexpr uint32_t kQ = R * kTile;
  static constexpr uint32_t kCtl = 3072;
  static constexpr int kFit = (int)((227 * 1024 - kCtl - kQBufs * kQ) / kTile);
  static constexpr int kK = kFit / 2, kV = kFit - kK;              // stages of keys and of values
  static constexpr uint32_t kSmem = kQBufs * kQ + (kK + kV) * kTile + kCtl;
  static constexpr int kFitBufs = (512 - R * D) / 128;
  static constexpr int kBufs = kFitBufs > 3 ? 3 : kFitBufs;        // of S
  static constexpr uint32_t kColO = kBufs * 128;
  static constexpr int kExtra = 1;                                 // an item's cost beside its tiles, in tiles
  static_assert(kK >= 2 && kBufs >= 2 && kSmem <= 227 * 1024, "shared memory");
};

constexpr int kMaxStages = 7, kSpecial = 3;         // tiles behind the context, at most: 127 + 256 keys
struct Ctl {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[kMaxStages], k_empty[kMaxStages], v_full[kMaxStages], v_empty[kMaxStages];
  uint64_t s_full[3], p_full[3], pv_done[3], o_free, mma_done;
  uint64_t pair[4][2];                              // two warps of the same rows
  uint32_t tmem_base;
  int abort;
  unsigned int bad[3][kSpecial * 4 + 1];            // of three segments in turn: keys, and whether any
  float word[2][2][kRows];                          // what the two threads of a row tell one another
  PagedPlan plan;
};
static_assert(sizeof(Ctl) <= 3072, "control block");

struct TcArgs {
  DraftBatch a;
  const uint8_t* v;
  void* o;
  float* lse;
  void* workspace;
  bool whole;                     // items are not split
  int box;                        // keys per box: the largest power of two that divides page_size, 128 at most
  float scale_log2;
};

// Shared-memory descriptor of an MN-major operand: rows of 128 bytes along K,
// 8-row groups 1 KB apart, 64-element parts along N `part` bytes apart.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr, uint32_t part) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)((part >> 4) & 0x3FFFu) << 16 | (uint64_t)(1024u >> 4) << 32 |
         (uint64_t)1u << 46 | (uint64_t)2u << 61;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

template <int D, int R>
__global__ void __launch_bounds__(kThreads, 1)
draft_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap, const TcArgs p) {
  using C = Cfg<D, R>;
  constexpr int NB = C::kBufs, kE = C::kExtra, kPartRows = R * kRows;
  extern __shared__ __align__(1024) uint8_t smem[];
  const DraftBatch& a = p.a;
  if (smem_u32(smem) & 1023) {                      // the swizzled tiles need it
    if (threadIdx.x == 0) {
      flag_device(a.status, kDevCheck);
      draft_partials(p.workspace, gridDim.x, kPartRows).open[blockIdx.x] = make_int4(-1, 0, 0, 0);
    }
    return;
  }
  uint8_t* sq = smem;
  uint8_t* sk = sq + C::kQBufs * C::kQ;
  uint8_t* sv = sk + C::kK * C::kTile;
  Ctl* ctl = reinterpret_cast<Ctl*>(sv + C::kV * C::kTile);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &ctl->abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->q_full[i], 1);
      mbar_init(&ctl->q_empty[i], 1);
    }
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&ctl->k_full[i], 1);
      mbar_init(&ctl->k_empty[i], 1);
      mbar_init(&ctl->v_full[i], 1);
      mbar_init(&ctl->v_empty[i], 1);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->p_full[i], kSoftmax);
      mbar_init(&ctl->pv_done[i], 1);
      for (int k = 0; k <= kSpecial * 4; ++k) ctl->bad[i][k] = 0;
    }
    mbar_init(&ctl->o_free, kSoftmax);
    mbar_init(&ctl->mma_done, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&ctl->pair[i][0], 2);
      mbar_init(&ctl->pair[i][1], 2);
    }
    ctl->abort = 0;
    fence_mbar_init();
    fence_async_shared();
  }
  if (threadIdx.x == 9 * 32) prefetch_tmap(&kmap);
  if (threadIdx.x == 10 * 32) prefetch_tmap(&vmap);
  if (threadIdx.x == 11 * 32) prefetch_tmap(&qmap);
  if (warp == 8) tmem_alloc(&ctl->tmem_base, kTmemCols);
  pdl_wait();
  pdl_trigger();
  tc_fence_before();
  draft_plan(a, kKeys, kE, blockIdx.x, gridDim.x, &ctl->plan, kThreads);
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  DraftWalk w;
  w.init(a, ctl->plan, kKeys, kE, p.whole);
  const int tile_tokens = a.tokens / R;             // of a row tile

  if (warp == 11) {
    // ---- queries, item by item ------------------------------------------------
    if (lane == 0) {
      uint32_t segs = 0;
      while (w.next(a, kKeys, kE)) {
        const DraftItem it = draft_item(a, w.seq.n, w.seg_item, w.seg_items);
        const int slot = segs % C::kQBufs, tiles = it.ni > tile_tokens ? R : 1;
        if (!mbar_wait(&ctl->q_empty[slot], ((segs / C::kQBufs) & 1) ^ 1, abort, a.status)) break;
        const uint32_t rows = tile_tokens * a.heads;
        mbar_arrive_expect_tx(&ctl->q_full[slot], tiles * (D / 64) * rows * 128);
        for (int r = 0; r < tiles; ++r)
          for (int h = 0; h < D / 64; ++h)
            tma_load_3d(sq + slot * C::kQ + r * C::kTile + h * C::kHalf, &qmap, &ctl->q_full[slot], h * 64,
                        it.kvh * a.G, w.seq.first + it.i0 + r * tile_tokens);
        ++segs;
      }
      // no copy may land after the CTA is gone
      for (uint32_t i = segs > C::kQBufs ? segs - C::kQBufs : 0; i < segs; ++i)
        mbar_wait(&ctl->q_full[i % C::kQBufs], (i / C::kQBufs) & 1, nullptr, a.status);
    }
  } else if (warp == 9 || warp == 10) {
    // ---- keys (warp 9) and values (10): a lane to each box of a tile -----------------
    const bool vals = warp == 10;
    const CUtensorMap* map = vals ? &vmap : &kmap;
    uint64_t* full = vals ? ctl->v_full : ctl->k_full;
    uint64_t* empty = vals ? ctl->v_empty : ctl->k_empty;
    uint8_t* ring = vals ? sv : sk;
    const int S = vals ? C::kV : C::kK;
    const int boxes = kKeys / p.box, rb = lane % boxes, half = lane / boxes;
    const bool mine = half < D / 64;
    const uint32_t dst = half * C::kHalf + rb * p.box * 128, ps = a.page_size;
    uint32_t n = 0;                                 // tiles fetched
    bool ok = true;
    while (ok && w.next(a, kKeys, kE)) {
      const DraftItem it = draft_item(a, w.seq.n, w.seg_item, w.seg_items);
      const int32_t* row = a.table + (int64_t)w.seg_b * a.max_pages;
      // the table is read a tile ahead
      auto page_of = [&](int64_t t) {
        const uint32_t x = (uint32_t)t * kKeys + rb * p.box;
        return mine && t < w.t1 && x < (uint32_t)w.seq.len ? row[x / ps] : -1;
      };
      int next = page_of(w.t0);
      for (int64_t t = w.t0; t < w.t1; ++t, ++n) {
        const uint32_t x = (uint32_t)t * kKeys + rb * p.box;
        const bool now = mine && x < (uint32_t)w.seq.len;
        const int page = next;
        next = page_of(t + 1);
        int z = page * a.Hkv + it.kvh;
        if (now && (uint32_t)page >= (uint32_t)a.n_pages) {
          flag_device(a.status, kDevCheck);
          z = a.n_pages * a.Hkv;                    // outside the map: reads as zeros
        }
        const int st = n % S;
        ok = mbar_wait_warp(&empty[st], ((n / S) & 1) ^ 1, abort, a.status);
        if (!ok) break;
        const uint32_t count = __popc(__ballot_sync(0xffffffffu, now));
        if (lane == 0) mbar_arrive_expect_tx(&full[st], count * p.box * 128);
        __syncwarp();
        if (now) tma_load_3d(ring + st * C::kTile + dst, map, &full[st], half * 64, (int)(x % ps), z);
      }
    }
    if (lane == 0)
      for (uint32_t i = n > (uint32_t)S ? n - S : 0; i < n; ++i)
        mbar_wait(&full[i % S], (i / S) & 1, nullptr, a.status);
  } else if (warp == 8) {
    // ---- products --------------------------------------------------------------------
    // S of a step is issued kBufs - 1 steps before its P V.
    struct Pending {
      uint32_t s, tile;
      int r, parts;                                 // row tile; 16-key parts
      bool first, last;                             // of the segment's tiles; of the tile's row tiles
    };
    const uint32_t id_s = idesc_bf16_f32(128, kKeys);
    const uint32_t id_o = idesc_bf16_f32(128, D) | (1u << 16);   // V MN-major
    const uint32_t qb = smem_u32(sq), kb = smem_u32(sk), vb = smem_u32(sv);
    const bool leader = elect_one();
    constexpr int kAhead = NB - 1;
    Pending ring[kAhead];
    uint32_t s = 0, done = 0, tile = 0, segs = 0, seg_done = 0;
    bool ok = true;
    auto pv = [&](const Pending& x) {
      const int buf = x.s % NB, st = x.tile % C::kV;
      if (x.r == 0 && !mbar_wait_warp(&ctl->v_full[st], (x.tile / C::kV) & 1, abort, a.status)) return false;
      if (!mbar_wait_warp(&ctl->p_full[buf], (x.s / NB) & 1, abort, a.status)) return false;
      if (x.first && x.r == 0) {                    // the output of the segment before has been read
        if (seg_done > 0 && !mbar_wait_warp(&ctl->o_free, (seg_done - 1) & 1, abort, a.status)) return false;
        ++seg_done;
      }
      tc_fence_after();
      if (leader) {
        const uint32_t v0 = vb + st * C::kTile, d = tmem + C::kColO + x.r * D, pc = tmem + buf * 128;
        for (int k = 0; k < x.parts; ++k) {
          const uint64_t vd = sdesc_mn(v0 + k * 2048, C::kHalf);
          const uint32_t at = pc + (k >> 2) * 64 + (k & 3) * 8;
          mma_bf16_ts(d, at, vd, id_o, !x.first || k > 0);
          mma_bf16_ts(d, at + 32, vd, id_o, 1u);
        }
        mma_commit(&ctl->pv_done[buf]);
        if (x.last) mma_commit(&ctl->v_empty[st]);
      }
      __syncwarp();
      return true;
    };
    while (ok && w.next(a, kKeys, kE)) {
      const DraftItem it = draft_item(a, w.seq.n, w.seg_item, w.seg_items);
      const int slot = segs % C::kQBufs, tiles = it.ni > tile_tokens ? R : 1;
      if (C::kQBufs == 1)                           // the queries' copy waits for nothing but S: do not hold up P V
        for (; ok && done < s; ++done) ok = pv(ring[done % kAhead]);
      ok = ok && mbar_wait_warp(&ctl->q_full[slot], (segs / C::kQBufs) & 1, abort, a.status);
      for (int64_t t = w.t0; ok && t < w.t1; ++t, ++tile) {
        const int st = tile % C::kK;
        ok = mbar_wait_warp(&ctl->k_full[st], (tile / C::kK) & 1, abort, a.status);
        const int parts = (int)(min64(kKeys, w.seq.len - t * kKeys) + 15) / 16;
        for (int r = 0; ok && r < tiles; ++r, ++s) {
          const int buf = s % NB;
          if (s >= NB) ok = mbar_wait_warp(&ctl->pv_done[buf], ((s / NB) - 1) & 1, abort, a.status);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            const uint32_t q0 = qb + slot * C::kQ + r * C::kTile, k0 = kb + st * C::kTile;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t off = (k >> 2) * C::kHalf + (k & 3) * 32;
              mma_bf16(tmem + buf * 128, sdesc_k128(q0 + off), sdesc_k128(k0 + off), id_s, k > 0);
            }
            mma_commit(&ctl->s_full[buf]);
            if (r == tiles - 1) {
              mma_commit(&ctl->k_empty[st]);
              if (t == w.t1 - 1) mma_commit(&ctl->q_empty[slot]);
            }
          }
          __syncwarp();
          if (s - done == (uint32_t)kAhead) {
            ok = pv(ring[done % kAhead]);
            ++done;
            if (!ok) break;
          }
          ring[s % kAhead] = {s, tile, r, parts, t == w.t0, r == tiles - 1};
        }
      }
      ++segs;
    }
    for (; ok && done < s; ++done) ok = pv(ring[done % kAhead]);
    if (leader) mma_commit(&ctl->mma_done);
    __syncwarp();
    mbar_wait_warp(&ctl->mma_done, 0, nullptr, a.status);
  } else {
    // ---- softmax --------------------------------------------------------------------------
    const int quad = warp & 3, side = warp >> 2, row = quad * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const DraftPartials part = draft_partials(p.workspace, gridDim.x, kPartRows);
    int4 open = make_int4(-1, 0, 0, 0);
    uint32_t s = 0, tile = 0, segs = 0, told = 0;
    bool ok = true;
    // the other thread of the row tells its value for this one's
    auto tell = [&](float mine, float& other) {
      ctl->word[told & 1][side][row] = mine;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->pair[quad][told & 1]);
      if (!mbar_wait_warp(&ctl->pair[quad][told & 1], (told >> 1) & 1, abort, a.status)) return false;
      other = ctl->word[told & 1][side ^ 1][row];
      ++told;
      return true;
    };
    while (ok && w.next(a, kKeys, kE)) {
      const DraftItem it = draft_item(a, w.seq.n, w.seg_item, w.seg_items);
      const int tiles = it.ni > tile_tokens ? R : 1;
      const int tok = row / a.heads, ctx = w.seq.len - w.seq.n;   // the row's token in its row tile
      unsigned int* bad = ctl->bad[segs % 3];
      if (threadIdx.x == 0)                         // nobody is in the segment before the last any more
        for (int k = 0; k <= kSpecial * 4; ++k) ctl->bad[(segs + 1) % 3][k] = 0;
      float m[R], l[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
      }
      for (int64_t t = w.t0; ok && t < w.t1; ++t, ++tile) {
        const int64_t x0 = t * kKeys + side * 64;
        const bool special = t * kKeys + kKeys > ctx;
        for (int r = 0; ok && r < tiles; ++r, ++s) {
          const int buf = s % NB, i = it.i0 + r * tile_tokens + tok;
          const bool valid = tok < tile_tokens && i < it.i0 + it.ni;
          const bool live = __any_sync(0xffffffffu, valid);
          ok = mbar_wait_warp(&ctl->s_full[buf], (s / NB) & 1, abort, a.status);
          if (!ok) break;
          tc_fence_after();
          if (live) {
            const uint32_t s_at = lanes + buf * 128 + side * 64, o_at = lanes + C::kColO + r * D + side * (D / 2);
            float x[64];
            tmem_ld64_sync(s_at, x);
            if (special) {
              const uint64_t see = valid ? draft_sees(a, w.seq, i, x0) : 0;
#pragma unroll
              for (int c = 0; c < 64; ++c)
                if (!(see >> c & 1)) x[c] = -INFINITY;
            }
            float pm[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int c = 4; c < 60; c += 8) {
              pm[0] = max3(pm[0], x[c], x[c + 1]);
              pm[1] = max3(pm[1], x[c + 2], x[c + 3]);
              pm[2] = max3(pm[2], x[c + 4], x[c + 5]);
              pm[3] = max3(pm[3], x[c + 6], x[c + 7]);
            }
            pm[0] = max3(pm[0], x[60], x[61]);
            pm[1] = max3(pm[1], x[62], x[63]);
            float mx = valid ? fmaxf(max3(pm[0], pm[1], pm[2]), pm[3]) : -INFINITY, other;
            ok = tell(mx, other);
            if (!ok) break;
            const float cand = fmaxf(mx, other) * p.scale_log2;
            float mr = R == 1 || r == 0 ? m[0] : m[R - 1], lr = R == 1 || r == 0 ? l[0] : l[R - 1];
            float corr = 1.f;
            const bool move = cand > mr + 8.f;
            if (move) {
              corr = ex2_approx(mr - cand);         // 0 on the first tile
              mr = cand;
            }
            if (t > w.t0 && __any_sync(0xffffffffu, move)) {
              const uint32_t before = s - tiles;    // the step whose P V this row tile's output waits for
              ok = mbar_wait_warp(&ctl->pv_done[before % NB], (before / NB) & 1, abort, a.status);
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D / 2; c += 32) {
                float ov[32];
                tmem_ld32_sync(o_at + c, ov);
#pragma unroll
                for (int e = 0; e < 32; ++e) ov[e] *= corr;
                tmem_st32(o_at + c, ov);
              }
              tmem_st_wait();
            }
            const float base = mr == -INFINITY ? 0.f : mr;
            float ps[4] = {0.f, 0.f, 0.f, 0.f};
            uint32_t hi[32], lo[32];
#pragma unroll
            for (int c = 0; c < 64; c += 2) {
              float e0, e1, c0, c1, r0, r1;
              ffma2(x[c], x[c + 1], p.scale_log2, p.scale_log2, -base, -base, e0, e1);
              e0 = ex2_approx(e0);
              e1 = ex2_approx(e1);
              if ((c >> 1) & 1) fadd2(ps[2], ps[3], e0, e1, ps[2], ps[3]);
              else fadd2(ps[0], ps[1], e0, e1, ps[0], ps[1]);
              constexpr float kBelow = 1.f - 1.f / 1024;
              fmul2(e0, e1, kBelow, kBelow, c0, c1);
              hi[c / 2] = __byte_perm(__float_as_uint(c0), __float_as_uint(c1), 0x7632);
              ffma2(bf16lo(hi[c / 2]), bf16hi(hi[c / 2]), -1.f, -1.f, e0, e1, r0, r1);
              lo[c / 2] = pack_bf16x2(r0, r1);
            }
            lr = lr * corr + ((ps[0] + ps[1]) + (ps[2] + ps[3]));
            if (R == 1 || r == 0) m[0] = mr, l[0] = lr;
            else m[R - 1] = mr, l[R - 1] = lr;
            __syncwarp();
            tmem_st32(s_at, reinterpret_cast<const float*>(hi));
            tmem_st32(s_at + 32, reinterpret_cast<const float*>(lo));
            tmem_st_wait();
          }
          if (special && r == 0) {
            // V as the product may read it
            const int st = tile % C::kV;
            ok = mbar_wait_warp(&ctl->v_full[st], (tile / C::kV) & 1, abort, a.status);
            if (!ok) break;
            const int left = (int)min64(kKeys, w.seq.len - t * kKeys), end = (left + 15) / 16 * 16;
            uint8_t* v0 = sv + st * C::kTile;
            for (int e = threadIdx.x; e < end * (D / 8); e += kSoftmax * 32) {
              const int key = e / (D / 8), c = e % (D / 8);
              uint8_t* at = v0 + (c >> 3) * C::kHalf + key * 128 + (c & 7) * 16;
              if (key >= left) {
                *reinterpret_cast<uint4*>(at) = make_uint4(0, 0, 0, 0);
              } else if (draft::clear_bad<bf16>(at)) {
                const int k = (int)(t - ctx / kKeys) * kKeys + key;
                atomicOr(&bad[k >> 5], 1u << (k & 31));
                bad[kSpecial * 4] = 1;
              }
            }
            fence_async_shared();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->p_full[buf]);
        }
      }
      if (!ok) break;
      // ---- the segment's output: complete with its last P V
      const uint32_t last = s - 1;
      ok = mbar_wait_warp(&ctl->pv_done[last % NB], (last / NB) & 1, abort, a.status);
      if (!ok) break;
      tc_fence_after();
      const bool whole = w.begins && w.ends, odd = bad[kSpecial * 4] != 0;
      const int64_t pslot = 2 * (int64_t)blockIdx.x + (w.begins ? 1 : 0);
#pragma unroll 1
      for (int r = 0; ok && r < tiles; ++r) {
        const int i = it.i0 + r * tile_tokens + tok, h = it.kvh * a.G + row % a.heads;
        const bool valid = tok < tile_tokens && i < it.i0 + it.ni;
        if (!__any_sync(0xffffffffu, valid)) continue;
        const float mr = R == 1 || r == 0 ? m[0] : m[R - 1], lr = R == 1 || r == 0 ? l[0] : l[R - 1];
        float lo;
        ok = tell(lr, lo);
        if (!ok) break;
        const float ll = side ? lo + lr : lr + lo;
        const int64_t tt = (int64_t)w.seq.first + i;
        const bool any = valid && draft_sees_any(a, w.seq, i);
        const float inv = any ? 1.f / ll : 0.f;
#pragma unroll 1
        for (int c = 0; c < D / 2; c += 32) {
          float ov[32];
          __syncwarp();
          tmem_ld32_sync(lanes + C::kColO + r * D + side * (D / 2) + c, ov);
          if (valid && odd) {
            for (int64_t t = max64(w.t0, ctx / kKeys); t < w.t1; ++t)
              for (int k = 0; k < 4; ++k) {
                const unsigned int there = bad[(int)(t - ctx / kKeys) * 4 + k];
                if (!there) continue;
                const int64_t x0 = t * kKeys + k * 32;
                unsigned int todo = there & (unsigned int)draft_sees(a, w.seq, i, x0);
                for (; todo; todo &= todo - 1) {
                  const int64_t x = x0 + __ffs(todo) - 1;
                  const int pg = (int)(x / a.page_size), id = a.table[(int64_t)w.seg_b * a.max_pages + pg];
                  const uint4* vr = reinterpret_cast<const uint4*>(
                      p.v + ((((int64_t)id * a.Hkv + it.kvh) * a.page_size + (x - (int64_t)pg * a.page_size)) * D +
                             side * (D / 2) + c) * 2);
#pragma unroll
                  for (int u = 0; u < 4; ++u) {
                    const uint4 q = vr[u];
                    const uint32_t z[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                      ov[8 * u + 2 * y] += draft::if_bad(bf16lo(z[y]));
                      ov[8 * u + 2 * y + 1] += draft::if_bad(bf16hi(z[y]));
                    }
                  }
                }
              }
          }
          if (valid && whole) {
            uint4* to = reinterpret_cast<uint4*>(static_cast<bf16*>(p.o) + (tt * a.H + h) * D + side * (D / 2) + c);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              uint4 x;
              x.x = pack_bf16x2(ov[8 * u] * inv, ov[8 * u + 1] * inv);
              x.y = pack_bf16x2(ov[8 * u + 2] * inv, ov[8 * u + 3] * inv);
              x.z = pack_bf16x2(ov[8 * u + 4] * inv, ov[8 * u + 5] * inv);
              x.w = pack_bf16x2(ov[8 * u + 6] * inv, ov[8 * u + 7] * inv);
              to[u] = any ? x : make_uint4(0, 0, 0, 0);
            }
          } else if (valid) {
            const int64_t slot = pslot * kPartRows + r * tile_tokens * a.heads + row;
            float4* to = reinterpret_cast<float4*>(part.o + slot * D + side * (D / 2) + c);
#pragma unroll
            for (int u = 0; u < 8; ++u) to[u] = make_float4(ov[4 * u], ov[4 * u + 1], ov[4 * u + 2], ov[4 * u + 3]);
            if (side == 0 && c == 0) *reinterpret_cast<float2*>(part.ml + slot * 2) = make_float2(mr, ll);
          }
        }
        if (whole && valid && side == 0 && p.lse) p.lse[(int64_t)h * a.T + tt] = draft::row_lse(mr, ll, any);
      }
      if (!ok) break;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->o_free);
      if (w.begins && !w.ends)
        open = make_int4(w.seg_b, w.seg_item, w.seg_items, w.parts(ctl->plan, kE, blockIdx.x, gridDim.x));
      ++segs;
    }
    if (threadIdx.x == 0) part.open[blockIdx.x] = open;
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, int R>
cudaError_t run(const DraftProblem& p, unsigned int* status, cudaStream_t s) {
  using C = Cfg<D, R>;
  static_assert(C::kK <= kMaxStages && C::kV <= kMaxStages, "barriers");
  TcArgs r = {};
  r.a = draft_batch(p, kRows, R, status);
  r.v = static_cast<const uint8_t*>(p.pool.v);
  r.o = p.o;
  r.lse = p.lse;
  r.workspace = p.workspace;
  r.whole = false;
  r.box = kKeys;
  while (p.pool.page_size % r.box) r.box >>= 1;
  r.scale_log2 = p.scale * 1.4426950408889634f;
  CUtensorMap maps[3];
  {
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)p.H, (uint64_t)p.T};
    const uint64_t strides[2] = {(uint64_t)D * 2, (uint64_t)p.q_stride * 2};
    const uint32_t box[3] = {64, (uint32_t)r.a.heads, (uint32_t)(r.a.tokens / R)};
    if (!make_tmap_bf16(&maps[0], p.q, 3, dims, strides, box)) return cudaErrorInvalidValue;
  }
  for (int i = 0; i < 2; ++i) {
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)p.pool.page_size, (uint64_t)p.pool.n_pages * p.pool.H};
    const uint64_t strides[2] = {(uint64_t)D * 2, (uint64_t)D * 2 * p.pool.page_size};
    const uint32_t box[3] = {64, (uint32_t)r.box, 1};
    if (!make_tmap_bf16(&maps[1 + i], i ? p.pool.v : p.pool.k, 3, dims, strides, box)) return cudaErrorInvalidValue;
  }
  const int ctas = min(sm_count(), kPagedMaxCtas);
  cudaError_t e = allow_smem_once<draft_tc_kernel<D, R>>(C::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(draft_tc_kernel<D, R>, dim3(ctas), dim3(kThreads), C::kSmem, s, maps[0], maps[1], maps[2], r);
  if (e != cudaSuccess || r.whole) return e;
  return launch_draft_join(NT_BF16, r.a, D, ctas, R * kRows, p.workspace, p.o, p.lse, s);
}

}  // namespace

bool draft_tc_supported(nt_dtype dt, const DraftProblem& p) {
  return dt == NT_BF16 && (p.d == 64 || p.d == 128) && p.pool.page_size % 8 == 0 && p.pool.n_pages > 0 &&
         p.H / p.pool.H <= kRows;
}

cudaError_t launch_draft_tc(const DraftProblem& p, unsigned int* status, cudaStream_t s) {
  // two row tiles to an item where sequences have more rows than one takes
  const int G = p.H / p.pool.H;
  const bool two = p.max_new > kRows / G;
  if (p.d == 64) return two ? run<64, 2>(p, status, s) : run<64, 1>(p, status, s);
  return two ? run<128, 2>(p, status, s) : run<128, 1>(p, status, s);
}

}  // namespace nt
