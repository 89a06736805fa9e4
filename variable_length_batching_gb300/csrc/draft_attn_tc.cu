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
//   S = Q K^T           (128 x 128 in TMEM)
//   P = 2^(scale S - m) as the sum of two bf16, written over S
//   O += P V            (two products, P from TMEM; O stays in TMEM)
// Steps alternate between two streams, each with its S, its O and its
// softmax warps, a row to a thread: with two row tiles a stream is a row tile;
// with one, the streams take every other key tile, and their sums are joined
// in the end.  So the products of one stream run under the softmax of the
// other, and the fetches under both.  Warps: 0 to 3 and 4 to 7 softmax, 8 issues
// Q K^T and 11 P V, each as soon as its operands are there (one warp for both
// took over 1,000 cycles a step to find out which), 9 fetches queries and keys,
// 10 values.  The running maximum m moves only when a tile's exceeds it by 8 (a
// factor of 256, which fp32 sums and the bf16 parts of P bear), so O is rescaled
// on few tiles.
//
// Measured in a graph: 152 contexts of 8,000 keys, 16 rows to a key head, 103 us at
// d = 128 (89% of the copy rate) and 69 at d = 64, where a row's 128 exponentials
// (1,550 cycles of a step's 2,900) are what a stream waits for; with 256 rows d = 128
// 178 and d = 64 139.  8 pieces of 256 tokens behind 2,000 to 16,000 keys, d = 128:
// 300 us, 866 TFLOP/s of the result's products, three of which are made for two (a
// call among others on cold inputs 319); a product of 128 x 128 x 16 takes some 93
// cycles here, 4,460 of a step's 4,750.
//
// Two bf16 for P: one would be off by 2^-8 of P, which shows in the output.
// The upper part is P cut short, the lower P (1 + 2^-20) less that, so that
// both are positive: an infinite value in the cache then gives the infinity
// that P times it is.
//
// Tiles behind the context (new tokens, the last key) are the only ones with a
// mask (applied where a warp's rows do not see all of one), and with rows of V that a product may not read as they are: those
// behind the last key hold anything and become zeros; values that are not
// finite are taken out, and added in the end to the rows that see them.
#include "draft_plan.cuh"
#include "draft_worker.cuh"

namespace nt {
namespace {

using namespace tc;

constexpr int kKeys = 128, kRows = 128;
constexpr int kSoftmax = 8;                         // warps, four to a stream
constexpr int kThreads = 12 * 32;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;                     // S of stream g at 128 g, O at kColO + D g

template <int D, int R>
struct Cfg {
  static constexpr uint32_t kHalf = kKeys * 128;                   // 64 columns of a tile
  static constexpr uint32_t kTile = kHalf * (D / 64);              // keys or values of a stage; a row tile of Q
  static constexpr int kQBufs = D == 128 && R == 2 ? 1 : 2;        // items whose queries are in flight or in use
  static constexpr uint32_t kQ = R * kTile;
  static constexpr uint32_t kCtl = 2944;
  static constexpr int kFit = (int)((227 * 1024 - kCtl - kQBufs * kQ) / kTile);
  static constexpr int kK = kFit / 2, kV = kFit - kK;              // stages of keys and of values
  static constexpr uint32_t kSmem = kQBufs * kQ + (kK + kV) * kTile + kCtl;
  // an item's cost beside its tiles, in tiles (pieces of 256 tokens, d = 128, in a graph: 332 us with two, 315 with four)
  static constexpr int kExtra = D == 64 ? (R == 1 ? 4 : 3) : R == 1 ? 3 : 4;
  static_assert(kK >= 2 && kSmem <= 227 * 1024, "shared memory");
};

constexpr int kMaxStages = 7, kSpecial = 3;         // tiles behind the context, at most: 127 + 256 keys
struct Ctl {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[kMaxStages], k_empty[kMaxStages], v_full[kMaxStages], v_empty[kMaxStages];
  uint64_t s_full[2], p_full[2][2], pv_done[2], o_free, s_end, pv_end;   // of a stream; P: of each half of its keys
  uint64_t pair[4];                                 // two warps of the same rows
  uint32_t tmem_base;
  int abort;
  unsigned int bad[3][kSpecial * 4 + 1];            // of three segments in turn: keys, and whether any
  float2 word[2][kRows];                            // maximum and sum of a row in a stream
  DraftPlanSums plan;
};
static_assert(sizeof(Ctl) <= 2944, "control block");

struct TcArgs {
  DraftBatch a;
  const uint8_t* v;
  void* o;
  float* lse;
  void* workspace;
  int box;                        // keys per box: the largest power of two that divides page_size, 128 at most
  int page_shift;                 // of a page_size that is a power of two, else -1
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

// mbar_wait, whose clock is read only after some tries; by one thread, and by
// a warp.
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned int* status) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait(bar, parity, abort, status);
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned int* status) {
  return __all_sync(0xffffffffu, wait_one(bar, parity, abort, status));
}

// Columns [c, c + 32) of what was taken out of the segment's tiles, added to
// the outputs of new token i where it sees them.
__device__ __forceinline__ void add_bad(const DraftBatch& a, const DraftWalk& w, const DraftItem& it, int i,
                                        const unsigned int* bad, const uint8_t* v, int c, int d, float (&ov)[32]) {
  const int64_t t0 = (w.seq.len - w.seq.n) / kKeys;
  for (int64_t t = max64(w.t0, t0); t < w.t1; ++t)
    for (int k = 0; k < 4; ++k) {
      const unsigned int there = bad[(int)(t - t0) * 4 + k];
      if (!there) continue;
      const int64_t x0 = t * kKeys + k * 32;
      unsigned int todo = there & (unsigned int)draft_sees(a, w.seq, i, x0);
      for (; todo; todo &= todo - 1) {
        const int64_t x = x0 + __ffs(todo) - 1;
        const int pg = (int)(x / a.page_size), id = a.table[(int64_t)w.seg_b * a.max_pages + pg];
        if ((unsigned)id >= (unsigned)a.n_pages) continue;
        const uint4* vr = reinterpret_cast<const uint4*>(
            v + ((((int64_t)id * a.Hkv + it.kvh) * a.page_size + (x - (int64_t)pg * a.page_size)) * d + c) * 2);
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

template <int D, int R>
__global__ void __launch_bounds__(kThreads, 1)
draft_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap, const TcArgs p) {
  using C = Cfg<D, R>;
  constexpr int kE = C::kExtra, kPartRows = R * kRows;
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
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->p_full[i][0], kSoftmax / 2);
      mbar_init(&ctl->p_full[i][1], kSoftmax / 2);
      mbar_init(&ctl->pv_done[i], 1);
    }
    for (int i = 0; i < 3; ++i)
      for (int k = 0; k <= kSpecial * 4; ++k) ctl->bad[i][k] = 0;
    mbar_init(&ctl->o_free, kSoftmax);
    mbar_init(&ctl->s_end, 1);
    mbar_init(&ctl->pv_end, 1);
    for (int i = 0; i < 4; ++i) mbar_init(&ctl->pair[i], 2);
    ctl->abort = 0;
    fence_mbar_init();
    fence_async_shared();
  }
  if (threadIdx.x == 9 * 32) {
    prefetch_tmap(&qmap);
    prefetch_tmap(&kmap);
  }
  if (threadIdx.x == 10 * 32) prefetch_tmap(&vmap);
  if (warp == 8) tmem_alloc(&ctl->tmem_base, kTmemCols);
  pdl_wait();
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const DraftPlan plan = draft_plan(a, kKeys, kE, blockIdx.x, gridDim.x, &ctl->plan, kThreads);
  DraftWalk w;
  w.init(a, plan, kKeys, kE);
  const int tile_tokens = a.tokens / R;             // of a row tile

  if (warp == 9 || warp == 10) {
    // ---- queries and keys (warp 9), values (10): a lane to each box of a tile ----------
    const bool vals = warp == 10;
    const CUtensorMap* map = vals ? &vmap : &kmap;
    uint64_t* full = vals ? ctl->v_full : ctl->k_full;
    uint64_t* empty = vals ? ctl->v_empty : ctl->k_empty;
    uint8_t* ring = vals ? sv : sk;
    const int S = vals ? C::kV : C::kK;
    const int boxes = kKeys / p.box, rb = lane % boxes, half = lane / boxes;
    const bool mine = half < D / 64;
    const uint32_t dst = half * C::kHalf + rb * p.box * 128, ps = a.page_size;
    uint32_t n = 0, segs = 0;                       // tiles and queries fetched
    bool ok = true;
    while (ok && w.next(a, kKeys, kE)) {
      const DraftItem& it = w.it;
      const int32_t* row = a.table + (int64_t)w.seg_b * a.max_pages;
      // the table is read a tile ahead
      auto page_of = [&](int64_t t) {
        const uint32_t x = (uint32_t)t * kKeys + rb * p.box;
        return mine && t < w.t1 && x < (uint32_t)w.seq.len ? row[p.page_shift >= 0 ? x >> p.page_shift : x / ps] : -1;
      };
      int next = page_of(w.t0);
      if (!vals) {
        const int slot = segs % C::kQBufs, tiles = it.ni > tile_tokens ? R : 1;
        ok = wait(&ctl->q_empty[slot], ((segs / C::kQBufs) & 1) ^ 1, abort, a.status);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&ctl->q_full[slot], tiles * (D / 64) * tile_tokens * a.heads * 128);
          for (int r = 0; r < tiles; ++r)
            for (int h = 0; h < D / 64; ++h)
              tma_load_3d(sq + slot * C::kQ + r * C::kTile + h * C::kHalf, &qmap, &ctl->q_full[slot], h * 64,
                          it.kvh * a.G, w.seq.first + it.i0 + r * tile_tokens);
        }
        ++segs;
      }
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
        ok = wait(&empty[st], ((n / S) & 1) ^ 1, abort, a.status);
        if (!ok) break;
        const uint32_t count = __popc(__ballot_sync(0xffffffffu, now));
        if (lane == 0) mbar_arrive_expect_tx(&full[st], count * p.box * 128);
        __syncwarp();
        if (now)
          tma_load_3d(ring + st * C::kTile + dst, map, &full[st], half * 64,
                      (int)(p.page_shift >= 0 ? x & (ps - 1) : x % ps), z);
      }
    }
    // no copy may land after the CTA is gone
    if (lane == 0) {
      for (uint32_t i = n > (uint32_t)S ? n - S : 0; i < n; ++i)
        mbar_wait(&full[i % S], (i / S) & 1, nullptr, a.status);
      for (uint32_t i = segs > C::kQBufs ? segs - C::kQBufs : 0; i < segs; ++i)
        mbar_wait(&ctl->q_full[i % C::kQBufs], (i / C::kQBufs) & 1, nullptr, a.status);
    }
  } else if (warp == 8) {
    // ---- S = Q K^T: step s of the CTA is stream s & 1's ------------------------------------
    if (elect_one()) {
      const uint32_t id_s = idesc_bf16_f32(128, kKeys);
      const uint64_t q_desc = sdesc_k128(smem_u32(sq)), k_desc = sdesc_k128(smem_u32(sk));
      uint32_t s = 0, st = 0, ph = 0, segs = 0;
      bool ok = true;
      while (ok && w.next(a, kKeys, kE)) {
        const DraftItem& it = w.it;
        const int slot = segs % C::kQBufs, tiles = it.ni > tile_tokens ? R : 1;
        ok = wait_one(&ctl->q_full[slot], (segs / C::kQBufs) & 1, abort, a.status);
        for (int t = (int)(w.t1 - w.t0); ok && t > 0; --t) {
          ok = wait_one(&ctl->k_full[st], ph, abort, a.status);
          const uint64_t k0 = k_desc + st * (C::kTile >> 4);
          uint64_t q0 = q_desc + slot * (C::kQ >> 4);
          for (int r = tiles; ok && r > 0; --r, ++s, q0 += C::kTile >> 4) {
            const uint32_t g = s & 1;
            if (s >= 2 && !(ok = wait_one(&ctl->pv_done[g], ((s >> 1) - 1) & 1, abort, a.status))) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t off = ((k >> 2) * C::kHalf + (k & 3) * 32) >> 4;
              mma_bf16(tmem + g * kKeys, q0 + off, k0 + off, id_s, k > 0);
            }
            mma_commit(&ctl->s_full[g]);
          }
          if (!ok) break;
          mma_commit(&ctl->k_empty[st]);
          if (t == 1) mma_commit(&ctl->q_empty[slot]);
          if (++st == C::kK) st = 0, ph ^= 1;
        }
        ++segs;
      }
      mma_commit(&ctl->s_end);
      mbar_wait(&ctl->s_end, 0, nullptr, a.status);
    }
  } else if (warp == 11) {
    // ---- O += P V ----------------------------------------------------------------------------
    if (elect_one()) {
      const uint32_t id_o = idesc_bf16_f32(128, D) | (1u << 16);   // V MN-major
      const uint64_t v_desc = sdesc_mn(smem_u32(sv), C::kHalf);
      uint32_t s = 0, st = 0, ph = 0, segs = 0;
      bool ok = true;
      while (ok && w.next(a, kKeys, kE)) {
        const DraftItem& it = w.it;
        const int tiles = it.ni > tile_tokens ? R : 1, tiles_k = (int)(w.t1 - w.t0);
        for (int t = 0; ok && t < tiles_k; ++t) {
          ok = wait_one(&ctl->v_full[st], ph, abort, a.status);
          const uint64_t v0 = v_desc + st * (C::kTile >> 4);
          for (int r = 0; ok && r < tiles; ++r, ++s) {
            const uint32_t g = s & 1;
            ok = wait_one(&ctl->p_full[g][0], (s >> 1) & 1, abort, a.status);
            // the output of the segment before has been read
            if (ok && t == 0 && r == 0 && segs > 0) ok = wait_one(&ctl->o_free, (segs - 1) & 1, abort, a.status);
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = tmem + kColO + g * D, pc = tmem + g * kKeys, add = tiles == 1 ? t > 1 : t > 0;
            const int left = w.seq.len - (int)(w.t0 + t) * kKeys;
            auto part = [&](int k) {                // 16 keys
              const uint32_t at = pc + (k >> 1) * 32 + (k & 1) * 8;
              mma_bf16_ts(d, at, v0 + k * (2048 >> 4), id_o, k > 0 ? 1u : add);
              mma_bf16_ts(d, at + 16, v0 + k * (2048 >> 4), id_o, 1u);
            };
            if (left >= kKeys) {
#pragma unroll
              for (int k = 0; k < kKeys / 32; ++k) part(k);
            } else {
              for (int k = 0; k < kKeys / 32 && k * 16 < left; ++k) part(k);
            }
            ok = wait_one(&ctl->p_full[g][1], (s >> 1) & 1, abort, a.status);
            if (!ok) break;
            tc_fence_after();
            if (left >= kKeys) {
#pragma unroll
              for (int k = kKeys / 32; k < kKeys / 16; ++k) part(k);
            } else {
              for (int k = kKeys / 32; k * 16 < left; ++k) part(k);
            }
            mma_commit(&ctl->pv_done[g]);
          }
          if (!ok) break;
          mma_commit(&ctl->v_empty[st]);
          if (++st == C::kV) st = 0, ph ^= 1;
        }
        ++segs;
      }
      mma_commit(&ctl->pv_end);
      mbar_wait(&ctl->pv_end, 0, nullptr, a.status);
    }
  } else {
    // ---- softmax --------------------------------------------------------------------------
    const int quad = warp & 3, g = warp >> 2, row = quad * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16), s_at = lanes + g * kKeys;
    const DraftPartials part = draft_partials(p.workspace, gridDim.x, kPartRows);
    const int tok = row / a.heads;                  // the row's token in its row tile
    int4 open = make_int4(-1, 0, 0, 0);
    uint32_t s0 = 0, tile0 = 0, segs = 0, told = 0;                // steps and tiles before the segment
    bool ok = true;
    while (ok && w.next(a, kKeys, kE)) {
      const DraftItem& it = w.it;
      const int tiles = it.ni > tile_tokens ? R : 1, ctx = w.seq.len - w.seq.n;
      const int e = g ^ (s0 & 1);                   // this stream's first step of the segment, and its row tile
      const int i = it.i0 + (tiles == 1 ? 0 : e * tile_tokens) + tok;
      const bool valid = tok < tile_tokens && i < it.i0 + it.ni;
      const bool live = __any_sync(0xffffffffu, valid);
      unsigned int* bad = ctl->bad[segs % 3];
      float m = -INFINITY, l = 0.f;
      DraftMask mask;
      mask.read(a, w.seq, i, valid);
      const int t_lo = (int)w.t0, t_hi = (int)w.t1, step = tiles == 1 ? 2 : 1, t_first = t_lo + (tiles == 1 ? e : 0);
      uint32_t s = s0 + e;
      for (int t = t_first; t < t_hi; t += step, s += 2) {
        const bool special = t * kKeys + kKeys > ctx;
        ok = wait(&ctl->s_full[g], (s >> 1) & 1, abort, a.status);
        if (!ok) break;
        tc_fence_after();
        if (live) {
          uint64_t see[2] = {~0ull, ~0ull};
          bool masked = false;                      // a row of the warp does not see all of the tile
          if (special) {
            see[0] = valid ? mask.sees(a, w.seq, i, t * kKeys) : ~0ull;
            see[1] = valid ? mask.sees(a, w.seq, i, t * kKeys + 64) : ~0ull;
            masked = __any_sync(0xffffffffu, (see[0] & see[1]) != ~0ull);
          }
          float mx = -INFINITY;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            float x[64];
            tmem_ld64_sync(s_at + 64 * h, x);
            if (masked) {
#pragma unroll
              for (int c = 0; c < 64; ++c)
                if (!((h ? see[1] : see[0]) >> c & 1)) x[c] = -INFINITY;
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
            mx = max3(mx, max3(pm[0], pm[1], pm[2]), pm[3]);
          }
          const float cand = valid ? mx * p.scale_log2 : -INFINITY;
          float corr = 1.f;
          const bool move = cand > m + 8.f;
          if (move) {
            corr = ex2_approx(m - cand);            // 0 on the first tile
            m = cand;
          }
          if (t > t_first && __any_sync(0xffffffffu, move)) {
            // the stream's P V before this step has completed: S was issued after that
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float ov[32];
              tmem_ld32_sync(lanes + kColO + g * D + c, ov);
#pragma unroll
              for (int y = 0; y < 32; ++y) ov[y] *= corr;
              tmem_st32(lanes + kColO + g * D + c, ov);
            }
            tmem_st_wait();
          }
          const float base = m == -INFINITY ? 0.f : m;
          float ps[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
          for (int c0 = 0; c0 < kKeys; c0 += 32) {
            float x[32];
            uint32_t pw[32];                        // upper parts, then lower parts
            tmem_ld32_sync(s_at + c0, x);
            if (masked) {
              const uint32_t there = (uint32_t)((c0 < 64 ? see[0] : see[1]) >> (c0 & 32));
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(there >> c & 1)) x[c] = -INFINITY;
            }
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              float e0, e1, r0, r1;
              ffma2(x[c], x[c + 1], p.scale_log2, p.scale_log2, -base, -base, e0, e1);
              e0 = ex2_approx(e0);
              e1 = ex2_approx(e1);
              if ((c >> 1) & 1) fadd2(ps[2], ps[3], e0, e1, ps[2], ps[3]);
              else fadd2(ps[0], ps[1], e0, e1, ps[0], ps[1]);
              pw[c / 2] = __byte_perm(__float_as_uint(e0), __float_as_uint(e1), 0x7632);
              constexpr float kAbove = 1.f + 1.f / (1 << 20);
              ffma2(e0, e1, kAbove, kAbove, __uint_as_float((__float_as_uint(e0) & 0xffff0000u) ^ 0x80000000u),
                    __uint_as_float((__float_as_uint(e1) & 0xffff0000u) ^ 0x80000000u), r0, r1);
              pw[16 + c / 2] = pack_bf16x2(r0, r1);
            }
            tmem_st32(s_at + c0, reinterpret_cast<const float*>(pw));
            if (c0 == 32 && !special) {             // the product of these may begin
              tmem_st_wait();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&ctl->p_full[g][0]);
            }
          }
          l = l * corr + ((ps[0] + ps[1]) + (ps[2] + ps[3]));
          tmem_st_wait();
        }
        if (special && (tiles == 1 || e == 0)) {
          // V as the product may read it
          const uint32_t tile = tile0 + (uint32_t)(t - t_lo);
          const int st = tile % C::kV;
          ok = wait(&ctl->v_full[st], (tile / C::kV) & 1, abort, a.status);
          if (!ok) break;
          const int left = min(kKeys, w.seq.len - t * kKeys), end = (left + 15) / 16 * 16;
          uint8_t* v0 = sv + st * C::kTile;
          // a thread has chunk c of every kApart-th key, four at a time
          constexpr int kApart = 128 / (D / 8);
          const int c = threadIdx.x % (D / 8), first = max(0, ctx - t * kKeys) / kApart * kApart;
          uint8_t* at0 = v0 + (c >> 3) * C::kHalf + (c & 7) * 16;
          for (int key0 = first + (threadIdx.x & 127) / (D / 8); key0 < end; key0 += 4 * kApart) {
            uint4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = *reinterpret_cast<const uint4*>(at0 + min(key0 + k * kApart, kKeys - 1) * 128);
            bool odd = key0 + 3 * kApart >= left;
#pragma unroll
            for (int k = 0; k < 4; ++k) odd |= draft::has_bad<bf16>(v[k]);
            if (!odd) continue;
            for (int key = key0; key < min(end, key0 + 4 * kApart); key += kApart) {
              uint8_t* at = at0 + key * 128;
              if (key >= left) {
                *reinterpret_cast<uint4*>(at) = make_uint4(0, 0, 0, 0);
              } else if (t * kKeys + key >= ctx && draft::clear_bad<bf16>(at)) {
                const int k = (t - ctx / kKeys) * kKeys + key;
                atomicOr(&bad[k >> 5], 1u << (k & 31));
                bad[kSpecial * 4] = 1;
              }
            }
          }
          fence_async_shared();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (special || !live) mbar_arrive(&ctl->p_full[g][0]);
          mbar_arrive(&ctl->p_full[g][1]);
        }
      }
      if (!ok) break;
      // ---- the segment's output: complete with its last P V
      const uint32_t steps = (uint32_t)(t_hi - t_lo) * tiles, mine = s - 2;
      const uint32_t other = s0 + steps - 1 == mine ? mine - 1 : mine + 1;
      const bool some = t_first < t_hi, join = tiles == 1 && steps > 1;
      // its own last P V first: the other stream's then has no phase but its last to wait for.
      // A P V of this segment was issued when all eight warps had left the one before (o_free).  A stream without a
      // step here (an item of one tile) waits for that itself, so that no warp is more than a segment ahead of
      // another: else it arrives twice in one phase of o_free, and O, the marks in `bad` or the streams' sums change
      // under the warps that are still behind.
      if (some) ok = wait(&ctl->pv_done[g], (mine >> 1) & 1, abort, a.status);
      else if (segs > 0) ok = wait(&ctl->o_free, (segs - 1) & 1, abort, a.status);
      if (ok && join) ok = wait(&ctl->pv_done[g ^ 1], (other >> 1) & 1, abort, a.status);
      if (!ok) break;
      tc_fence_after();
      if (live && some) {
        float f = 1.f, f_other = 0.f;               // of this stream's sums, and of the other's
        if (join) {
          ctl->word[g][row] = make_float2(m, l);
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->pair[quad]);
          ok = wait(&ctl->pair[quad], told & 1, abort, a.status);
          if (!ok) break;
          ++told;
          const float2 o = ctl->word[g ^ 1][row];
          const float mm = fmaxf(m, o.x), base = mm == -INFINITY ? 0.f : mm;
          f = ex2_approx(m - base);
          f_other = ex2_approx(o.x - base);
          const float own = l * f, others = o.y * f_other;
          l = own + others;
          m = mm;
        }
        const bool whole = w.begins && w.ends, odd = bad[kSpecial * 4] != 0;
        const int h = it.kvh * a.G + row - tok * a.heads;
        const int64_t tt = (int64_t)w.seq.first + i;
        const int64_t slot =
            (2 * (int64_t)blockIdx.x + (w.begins ? 1 : 0)) * kPartRows + (i - it.i0 - tok) * a.heads + row;
        const bool any = valid && mask.sees_any(a, w.seq);
        const float inv = any ? 1.f / l : 0.f;
        // joined, the streams' threads of a row share its columns
        const int c_lo = join ? e * (D / 2) : 0, c_hi = join ? c_lo + D / 2 : D;
#pragma unroll 1
        for (int c = c_lo; c < c_hi; c += 32) {
          float ov[32];
          __syncwarp();
          tmem_ld32_sync(lanes + kColO + g * D + c, ov);
          if (join) {
            float x[32];
            tmem_ld32_sync(lanes + kColO + (g ^ 1) * D + c, x);
#pragma unroll
            for (int y = 0; y < 32; ++y) ov[y] = ov[y] * f + x[y] * f_other;
          }
          if (valid && odd) add_bad(a, w, it, i, bad, p.v, c, D, ov);
          if (valid && whole) {
            uint4* to = reinterpret_cast<uint4*>(static_cast<bf16*>(p.o) + (tt * a.H + h) * D + c);
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
            float4* to = reinterpret_cast<float4*>(part.o + slot * D + c);
#pragma unroll
            for (int u = 0; u < 8; ++u) to[u] = make_float4(ov[4 * u], ov[4 * u + 1], ov[4 * u + 2], ov[4 * u + 3]);
          }
        }
        if (valid && (!join || e == 0)) {
          if (!whole) *reinterpret_cast<float2*>(part.ml + slot * 2) = make_float2(m, l);
          else if (p.lse) p.lse[(int64_t)h * a.T + tt] = draft::row_lse(m, l, any);
        }
      }
      // of the segment before, which nobody is in any more; none is in the segment after the next, whose they will be
      if (threadIdx.x == 0)
        for (int k = 0; k <= kSpecial * 4; ++k) ctl->bad[(segs + 2) % 3][k] = 0;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->o_free);
      if (w.begins && !w.ends)
        open = make_int4(w.seg_b, w.seg_item, w.seg_items, w.parts(plan, blockIdx.x));
      s0 += steps;
      tile0 += (uint32_t)(t_hi - t_lo);
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
  r.box = kKeys;
  while (p.pool.page_size % r.box) r.box >>= 1;
  r.page_shift = -1;
  for (int k = 0; k <= 16; ++k)
    if (p.pool.page_size == 1 << k) r.page_shift = k;
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
  if (e != cudaSuccess) return e;
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
