// Attention of drafted tokens over a paged cache, any page size, head width
// 32, 64 or 128, bf16 and fp32: the general kernel.
//
// Work, split and partial results as draft_plan.cuh says.  An item has up to
// 64 rows (tokens times query heads of one key head); a tile is 64 keys, whose
// rows are fetched one by one through the block table with cp.async, a tile
// ahead.  Each row keeps a running maximum, sum and output:
//   S = Q K^T,  m' = max(m, scale S),  P = 2^(scale S - m'),
//   l = l 2^(m - m') + sum P,  O = O 2^(m - m') + P V
// with the scores that a row does not see at -infinity.  bf16: matrix products
// of 16 rows a warp, P as the sum of two bf16 (one would be off by 2^-8 of P,
// which shows in the output).  fp32: packed multiply-adds, 4 x 4 scores and 4
// x D / 16 outputs to a thread; with 32 rows or fewer, groups of threads take
// a half or a quarter of a tile's keys each and merge their results at the end.
// Barriers around each tile's fetch leave 27% of the issue slots busy.  fp32, 13
// contexts of 5,120 keys, 24 rows to a key head, d = 64: 154 us; a page's place is
// looked up two tiles ahead, masks before the scores (13 ragged contexts of up to
// 5,000: 36.5 -> 33 us).
//
// A value that is not finite may stand at a key that only some of the rows
// see, and 0 times it is not 0; such values are taken out of the tile and
// added to the rows that do see them (only where new tokens are: older keys
// are seen by all).
#include "draft_plan.cuh"
#include "draft_worker.cuh"

namespace nt {
namespace {

using namespace draft;

constexpr int kKeys = 64;

// kGroups: groups of threads with 64 / kGroups rows and as many keys of a tile each
template <typename T, int D, int kGroups>
struct Cfg {
  static constexpr int kRows = 64 / kGroups;
  static constexpr bool kBf16 = sizeof(T) == 2;
  static constexpr int kThreads = kBf16 ? 128 : 256;
  static constexpr uint32_t kRow = D * sizeof(T);
  static constexpr uint32_t kSide = kKeys * kRow;
  static constexpr uint32_t kScratch = kBf16 ? 0 : kRows * kRow + 64 * (kKeys / kGroups + 4) * 4;   // queries, probabilities
  static constexpr uint32_t kSmem = 4 * kSide + kScratch;
  static_assert(kGroups == 1 || (64 * D + 128) * 4 <= 4 * kSide, "results to merge");
  static constexpr int kPerSm = kSmem <= 110 * 1024 ? 2 : 1;       // CTAs
};

struct RowsArgs {
  DraftBatch a;
  const void* q;
  int64_t q_stride;
  const void* k;
  const void* v;
  void* o;
  float* lse;
  void* workspace;
  float scale_log2;
};

struct Shared {
  DraftPlanSums plan;
  int64_t off[3][kKeys];       // byte offsets in the pool of a tile's rows, -1 none
  unsigned long long bad;      // keys of the tile with values that are not finite
};

template <typename T, int D, int kGroups>
__global__ void __launch_bounds__((Cfg<T, D, kGroups>::kThreads), (Cfg<T, D, kGroups>::kPerSm))
    draft_rows_kernel(const RowsArgs p) {
  using C = Cfg<T, D, kGroups>;
  using W = Rows<T, D, kGroups>;
  constexpr int kRows = C::kRows;
  constexpr int kThreads = C::kThreads, kChunks = D * (int)sizeof(T) / 16;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Shared sh;
  const DraftBatch& a = p.a;
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  const DraftPlan plan = draft_plan(a, kKeys, 1, blockIdx.x, gridDim.x, &sh.plan, kThreads);
  DraftWalk w;
  w.init(a, plan, kKeys, 1);
  const DraftPartials part = draft_partials(p.workspace, gridDim.x, kRows);
  int4 open = make_int4(-1, 0, 0, 0);
  const int64_t head_bytes = (int64_t)a.page_size * C::kRow;
  W me(smem + 4 * C::kSide);

  while (w.next(a, kKeys, 1)) {
    const DraftItem& it = w.it;
    auto rows_of = [&](int t, int64_t* offs) {     // offsets of tile t's rows
      if (tid < kKeys) {
        const uint32_t x = (uint32_t)t * kKeys + tid;
        int64_t off = -1;
        if (x < (uint32_t)w.seq.len) {
          const uint32_t pg = x / (uint32_t)a.page_size;
          const int id = a.table[(int64_t)w.seg_b * a.max_pages + pg];
          if ((unsigned)id < (unsigned)a.n_pages)
            off = ((int64_t)id * a.Hkv + it.kvh) * head_bytes + (int64_t)(x - pg * a.page_size) * C::kRow;
          else
            flag_device(a.status, kDevCheck);
        }
        offs[tid] = off;
      }
    };
    auto fetch = [&](int t, const int64_t* offs) {
      uint8_t* st = smem + (t & 1) * 2 * C::kSide;
      for (int e = tid; e < 2 * kKeys * kChunks; e += kThreads) {
        const int side = e / (kKeys * kChunks), r = e / kChunks % kKeys, c = e % kChunks;
        const int64_t off = offs[r];
        uint8_t* to = st + side * C::kSide + swizzled<C::kRow>(r, c);
        if (off >= 0) cp_async16(to, static_cast<const uint8_t*>(side ? p.v : p.k) + off + c * 16);
        else *reinterpret_cast<uint4*>(to) = make_uint4(0, 0, 0, 0);
      }
      cp_async_commit();
    };
    __syncthreads();
    // a tile's offsets are looked up while the tile before the one before it is worked on
    int64_t *off = sh.off[0], *off1 = sh.off[1], *off2 = sh.off[2];
    rows_of(w.t0, off);
    rows_of(w.t0 + 1, off1);
    me.load_q(static_cast<const T*>(p.q), p.q_stride, w.seq.first + it.i0, it.kvh * a.G + it.h0, it.ni, it.nh);
    __syncthreads();
    fetch(w.t0, off);
    for (int t = w.t0; t < w.t1; ++t) {
      if (tid == 0) sh.bad = 0;
      if (t + 1 < w.t1) fetch(t + 1, off1);
      else cp_async_commit();
      if (t + 2 < w.t1) rows_of(t + 2, off2);
      cp_async_wait1();
      __syncthreads();
      uint8_t* st = smem + (t & 1) * 2 * C::kSide;
      const int64_t x0 = (int64_t)t * kKeys;
      const int ctx = w.seq.len - w.seq.n;
      const bool all = x0 + kKeys <= ctx;          // every row sees every key
      if (!all) {
        for (int e = tid; e < kKeys * kChunks; e += kThreads)
          if (clear_bad<T>(st + C::kSide + swizzled<C::kRow>(e / kChunks, e % kChunks)))
            atomicOr(&sh.bad, 1ull << (e / kChunks));
        __syncthreads();
      }
      me.tile(a, w.seq, it, st, st + C::kSide, x0, all, p.scale_log2);
      if (!all && sh.bad) {
        const uint64_t bad = sh.bad;
        me.add_bad(a, w.seq, it, x0, bad, static_cast<const uint8_t*>(p.v), off);
      }
      __syncthreads();
      int64_t* o3 = off;
      off = off1;
      off1 = off2;
      off2 = o3;
    }
    cp_async_wait0();
    me.merge(reinterpret_cast<float*>(smem));
    const bool whole = w.begins && w.ends;
    if (whole) {
      me.store(a, w.seq, it, static_cast<T*>(p.o), p.lse);
    } else {
      const int64_t slot = 2 * (int64_t)blockIdx.x + (w.begins ? 1 : 0);
      me.store_part(part.ml + slot * kRows * 2, part.o + slot * kRows * D);
    }
    if (w.begins && !w.ends)
      open = make_int4(w.seg_b, w.seg_item, w.seg_items, w.parts(plan, 1, blockIdx.x));
  }
  if (tid == 0) part.open[blockIdx.x] = open;
}

template <typename T, int D, int kGroups = 1>
cudaError_t run(const DraftProblem& p, unsigned int* status, cudaStream_t s) {
  using C = Cfg<T, D, kGroups>;
  RowsArgs r = {};
  r.a = draft_batch(p, C::kRows, 1, status);
  r.q = p.q;
  r.q_stride = p.q_stride;
  r.k = p.pool.k;
  r.v = p.pool.v;
  r.o = p.o;
  r.lse = p.lse;
  r.workspace = p.workspace;
  r.scale_log2 = p.scale * 1.4426950408889634f;
  const int ctas = min(C::kPerSm * sm_count(), kPagedMaxCtas);
  cudaError_t e = allow_smem_once<draft_rows_kernel<T, D, kGroups>>(C::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(draft_rows_kernel<T, D, kGroups>, dim3(ctas), dim3(C::kThreads), C::kSmem, s, r);
  if (e != cudaSuccess) return e;
  return launch_draft_join(C::kBf16 ? NT_BF16 : NT_F32, r.a, D, ctas, C::kRows, p.workspace, p.o, p.lse, s);
}

template <int D>
cudaError_t run_f32(const DraftProblem& p, unsigned int* status, cudaStream_t s) {
  const int64_t rows = (int64_t)p.max_new * (p.H / p.pool.H);
  if (rows <= 16) return run<float, D, 4>(p, status, s);
  return rows <= 32 ? run<float, D, 2>(p, status, s) : run<float, D>(p, status, s);
}

}  // namespace

cudaError_t launch_draft_rows(nt_dtype dt, const DraftProblem& p, unsigned int* status, cudaStream_t s) {
  if (dt == NT_BF16) {
    if (p.d == 32) return run<bf16, 32>(p, status, s);
    return p.d == 64 ? run<bf16, 64>(p, status, s) : run<bf16, 128>(p, status, s);
  }
  if (p.d == 32) return run_f32<32>(p, status, s);
  return p.d == 64 ? run_f32<64>(p, status, s) : run_f32<128>(p, status, s);
}

}  // namespace nt
