// Attention of drafted tokens over a paged cache, any page size, head width
// 32, 64 or 128, bf16 and fp32: the general kernel.
//
// Work, split and partial results as draft_plan.cuh says.  An item has up to
// 64 rows (tokens times query heads of one key head); a tile is 64 keys, whose
// rows are fetched one by one through the block table with cp.async, a tile
// ahead; their pages are looked up two tiles ahead.  Each row keeps a running
// maximum, sum and output:
//   S = Q K^T,  m' = max(m, scale S),  P = 2^(scale S - m'),
//   l = l 2^(m - m') + sum P,  O = O 2^(m - m') + P V
// with the scores that a row does not see at -infinity.  bf16: matrix products
// of 16 rows a warp, P as the sum of two bf16 (one would be off by 2^-8 of P,
// which shows in the output).  fp32: products of tf32 parts (draft_worker.cuh);
// warps have 16 of 64, 32 or 16 rows and a half, a quarter or an eighth of a
// tile's keys, and merge their results at the end.
//
// fp32, d = 64, 13 contexts of 5,120 keys, 24 rows to a key head: 123 us; packed
// multiply-adds took 154 (three shared-memory cycles to each four multiply-adds of a
// scheduler), most of the rest are the matrix instructions (32 x 64 x 64 x 2 of them three
// times are 1,570 of a tile's 3,800 cycles).  bf16, d = 128, 152 contexts of 8,000, 64
// rows: 203 us.  Whole rows by bulk copies were slower (a warp issues one every 100
// cycles: bf16, d = 64, 110 us -> 161).
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
  static constexpr uint32_t kSide = kKeys * (kRow + 16);
  static constexpr uint32_t kScratch = kBf16 ? 0 : 2 * kRows * kRow;        // two parts of the queries
  static constexpr uint32_t kSmem = 4 * kSide + kScratch;
  static_assert(kBf16 || (128 * D + 256) * 4 <= 4 * kSide, "results to merge");
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
  int64_t off[2][kKeys];       // places in the pool of a tile's rows (of the next one's), -1 none
  unsigned long long bad[2];   // keys of the tile (of the next one) with values that are not finite
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
  // The first 64 threads have a key of each tile: its page is looked up two tiles ahead, its place stored one ahead.
  auto page_of = [&](int t) {                      // (used by place(), so that nothing waits for it here)
    const uint32_t x = (uint32_t)t * kKeys + tid;
    return tid < kKeys && x < (uint32_t)w.seq.len
               ? a.table[(int64_t)w.seg_b * a.max_pages + x / (uint32_t)a.page_size] : 0;
  };
  auto place = [&](int t, int id) {
    if (tid >= kKeys) return;
    const uint32_t x = (uint32_t)t * kKeys + tid;
    int64_t off = -1;
    if (x < (uint32_t)w.seq.len) {
      if ((unsigned)id < (unsigned)a.n_pages)
        off = ((int64_t)id * a.Hkv + w.it.kvh) * head_bytes + (int64_t)(x % (uint32_t)a.page_size) * C::kRow;
      else
        flag_device(a.status, kDevCheck);
    }
    sh.off[t & 1][tid] = off;
  };
  // A thread has the same chunk of some rows, keys and values.
  constexpr int kStep = kThreads / kChunks, kRowsEach = kKeys / kStep;
  static_assert(kThreads % kChunks == 0 && kKeys % kStep == 0, "chunks of a thread");
  const int my_row = tid / kChunks, chunk = tid % kChunks;
  const uint32_t my_place = padded<C::kRow>(my_row, chunk);
  auto fetch = [&](int t) {
    const uint32_t to = smem_u32(smem) + (t & 1) * 2 * C::kSide + my_place;
    int64_t off[kRowsEach];
#pragma unroll
    for (int k = 0; k < kRowsEach; ++k) off[k] = sh.off[t & 1][my_row + k * kStep];
#pragma unroll
    for (int k = 0; k < kRowsEach; ++k) {
      const bool there = off[k] >= 0;
      const int64_t at = there ? off[k] + chunk * 16 : 0;
      cp_async16(to + k * kStep * (C::kRow + 16), static_cast<const uint8_t*>(p.k) + at, there);
      cp_async16(to + k * kStep * (C::kRow + 16) + C::kSide, static_cast<const uint8_t*>(p.v) + at, there);
    }
    cp_async_commit();
  };
  while (w.next(a, kKeys, 1)) {
    __syncthreads();
    if (tid < 2) sh.bad[tid] = 0;
    const int first = page_of(w.t0), second = page_of(w.t0 + 1);
    place(w.t0, first);
    place(w.t0 + 1, second);
    me.load_q(static_cast<const T*>(p.q), p.q_stride, w.seq.first + w.it.i0, w.it.kvh * a.G + w.it.h0, w.it.ni,
              w.it.nh);
    __syncthreads();
    fetch(w.t0);
    for (int t = w.t0; t < w.t1; ++t) {
      if (t + 1 < w.t1) fetch(t + 1);
      else cp_async_commit();
      const int ahead = page_of(t + 2);
      cp_async_wait1();
      uint8_t* st = smem + (t & 1) * 2 * C::kSide;
      const int64_t x0 = (int64_t)t * kKeys;
      const bool all = x0 + kKeys <= w.seq.len - w.seq.n;        // every row sees every key
      unsigned long long* bad = &sh.bad[t & 1];
      if (!C::kBf16 || !all) {                     // in the chunks that this thread has fetched
        uint8_t* mine = st + C::kSide + my_place;
        uint4 v[kRowsEach];
        bool any = false;
#pragma unroll
        for (int k = 0; k < kRowsEach; ++k) v[k] = *reinterpret_cast<const uint4*>(mine + k * kStep * (C::kRow + 16));
#pragma unroll
        for (int k = 0; k < kRowsEach; ++k) any |= has_bad<T>(v[k]);
        if (any) {
          for (int k = 0; k < kRowsEach; ++k)
            if (clear_bad<T>(mine + k * kStep * (C::kRow + 16))) atomicOr(bad, 1ull << (my_row + k * kStep));
        }
      }
      __syncthreads();
      if (tid == 0) sh.bad[(t & 1) ^ 1] = 0;
      me.tile(a, w.seq, w.it, st, st + C::kSide, x0, all, p.scale_log2);
      if (*bad) {
        me.add_bad(a, w.seq, w.it, x0, *bad, static_cast<const uint8_t*>(p.v), sh.off[t & 1]);
        __syncthreads();
      }
      place(t + 2, ahead);
      __syncthreads();
    }
    cp_async_wait0();
    me.merge(reinterpret_cast<float*>(smem));
    if (w.begins && w.ends) {
      me.store(a, w.seq, w.it, static_cast<T*>(p.o), p.lse);
    } else {
      const int64_t slot = 2 * (int64_t)blockIdx.x + (w.begins ? 1 : 0);
      me.store_part(part.ml + slot * kRows * 2, part.o + slot * kRows * D);
    }
    if (w.begins && !w.ends)
      open = make_int4(w.seg_b, w.seg_item, w.seg_items, w.parts(plan, blockIdx.x));
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
