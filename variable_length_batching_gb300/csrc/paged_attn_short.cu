// Attention of one new token per sequence over many short paged contexts: one
// warp per item (a sequence's key head with up to HP of its query heads).
//
// With block tables of a few pages there is nothing to split and little to
// stream; what an item costs is the chain length -> pages -> keys -> scores ->
// output, and the tile kernel's hand-offs between warps (about 1.3 us an
// item, one item at a time on an SM).  Here a warp does all of it, with no
// barrier, and an SM has a dozen items in hand: 200 contexts of up to 4 keys
// with 16 query heads to each of 12 key heads take 10.1 us instead of 33.6.
// The warp copies the rows of its
// next slices of 16 keys (of the next items, when this one's end) into its own
// ring with cp.async, row by row, so any page size will do; layout and
// arithmetic are paged_worker.cuh's.
#include "paged_plan.cuh"
#include "paged_worker.cuh"

namespace nt {
namespace {

using namespace paged;

template <typename T, int D, int HP>
struct Cfg {
  static constexpr bool kBf16 = sizeof(T) == 2;
  static constexpr uint32_t kRow = D * sizeof(T);
  static constexpr uint32_t kSide = 16 * kRow;                     // keys or values of a slice
  static constexpr uint32_t kSlot = 2 * kSide;
  static constexpr uint32_t kOut = HP * kRow;                      // bf16: the output's rows; fp32: the query's
  static constexpr uint32_t kScratch = Worker<T, D, HP>::kScratch;
  // few slots, many warps: 12 to 24 on an SM (6 in fp32 with d = 128)
  static constexpr int kSlots = D == 128 || (!kBf16 && D == 64) ? 2 : 3;
  static constexpr int kWarps = !kBf16 && D == 128 ? 6 : 4;
  static constexpr uint32_t kWarpBytes = (kSlots * kSlot + kOut + kScratch + 127) / 128 * 128;
  static constexpr uint32_t kSmem = kWarps * kWarpBytes;
  static constexpr int kPerSm = (int)(225 * 1024 / (kSmem + 1024)) < 6 ? (int)(225 * 1024 / (kSmem + 1024)) : 6;
  static_assert(kWarpBytes % 128 == 0 && kPerSm >= 1 && kSmem <= 227 * 1024, "shared memory");
};

struct ShortArgs {
  const void* q;
  int64_t q_stride;
  const void* k;
  const void* v;
  const int32_t* table;
  const int32_t* lengths;
  void* o;
  float* lse;
  int B, H, G, Hkv, max_pages, page_size, n_pages, items, hgroups;
  float scale_log2;
  unsigned int* status;
};

template <typename T, int D, int HP>
__global__ void __launch_bounds__((Cfg<T, D, HP>::kWarps * 32)) paged_attn_short_kernel(const ShortArgs a) {
  using C = Cfg<T, D, HP>;
  constexpr int kWarps = C::kWarps;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = smem + warp * C::kWarpBytes;
  T* out_rows = reinterpret_cast<T*>(ring + C::kSlots * C::kSlot);
  const int64_t cap = min64((int64_t)a.max_pages * a.page_size, 0x7fffffff);
  const int64_t total = (int64_t)a.B * a.items;
  const int64_t step = (int64_t)gridDim.x * kWarps;
  pdl_wait();
  pdl_trigger();

  // ---- the copies' place: item, its slice, a window of its table ---------------
  int64_t next = (int64_t)blockIdx.x * kWarps + warp;      // the item in hand for copying
  int len = next < total ? paged_length(a.lengths, (int)paged_div(next, a.items), cap, a.status) : 0;
  int len_after = next + step < total ? paged_length(a.lengths, (int)paged_div(next + step, a.items), cap, a.status) : 0;
  // the first 32 entries of a sequence's table row (some may be behind its end, and unused)
  auto window = [&](int64_t item) {
    return item < total && lane < a.max_pages
               ? a.table[paged_div(item, a.items) * a.max_pages + lane] : -1;
  };
  int kb = 0, win = 0, ids = window(next), ids_after = window(next + step);
  auto copy = [&](int slot) {
    while (next < total && kb >= len) {            // the next item with a key
      next += step;
      len = len_after;
      len_after = next + step < total ? paged_length(a.lengths, (int)paged_div(next + step, a.items), cap, a.status) : 0;
      kb = 0;
      win = 0;
      ids = ids_after;
      ids_after = window(next + step);
    }
    if (next < total) {
      const int b = (int)paged_div(next, a.items), kvh = (int)(next - (int64_t)b * a.items) / a.hgroups;
      const int ps = a.page_size, first = kb / ps, last = min(kb + 15, len - 1) / ps;
      if (last >= win + 32) {
        win = first;
        const int64_t i = (int64_t)win + lane;
        ids = i * ps < len ? a.table[(int64_t)b * a.max_pages + i] : -1;
      }
      // lanes 0..15: the row of key kb + lane
      const int key = kb + (lane & 15), pg = key / ps;
      const int id = __shfl_sync(0xffffffffu, ids, (pg - win) & 31);
      const bool in = key < len, good = id >= 0 && id < a.n_pages;
      if (in && !good) flag_device(a.status, kDevCheck);
      const int64_t row = in && good ? ((int64_t)id * a.Hkv + kvh) * ps + (key - pg * ps) : -1;
      copy_slice<T, D>(smem_u32(ring + slot * C::kSlot), a.k, a.v, row);
      kb += 16;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int s = 0; s < C::kSlots; ++s) copy(s);

  // ---- the items ------------------------------------------------------------------
  Worker<T, D, HP> me(16, 0, ring + C::kSlots * C::kSlot + C::kOut);
  int slot = 0;
  for (int64_t item = (int64_t)blockIdx.x * kWarps + warp; item < total; item += step) {
    const int b = (int)paged_div(item, a.items), j = (int)(item - (int64_t)b * a.items);
    const int n = paged_length(a.lengths, b, cap, nullptr);
    const int h0 = j % a.hgroups * HP, nh = min(HP, a.G - h0);
    const int64_t hq = (int64_t)(j / a.hgroups) * a.G + h0;      // the first query head
    T* o = static_cast<T*>(a.o) + ((int64_t)b * a.H + hq) * D;
    if (n == 0) {
      for (int e = lane; e < nh * D; e += 32) o[e] = from_f32<T>(0.f);
      if (a.lse && lane < nh) a.lse[(hq + lane) * a.B + b] = -INFINITY;
      continue;
    }
    const T* q = static_cast<const T*>(a.q) + b * a.q_stride + hq * D;
    if constexpr (Worker<T, D, HP>::kKeepsQ) {
      for (int e = lane; e < nh * (D / 4); e += 32)
        reinterpret_cast<float4*>(out_rows)[e] = reinterpret_cast<const float4*>(q)[e];
      __syncwarp();
      q = out_rows;
    }
    me.load_q(q, nh);
    for (int k0 = 0; k0 < n; k0 += 16) {
      asm volatile("cp.async.wait_group %0;" ::"n"(C::kSlots - 1) : "memory");
      __syncwarp();
      me.tile(ring + slot * C::kSlot, C::kSide, min(16, n - k0), a.scale_log2);
      __syncwarp();
      copy(slot);
      slot = slot + 1 == C::kSlots ? 0 : slot + 1;
    }
    me.finish(out_rows, o, nh);
    if (a.lse) me.store_lse(a.lse + hq * a.B + b, a.B, nh);
  }
}

template <typename T, int D, int HP>
cudaError_t run(const PagedAttnProblem& p, unsigned int* status, cudaStream_t s) {
  using C = Cfg<T, D, HP>;
  ShortArgs a;
  a.q = p.q;
  a.q_stride = p.q_stride;
  a.k = p.pool.k;
  a.v = p.pool.v;
  a.table = p.table;
  a.lengths = p.lengths;
  a.o = p.o;
  a.lse = p.lse;
  a.B = p.B;
  a.H = p.H;
  a.G = p.H / p.pool.H;
  a.Hkv = p.pool.H;
  a.max_pages = p.max_pages;
  a.page_size = p.pool.page_size;
  a.n_pages = p.pool.n_pages;
  a.hgroups = (a.G + HP - 1) / HP;
  a.items = a.Hkv * a.hgroups;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  a.status = status;
  const cudaError_t e = allow_smem_once<paged_attn_short_kernel<T, D, HP>>(C::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t items = (int64_t)p.B * a.items;
  const int grid = (int)min64((items + C::kWarps - 1) / C::kWarps, (int64_t)sm_count() * C::kPerSm);
  return launch_pdl(paged_attn_short_kernel<T, D, HP>, dim3(grid), dim3(C::kWarps * 32), C::kSmem, s, a);
}

template <int D>
cudaError_t run_d(nt_dtype dt, const PagedAttnProblem& p, unsigned int* status, cudaStream_t s) {
  const int G = p.H / p.pool.H;
  if (dt == NT_BF16) return G <= 8 ? run<bf16, D, 8>(p, status, s) : run<bf16, D, 16>(p, status, s);
  if (G == 1) return run<float, D, 1>(p, status, s);
  if (G == 2) return run<float, D, 2>(p, status, s);
  if (G <= 4) return run<float, D, 4>(p, status, s);
  return run<float, D, 8>(p, status, s);
}

}  // namespace

// About 1 us, 1.6 us an item and t a slice of 16 keys, more when all warps are
// busy; as long as the longest item, or as the warps' shares.  (200 contexts
// with 12 heads of 64, of up to 200 keys: 19 us here, 24 on the tile kernel;
// of up to 1,000: 73 and 55.)
double paged_attn_short_us(nt_dtype dt, const PagedAttnProblem& p) {
  const int64_t cap = paged_cap(p);
  if (cap > kPagedShortKeys || p.pool.n_pages == 0) return INFINITY;
  const int G = p.H / p.pool.H, HP = dt == NT_BF16 && G > 8 ? 16 : 8;
  const double rounds = (double)paged_items(p, HP) / (double)(sm_count() * (dt == NT_BF16 || p.d < 128 ? 12 : 6));
  const double t = (dt == NT_F32 ? (p.d == 128 ? 1.65 : 0.9) : HP == 16 ? 0.95 : 0.85) +
                   (p.d == 128 && (HP == 16 || dt == NT_F32) ? 1.0 : 0.5) * fmin(1, rounds);
  const double keys = (double)((cap + 15) / 16) * t;
  const double bytes = (double)p.B * p.pool.H * cap * p.d * 2 * (dt == NT_BF16 ? 2 : 4) * paged_mean_part(p);
  return fmax(1.0 + fmax(1.6 + keys, rounds * (1.6 + keys * paged_mean_part(p))), 3.8 + bytes / 6.1e6);
}

cudaError_t launch_paged_attn_short(nt_dtype dt, const PagedAttnProblem& p, unsigned int* status, cudaStream_t s) {
  if (p.d == 32) return run_d<32>(dt, p, status, s);
  if (p.d == 64) return run_d<64>(dt, p, status, s);
  return run_d<128>(dt, p, status, s);
}

}  // namespace nt
