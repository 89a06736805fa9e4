// Attention of drafted tokens over a paged cache, a cluster of CTAs per item (a
// key head and up to 16 rows, tokens times query heads; 8 in fp32): where there
// is little to read, for any page size and type.
//
// As for one new token per sequence (paged_attn_spread.cu), a small call waits
// for latencies, and nothing else is left here: no plan, no second launch.  The
// CTAs' warps take the item's slices of 16 keys in turn, each from its own ring
// of slots filled row by row with cp.async; the warps' results are merged in
// the CTA, and the CTAs' through distributed shared memory.  A sequence has as
// many items as max_new may need; clusters whose tokens are not there leave at
// once.  One context of 777 keys, eight tokens and 12 heads of 64: 6.2 us, 9.7
// to 11.5 on the kernels that deal tiles out.
#include <atomic>
#include <type_traits>

#include "draft_plan.cuh"
#include "draft_worker.cuh"

namespace nt {
namespace {

using namespace draft;

constexpr int kMaxCluster = kPagedMaxCluster;
constexpr int64_t kMaxClusters = 1 << 24;    // of a launch

template <typename T, int D>
struct Cfg {
  static constexpr bool kBf16 = sizeof(T) == 2;
  static constexpr int kRows = kBf16 ? 16 : 8;
  static constexpr uint32_t kRow = D * sizeof(T), kSide = 16 * kRow;
  static constexpr uint32_t kSlot = 2 * kSide;                     // keys and values of a slice
  // half an SM's shared memory at most: two CTAs on each, so that clusters are twice as many
  static constexpr int kWarps = kRow <= 128 ? 8 : kRow == 256 ? 6 : 3;
  static constexpr int kSlots = kRow <= 128 ? 3 : 2;
  static constexpr uint32_t kWarpBytes = kSlots * kSlot;
  static constexpr uint32_t kPart = kRows * D * 4;                 // the CTA's output; before, fp32: its query rows
  static constexpr uint32_t kScratch = kBf16 ? 0 : Worker<float, D, 8>::kScratch;      // of a warp
  static constexpr uint32_t kSmem = kWarps * (kWarpBytes + kScratch) + kPart;
  static constexpr int kRedStride = D + 4;
  static_assert(kRows * kRedStride * 4 <= kWarpBytes && kSmem <= 111 * 1024, "shared memory");
};

struct SpreadArgs {
  DraftBatch a;
  const void* q;
  int64_t q_stride;
  const uint8_t* k;
  const uint8_t* v;
  void* o;
  float* lse;
  int cluster, items;                      // of a sequence, at most
  float scale_log2;
};

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// the same place in CTA `rank`'s shared memory
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float2 cluster_load2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// A running maximum (base 2), sum and four outputs, joined with another's.
// sum -1: nothing in it.
struct Sum {
  float m = -INFINITY, l = -1.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
};
template <int N>
__device__ __forceinline__ Sum join_sums(const float2 (&ml)[N], const float4 (&v)[N]) {
  Sum s;
  bool any = false;
#pragma unroll
  for (int x = 0; x < N; ++x) {
    if (ml[x].y != -1.f) any = true;
    s.m = fmaxf(s.m, ml[x].x);
  }
  if (!any) return s;
  s.l = 0.f;
  const float base = s.m == -INFINITY ? 0.f : s.m;
#pragma unroll
  for (int x = 0; x < N; ++x) {
    if (ml[x].y == -1.f) continue;
    const float f = ex2_approx(ml[x].x - base);
    s.l += f * ml[x].y;
    s.o.x += f * v[x].x;
    s.o.y += f * v[x].y;
    s.o.z += f * v[x].z;
    s.o.w += f * v[x].w;
  }
  return s;
}

// What a warp does with a slice, for both types.
template <typename T, int D>
struct Unit;
template <int D>
struct Unit<bf16, D> : Slice<D, Cfg<bf16, D>::kSide> {
  using Base = Slice<D, Cfg<bf16, D>::kSide>;
  __device__ __forceinline__ explicit Unit(void*) : Base(16) {}
  __device__ __forceinline__ int row(int r) const { return this->g + 8 * r; }       // the lane's rows
  __device__ __forceinline__ void slice(uint8_t* slot, int left, bool all, const uint32_t (&see)[2], float scale_log2) {
    this->tile(smem_u32(slot), 0, all, see, scale_log2);
  }
};
template <int D>
struct Unit<float, D> : Worker<float, D, 8> {
  using Base = Worker<float, D, 8>;
  __device__ __forceinline__ explicit Unit(void* scratch) : Base(16, 0, scratch) {}
  __device__ __forceinline__ int row(int r) const { return 2 * r + this->half; }
  __device__ __forceinline__ void slice(uint8_t* slot, int left, bool all, const uint32_t (&see)[4], float scale_log2) {
    if (all) this->tile(slot, Cfg<float, D>::kSide, 16, scale_log2);
    else this->template tile<true>(slot, Cfg<float, D>::kSide, left, scale_log2, see);
  }
  // As Slice::clean.
  __device__ __forceinline__ uint32_t clean(uint8_t* slot, int, int left) const {
    uint32_t found = 0;
    for (int e = threadIdx.x & 31; e < 16 * (D / 4); e += 32) {
      const int key = e / (D / 4), ch = e % (D / 4);
      if (key < left && clear_bad<float>(slot + Cfg<float, D>::kSide + (ch >> 3) * 2048 + key * 128 + (ch & 7) * 16))
        found |= 1u << key;
    }
    __syncwarp();
    return __reduce_or_sync(0xffffffffu, found);
  }
};

template <typename T, int D>
__global__ void __launch_bounds__((Cfg<T, D>::kWarps * 32), 2) draft_spread_kernel(const SpreadArgs p) {
  using C = Cfg<T, D>;
  constexpr int kWarps = C::kWarps, kCols = D / 4, kMine = C::kBf16 ? 2 : 4;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ float rm[kWarps][16], rl[kWarps][16];
  __shared__ float2 part_ml[C::kRows];                      // the CTA's maxima and sums
  __shared__ unsigned int bad[kBadWords + 1];               // keys of its slices with values taken out, and whether any
  const DraftBatch& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = smem + warp * C::kWarpBytes;
  float* part_o = reinterpret_cast<float*>(smem + kWarps * C::kWarpBytes);
  const uint32_t rank = blockIdx.x % p.cluster;
  const int64_t total = (int64_t)a.B * p.items;
  pdl_wait();
  pdl_trigger();
  for (int64_t item = blockIdx.x / p.cluster; item < total; item += gridDim.x / p.cluster) {
    const int b = (int)paged_div(item, p.items), j = (int)(item - (int64_t)b * p.items);
    const DraftSeq seq = draft_seq(a, b, j == 0 && rank == 0 ? a.status : nullptr);
    const int per = a.Hkv * a.hgroups, group = j / per, head = j - group * per, kvh = head / a.hgroups;
    if (group * a.tokens >= seq.n) continue;                  // the whole cluster
    const DraftItem it = draft_item(a, seq.n, kvh, head - kvh * a.hgroups, group);
    const int rows = it.ni * it.nh, n = draft_visible(a, seq, it), ctx = seq.len - seq.n, new16 = ctx & ~15;
    const int64_t token = (int64_t)seq.first + it.i0;
    const int hq = kvh * a.G + it.h0;                         // the first query head

    // ---- slices first, first + step, ... ---------------------------------------------
    const uint32_t slices = ((uint32_t)n + 15) / 16, step = p.cluster * kWarps, first = warp * p.cluster + rank;
    const int32_t* table = a.table + (int64_t)b * a.max_pages;
    const uint32_t ps = a.page_size;
    // page and row of key lane % 16 of a slice
    struct Place {
      int id;
      uint32_t row;
    };
    auto place = [&](uint32_t s) {
      const uint32_t key = s * 16 + (lane & 15), pg = key / ps;
      return s < slices && key < (uint32_t)n ? Place{table[pg], key - pg * ps} : Place{-1, ~0u};
    };
    auto copy = [&](int slot, uint32_t s, const Place& at) {
      if (s < slices) {
        const bool in = at.row != ~0u, good = at.id >= 0 && at.id < a.n_pages;
        if (in && !good) flag_device(a.status, kDevCheck);
        copy_slice<T, D>(smem_u32(ring + slot * C::kSlot), p.k, p.v,
                         in && good ? ((int64_t)at.id * a.Hkv + kvh) * ps + at.row : -1);
      }
      cp_async_commit();
    };
    Place at[C::kSlots];
#pragma unroll
    for (int s = 0; s < C::kSlots; ++s) at[s] = place(first + s * step);
    if (threadIdx.x <= kBadWords) bad[threadIdx.x] = 0;
    Unit<T, D> me(smem + kWarps * C::kWarpBytes + C::kPart + warp * C::kScratch);
    auto row_of = [&](int r) {                                // of q
      const int i = r / it.nh;
      return static_cast<const T*>(p.q) + (token + i) * p.q_stride + (int64_t)(hq + r - i * it.nh) * D;
    };
    int mine[kMine];                                          // the tokens of the lane's rows
    DraftMask mask[kMine];
#pragma unroll
    for (int r = 0; r < kMine; ++r) {
      mine[r] = it.i0 + me.row(r) / it.nh;
      mask[r].read(a, seq, mine[r], me.row(r) < rows);
    }
    if constexpr (C::kBf16) {
      me.load_q(me.row(0) < rows ? row_of(me.row(0)) : nullptr, me.row(1) < rows ? row_of(me.row(1)) : nullptr);
    } else {
      for (int e = threadIdx.x; e < C::kRows * kCols; e += kWarps * 32) {
        const int r = e / kCols;
        reinterpret_cast<float4*>(part_o)[e] =
            r < rows ? reinterpret_cast<const float4*>(row_of(r))[e - r * kCols] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      __syncthreads();
      me.load_q(part_o, rows);
    }
#pragma unroll
    for (int s = 0; s < C::kSlots; ++s) copy(s, first + s * step, at[s]);
    Place ahead = place(first + C::kSlots * step);            // of the next slice to copy
    __syncthreads();                                          // `bad` is cleared
    int slot = 0;
    for (uint32_t s = first; s < slices; s += step) {
      asm volatile("cp.async.wait_group %0;" ::"n"(C::kSlots - 1) : "memory");
      __syncwarp();
      uint8_t* stage = ring + slot * C::kSlot;
      const int x = (int)s * 16, left = n - x;
      const bool all = x + 16 <= ctx;
      uint32_t see[kMine] = {};
      if (!all) {
        const uint32_t found = me.clean(stage, 0, left);
        if (found && lane == 0) {
          atomicOr(&bad[(x - new16) >> 5], found << ((x - new16) & 31));
          bad[kBadWords] = 1;
        }
#pragma unroll
        for (int r = 0; r < kMine; ++r)
          see[r] = me.row(r) < rows ? (uint32_t)mask[r].sees(a, seq, mine[r], x) & 0xffffu : 0;
        __syncwarp();
      }
      me.slice(stage, left, all, see, p.scale_log2);
      __syncwarp();
      copy(slot, s + C::kSlots * step, ahead);
      ahead = place(s + (C::kSlots + 1) * step);
      slot = slot + 1 == C::kSlots ? 0 : slot + 1;
    }
    // the warp's result, over its own ring
    cp_async_wait0();
    if constexpr (C::kBf16) me.result(rm[warp], rl[warp], reinterpret_cast<float*>(ring), first < slices);
    else me.result(rm[warp], rl[warp], reinterpret_cast<float*>(ring), rows, first < slices);
    __syncthreads();

    // ---- the CTA's sum, then the cluster's ------------------------------------------------
    const bool odd = bad[kBadWords] != 0;
    for (int e = threadIdx.x; e < rows * kCols; e += kWarps * 32) {
      const int h = e / kCols, c = e % kCols * 4;
      float2 ml[kWarps];
      float4 v[kWarps];
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        ml[x] = make_float2(rm[x][h], rl[x][h]);
        v[x] = ml[x].y == -1.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                               : *reinterpret_cast<const float4*>(smem + x * C::kWarpBytes +
                                                                  (h * C::kRedStride + c) * 4);
      }
      Sum s = join_sums(ml, v);
      if (odd) {
        const int i = it.i0 + h / it.nh;
        for (int k = 0; k < kBadWords; ++k) {
          const int x0 = new16 + k * 32;
          uint32_t todo = bad[k] ? bad[k] & (uint32_t)draft_sees(a, seq, i, x0) : 0;
          for (; todo; todo &= todo - 1) {
            const int x = x0 + __ffs(todo) - 1, pg = x / (int)ps, id = table[pg];
            if ((unsigned)id >= (unsigned)a.n_pages) continue;
            const uint8_t* vr =
                p.v + (((int64_t)id * a.Hkv + kvh) * ps + (x - pg * (int)ps)) * C::kRow + c * (int)sizeof(T);
            if constexpr (C::kBf16) {
              const uint2 q = *reinterpret_cast<const uint2*>(vr);
              s.o.x += if_bad(bf16lo(q.x));
              s.o.y += if_bad(bf16hi(q.x));
              s.o.z += if_bad(bf16lo(q.y));
              s.o.w += if_bad(bf16hi(q.y));
            } else {
              const float4 q = *reinterpret_cast<const float4*>(vr);
              s.o.x += if_bad(q.x);
              s.o.y += if_bad(q.y);
              s.o.z += if_bad(q.z);
              s.o.w += if_bad(q.w);
            }
          }
        }
      }
      *reinterpret_cast<float4*>(part_o + h * D + c) = s.o;
      if (c == 0) part_ml[h] = make_float2(s.m, s.l);
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    // runs of 32 columns, dealt out to the CTAs, then to their warps
    for (int e = (warp * p.cluster + rank) * 32 + lane; e < rows * kCols; e += kWarps * p.cluster * 32) {
      const int h = e / kCols, c = e % kCols * 4, i = h / it.nh;
      float2 ml[kMaxCluster];
      float4 v[kMaxCluster];
#pragma unroll
      for (int x = 0; x < kMaxCluster; ++x) {
        ml[x] = make_float2(-INFINITY, -1.f);
        v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (x < p.cluster) {
          ml[x] = cluster_load2(in_cta(smem_u32(&part_ml[h]), x));
          v[x] = cluster_load4(in_cta(smem_u32(part_o + h * D + c), x));
        }
      }
      const Sum s = join_sums(ml, v);
      const bool any = draft_sees_any(a, seq, it.i0 + i);
      const float inv = any ? 1.f / s.l : 0.f;
      const int64_t t = token + i, head_q = hq + h - i * it.nh;
      T* to = static_cast<T*>(p.o) + (t * a.H + head_q) * D + c;
      if constexpr (C::kBf16)
        *reinterpret_cast<uint2*>(to) = any ? make_uint2(pack_bf16x2(s.o.x * inv, s.o.y * inv),
                                                         pack_bf16x2(s.o.z * inv, s.o.w * inv))
                                            : make_uint2(0u, 0u);
      else
        *reinterpret_cast<float4*>(to) = any ? make_float4(s.o.x * inv, s.o.y * inv, s.o.z * inv, s.o.w * inv)
                                             : make_float4(0.f, 0.f, 0.f, 0.f);
      if (p.lse && c == 0) p.lse[head_q * a.T + t] = row_lse(s.m, s.l, any);
    }
    __syncwarp();
    cluster_arrive();                                         // no CTA leaves, or goes on, while another reads it
    cluster_wait();
  }
}

template <typename T, int D>
cudaError_t allow_spread() {
  return allow_smem_once<draft_spread_kernel<T, D>, true>(Cfg<T, D>::kSmem);
}
template <typename T, int D>
cudaLaunchConfig_t spread_config(int cluster, cudaLaunchAttribute (&attr)[2]) {
  using C = Cfg<T, D>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster);
  cfg.blockDim = dim3(C::kWarps * 32);
  cfg.dynamicSmemBytes = C::kSmem;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}
// Clusters that run at once, asked for once per device.  0 if that fails.
template <typename T, int D>
int clusters_fit(int dev, int cluster) {
  static std::atomic<int> known[64][kMaxCluster + 1];                // plus 1; 0: not asked yet
  int n = 0;
  if (dev < 64 && (n = known[dev][cluster].load(std::memory_order_relaxed)) > 0) return n - 1;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = spread_config<T, D>(cluster, attr);
  n = 0;
  if (allow_spread<T, D>() != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, draft_spread_kernel<T, D>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  if (dev < 64) known[dev][cluster].store(n + 1, std::memory_order_relaxed);
  return n;
}

template <typename T, int D>
cudaError_t run(const DraftProblem& p, int cluster, unsigned int* status, cudaStream_t s) {
  using C = Cfg<T, D>;
  SpreadArgs r = {};
  r.a = draft_batch(p, C::kRows, 1, status);
  r.q = p.q;
  r.q_stride = p.q_stride;
  // no pages: nothing is read, from any address that is one
  r.k = static_cast<const uint8_t*>(p.pool.n_pages ? p.pool.k : p.q);
  r.v = static_cast<const uint8_t*>(p.pool.n_pages ? p.pool.v : p.q);
  r.o = p.o;
  r.lse = p.lse;
  r.cluster = cluster;
  r.items = draft_items_most(r.a);
  r.scale_log2 = p.scale * 1.4426950408889634f;
  const cudaError_t e = allow_spread<T, D>();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = spread_config<T, D>(cluster, attr);
  cfg.gridDim = dim3((unsigned)(min64((int64_t)p.B * r.items, kMaxClusters) * cluster));
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, draft_spread_kernel<T, D>, r);
}

// Estimated time (us) and the cluster's size.  A cluster's time beside its
// slices of keys, a warp's slice while it waits for no other, a further wave of
// clusters, and a slice of every resident warp where the SMs are full; fitted
// with the other kernels' rates (draft_attn.cu).
template <typename T, int D>
double estimate(const DraftProblem& p, int* cluster) {
  using C = Cfg<T, D>;
  constexpr int w = D == 32 ? 0 : D == 64 ? 1 : 2;
  constexpr double kFirst = C::kBf16 ? (w == 0 ? 5.75 : w == 1 ? 6.66 : 8.45) : (w == 0 ? 8.0 : w == 1 ? 7.6 : 8.8);
  constexpr double kSlice = C::kBf16 ? (w == 0 ? 0.89 : w == 1 ? 1.2 : 1.22) : (w == 0 ? 1.56 : w == 1 ? 2.46 : 1.83);
  constexpr double kWave = C::kBf16 ? (w == 0 ? 3.9 : w == 1 ? 4.1 : 5.7) : (w == 0 ? 5.7 : w == 1 ? 4.4 : 4.76);
  constexpr double kLoaded = C::kBf16 ? (w == 0 ? 1.09 : w == 1 ? 2.25 : 3.2) : (w == 0 ? 2.73 : w == 1 ? 3.9 : 4.46);
  const DraftBatch a = draft_batch(p, C::kRows, 1, nullptr);
  const int64_t items = (int64_t)p.B * draft_items_most(a), slices = (a.cap + 15) / 16;
  const double all = p.B * draft_items_mean(p, a) * (draft_mean_keys(p, a) / 16 + 0.5);
  const double load = all / (2.0 * sm_count() * C::kWarps) * kLoaded;
  double best = INFINITY;
  *cluster = 1;
  int dev = 64;                                                      // 64: asked for every time
  if (cudaGetDevice(&dev) != cudaSuccess) cudaGetLastError();
  for (int c = 1; c <= kMaxCluster; ++c) {
    if (c > 1 && (int64_t)(c - 1) * C::kWarps >= slices) break;    // the CTAs before it have them all
    const int64_t fit = c > 1 ? clusters_fit<T, D>(dev, c) : max(clusters_fit<T, D>(dev, 1), 1);
    if (fit <= 0) continue;
    const double waves = (double)((items + fit - 1) / fit);
    const double rounds = fmax(1, (double)((slices + c * C::kWarps - 1) / (c * C::kWarps)));
    const double us = kFirst + fmax((rounds - 1) * kSlice, load) + (waves - 1) * kWave;
    if (us < best) {
      best = us;
      *cluster = c;
    }
  }
  return best;
}

template <typename F>
auto with_types(nt_dtype dt, const DraftProblem& p, const F& f) {
  auto widths = [&](auto t) {
    using T = decltype(t);
    if (p.d == 32) return f(t, std::integral_constant<int, 32>());
    if (p.d == 64) return f(t, std::integral_constant<int, 64>());
    return f(t, std::integral_constant<int, 128>());
  };
  return dt == NT_BF16 ? widths(bf16()) : widths(float());
}

}  // namespace

double draft_spread_us(nt_dtype dt, const DraftProblem& p, int* cluster) {
  return with_types(dt, p, [&](auto t, auto d) { return estimate<decltype(t), decltype(d)::value>(p, cluster); });
}
cudaError_t launch_draft_spread(nt_dtype dt, const DraftProblem& p, int cluster, unsigned int* status, cudaStream_t s) {
  return with_types(dt, p, [&](auto t, auto d) { return run<decltype(t), decltype(d)::value>(p, cluster, status, s); });
}

}  // namespace nt
