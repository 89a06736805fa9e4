// Attention of one new token per sequence over a paged cache, a cluster of
// CTAs per item (a sequence's key head with up to HP of its query heads):
// where there are few items, and for any page size.
//
// A decoding step of one or a few sequences waits for latencies, not for
// bandwidth: launch, length, pages, keys, and the joins.  Here nothing else is
// left.  There is no plan: cluster i has item i.  Its CTAs' warps take the
// item's slices of 16 keys in turn, each warp with its own ring of slots,
// filled row by row with cp.async, and no barrier while it has slices.  Then
// the warps' results are merged in the CTA, and the CTAs' through distributed
// shared memory, each CTA joining its share of the output columns, in place
// of a second launch.  A context of 777 keys and 12 heads of 64 takes 4.2 us
// (8.3 on the tile kernel), four of 4,000 with 8 key heads of 128 14.1 (18.3).
#include <type_traits>

#include "paged_plan.cuh"
#include "paged_worker.cuh"

namespace nt {
namespace {

using namespace paged;

constexpr int kMaxCluster = kPagedMaxCluster;
constexpr int64_t kMaxClusters = 1 << 24;    // of a launch

template <typename T, int D, int HP>
struct Cfg {
  static constexpr bool kBf16 = sizeof(T) == 2;
  static constexpr uint32_t kRow = D * sizeof(T);
  static constexpr uint32_t kSlot = 2 * 16 * kRow;                 // keys and values of a slice
  // half an SM's shared memory at most: two CTAs on each, so that clusters are twice as many
  static constexpr int kWarps = kRow <= 128 ? 8 : kRow == 256 ? 6 : 3;
  static constexpr int kSlots = kRow <= 128 ? 3 : 2;
  static constexpr uint32_t kWarpBytes = kSlots * kSlot;
  static constexpr uint32_t kPart = HP * D * 4;                    // the CTA's output; before, fp32: its query rows
  static constexpr uint32_t kScratch = Worker<T, D, HP>::kScratch; // of a warp
  static constexpr uint32_t kSmem = kWarps * (kWarpBytes + kScratch) + kPart;
  static constexpr int kRedStride = D + 4;
  static_assert(HP * kRedStride * 4 <= kWarpBytes && kSmem <= 111 * 1024, "shared memory");
};

struct SpreadArgs {
  const void* q;
  int64_t q_stride;
  const void* k;
  const void* v;
  const int32_t* table;
  const int32_t* lengths;
  void* o;
  float* lse;
  int B, H, G, Hkv, max_pages, page_size, n_pages, items, hgroups, cluster;
  float scale_log2;
  unsigned int* status;
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

template <typename T, int D, int HP>
__global__ void __launch_bounds__((Cfg<T, D, HP>::kWarps * 32), 2) paged_attn_spread_kernel(const SpreadArgs a) {
  using C = Cfg<T, D, HP>;
  constexpr int kWarps = C::kWarps, kCols = D / 4;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ float rm[kWarps][16], rl[kWarps][16];
  __shared__ float2 part_ml[HP];                            // the CTA's maxima and sums
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = smem + warp * C::kWarpBytes;
  float* part_o = reinterpret_cast<float*>(smem + kWarps * C::kWarpBytes);
  const uint32_t rank = blockIdx.x % a.cluster;
  const int64_t cap = min64((int64_t)a.max_pages * a.page_size, 0x7fffffff), total = (int64_t)a.B * a.items;
  pdl_wait();
  pdl_trigger();
  for (int64_t item = blockIdx.x / a.cluster; item < total; item += gridDim.x / a.cluster) {
    const int b = (int)paged_div(item, a.items), j = (int)(item - (int64_t)b * a.items), kvh = j / a.hgroups;
    const int h0 = j % a.hgroups * HP, nh = min(HP, a.G - h0);
    const int64_t hq = (int64_t)kvh * a.G + h0;               // the first query head
    const int n = paged_length(a.lengths, b, cap, a.status);
    T* o = static_cast<T*>(a.o) + ((int64_t)b * a.H + hq) * D;
    if (n == 0) {                                             // the whole cluster
      if (rank == 0) {
        for (int e = threadIdx.x; e < nh * D; e += kWarps * 32) o[e] = from_f32<T>(0.f);
        if (a.lse && threadIdx.x < nh) a.lse[(hq + threadIdx.x) * a.B + b] = -INFINITY;
      }
      continue;
    }

    // ---- slices first, first + step, ... ---------------------------------------------
    const uint32_t slices = ((uint32_t)n + 15) / 16, step = a.cluster * kWarps, first = warp * a.cluster + rank;
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
        copy_slice<T, D>(smem_u32(ring + slot * C::kSlot), a.k, a.v,
                         in && good ? ((int64_t)at.id * a.Hkv + kvh) * ps + at.row : -1);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    Place at[C::kSlots];
  #pragma unroll
    for (int s = 0; s < C::kSlots; ++s) at[s] = place(first + s * step);
    Worker<T, D, HP> me(16, 0, smem + kWarps * C::kWarpBytes + C::kPart + warp * C::kScratch);
    const T* q = static_cast<const T*>(a.q) + b * a.q_stride + hq * D;
    if constexpr (Worker<T, D, HP>::kKeepsQ) {
      for (int e = threadIdx.x; e < nh * kCols; e += kWarps * 32)
        reinterpret_cast<float4*>(part_o)[e] = reinterpret_cast<const float4*>(q)[e];
      __syncthreads();
      q = part_o;
    }
    me.load_q(q, nh);
  #pragma unroll
    for (int s = 0; s < C::kSlots; ++s) copy(s, first + s * step, at[s]);
    Place ahead = place(first + C::kSlots * step);            // of the next slice to copy
    int slot = 0;
    for (uint32_t s = first; s < slices; s += step) {
      asm volatile("cp.async.wait_group %0;" ::"n"(C::kSlots - 1) : "memory");
      __syncwarp();
      me.tile(ring + slot * C::kSlot, C::kSlot / 2, (int)min((uint32_t)n - s * 16, 16u), a.scale_log2);
      __syncwarp();
      copy(slot, s + C::kSlots * step, ahead);
      ahead = place(s + (C::kSlots + 1) * step);
      slot = slot + 1 == C::kSlots ? 0 : slot + 1;
    }
    // the warp's result, over its own ring
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    me.result(rm[warp], rl[warp], reinterpret_cast<float*>(ring), nh, first < slices);
    __syncthreads();

    // ---- the CTA's sum, then the cluster's ------------------------------------------------
    for (int e = threadIdx.x; e < nh * kCols; e += kWarps * 32) {
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
      const Sum s = join_sums(ml, v);
      *reinterpret_cast<float4*>(part_o + h * D + c) = s.o;
      if (c == 0) part_ml[h] = make_float2(s.m, s.l);
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    // runs of 32 columns, dealt out to the CTAs, then to their warps
    for (int e = (warp * a.cluster + rank) * 32 + lane; e < nh * kCols; e += kWarps * a.cluster * 32) {
      const int h = e / kCols, c = e % kCols * 4;
      float2 ml[kMaxCluster];
      float4 v[kMaxCluster];
  #pragma unroll
      for (int x = 0; x < kMaxCluster; ++x) {
        ml[x] = make_float2(-INFINITY, -1.f);
        v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (x < a.cluster) {
          ml[x] = cluster_load2(in_cta(smem_u32(&part_ml[h]), x));
          v[x] = cluster_load4(in_cta(smem_u32(part_o + h * D + c), x));
        }
      }
      const Sum s = join_sums(ml, v);
      const float inv = 1.f / s.l;
      if constexpr (C::kBf16)
        *reinterpret_cast<uint2*>(o + h * D + c) = make_uint2(pack_bf16x2(s.o.x * inv, s.o.y * inv),
                                                              pack_bf16x2(s.o.z * inv, s.o.w * inv));
      else
        *reinterpret_cast<float4*>(o + h * D + c) = make_float4(s.o.x * inv, s.o.y * inv, s.o.z * inv, s.o.w * inv);
      if (a.lse && c == 0) a.lse[(hq + h) * a.B + b] = (s.m + log2f(s.l)) * 0.6931471805599453f;
    }
    __syncwarp();
    cluster_arrive();                                         // no CTA leaves, or goes on, while another reads it
    cluster_wait();
  }
}

template <typename T, int D, int HP>
cudaError_t allow_spread() {
  return allow_smem_once<paged_attn_spread_kernel<T, D, HP>, true>(Cfg<T, D, HP>::kSmem);
}
template <typename T, int D, int HP>
cudaLaunchConfig_t spread_config(int cluster, cudaLaunchAttribute (&attr)[2]) {
  using C = Cfg<T, D, HP>;
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
// Clusters that run at once, asked for once per device (GPCs differ in size,
// so it is not the SMs' number over the cluster's).  0 if that fails.
template <typename T, int D, int HP>
int clusters_fit(int dev, int cluster) {
  static std::atomic<int> known[64][kMaxCluster + 1];                // plus 1; 0: not asked yet
  int n = 0;
  if (dev < 64 && (n = known[dev][cluster].load(std::memory_order_relaxed)) > 0) return n - 1;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = spread_config<T, D, HP>(cluster, attr);
  n = 0;
  if (allow_spread<T, D, HP>() != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, paged_attn_spread_kernel<T, D, HP>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  if (dev < 64) known[dev][cluster].store(n + 1, std::memory_order_relaxed);
  return n;
}

template <typename T, int D, int HP>
cudaError_t run(const PagedAttnProblem& p, int cluster, unsigned int* status, cudaStream_t s) {
  using C = Cfg<T, D, HP>;
  SpreadArgs a;
  a.q = p.q;
  a.q_stride = p.q_stride;
  a.k = p.pool.n_pages ? p.pool.k : p.q;          // no pages: nothing is read, from any address that is one
  a.v = p.pool.n_pages ? p.pool.v : p.q;
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
  a.cluster = cluster;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  a.status = status;
  const cudaError_t e = allow_spread<T, D, HP>();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = spread_config<T, D, HP>(cluster, attr);
  cfg.gridDim = dim3((unsigned)(min64((int64_t)p.B * a.items, kMaxClusters) * cluster));
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, paged_attn_spread_kernel<T, D, HP>, a);
}

// Estimated time (us) and the cluster's size.  A CTA takes about 4 us with one
// round of slices on its warps, and t for each further one.  The clusters that
// fit on the device at once (two CTAs on an SM) run together.  A batch waits for
// its longest items, so theirs count a quarter more: 16 contexts of up to 4,688
// keys, most of them far shorter, 8 key heads of 128, take 27.4 us here and
// 17.6 on the tile kernel, which deals them out evenly; all of 4,000 42.7 and
// 46.9.  HBM gives 6.8 TB/s.
template <typename T, int D, int HP>
double estimate(const PagedAttnProblem& p, int* cluster) {
  using C = Cfg<T, D, HP>;
  const double first = HP == 16 ? 5.0 : C::kRow <= 128 ? 3.9 : 4.1;
  const double t = C::kBf16 ? (HP == 16 ? 1.35 : D == 128 ? 0.9 : D == 64 ? 0.75 : 0.6) : (D == 128 ? 1.7 : D == 64 ? 1.3 : 0.9) * (HP == 8 ? 1.5 : 1);
  const int64_t items = paged_items(p, HP), cap = paged_cap(p), slices = (cap + 15) / 16;
  double best = INFINITY;
  *cluster = 1;
  int dev = 64;                                                      // 64: asked for every time
  if (cudaGetDevice(&dev) != cudaSuccess) cudaGetLastError();
  for (int c = 1; c <= kMaxCluster; ++c) {
    if (c > 1 && (int64_t)(c - 1) * C::kWarps >= slices) break;    // the CTAs before it have them all
    const int64_t fit = c > 1 ? clusters_fit<T, D, HP>(dev, c) : max(clusters_fit<T, D, HP>(dev, 1), 1);
    if (fit <= 0) continue;
    const double waves = (double)((items + fit - 1) / fit);
    const double rounds = fmax(1, (double)((slices + c * C::kWarps - 1) / (c * C::kWarps)));
    const double more = (rounds - 1) * t, us = first + more * (p.B > 1 ? 1.25 : 1) + (waves - 1) * (5.3 + more);
    if (us < best) {
      best = us;
      *cluster = c;
    }
  }
  const double bytes = (double)p.B * p.pool.H * cap * 2 * C::kRow * paged_mean_part(p);
  return fmax(best, 3.8 + bytes / 6.8e6);
}

template <typename T_, int D_, int HP_>
struct Types {
  using T = T_;
  static constexpr int D = D_, HP = HP_;
};
// f(Types) for the problem's type and sizes.
template <typename F>
auto with_types(nt_dtype dt, const PagedAttnProblem& p, const F& f) {
  const int G = p.H / p.pool.H;
  auto heads = [&](auto d) {
    constexpr int D = decltype(d)::value;
    if (dt == NT_BF16) return G <= 8 ? f(Types<bf16, D, 8>()) : f(Types<bf16, D, 16>());
    if (G == 1) return f(Types<float, D, 1>());
    if (G == 2) return f(Types<float, D, 2>());
    if (G <= 4) return f(Types<float, D, 4>());
    return f(Types<float, D, 8>());
  };
  if (p.d == 32) return heads(std::integral_constant<int, 32>());
  if (p.d == 64) return heads(std::integral_constant<int, 64>());
  return heads(std::integral_constant<int, 128>());
}

}  // namespace

double paged_attn_spread_us(nt_dtype dt, const PagedAttnProblem& p, int* cluster) {
  return with_types(dt, p, [&](auto k) {
    using K = decltype(k);
    return estimate<typename K::T, K::D, K::HP>(p, cluster);
  });
}
cudaError_t launch_paged_attn_spread(nt_dtype dt, const PagedAttnProblem& p, int cluster, unsigned int* status,
                                     cudaStream_t s) {
  return with_types(dt, p, [&](auto k) {
    using K = decltype(k);
    return run<typename K::T, K::D, K::HP>(p, cluster, status, s);
  });
}

}  // namespace nt
