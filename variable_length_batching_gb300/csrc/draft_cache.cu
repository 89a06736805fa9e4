// What a step with drafted tokens needs around its attention: block tables
// and slot maps from request lengths, the tree's masks and positions, and the
// accepted tokens' keys and values moved up.  All three are latencies: a
// launch, and a few dependent loads.
#include <atomic>

#include "nt_common.cuh"

namespace nt {
namespace {

// ---- block tables and slot maps -------------------------------------------------
//
// One cluster of CTAs for the whole call, so that a phase may read what the one
// before it wrote with no second launch: the scan of what each row releases,
// takes and adds; then the released pages, then the taken ones, then the
// slots.  Every CTA scans all rows (their lengths are a load that all do at
// once), a thread a strip of them; pages and tokens are then dealt out one by
// one over all threads, however they lie in the rows, several searches side
// by side.  512 prompts of 65,000 tokens and back: 25 us by one CTA, 16.5 by eight,
// 12.4 by 16 (0.2 more for the flag of pages below 0); 16 sequences and back: 13.2,
// 8.4 and 8.3, the launches, cluster barriers and the loads between them.
constexpr int kResizeThreads = 512;
constexpr int kResizeCtas = 16, kResizePortable = 8;
constexpr int kResizeUnroll = 4;

struct ResizeArgs {
  const int32_t* new_lengths;
  int32_t* lengths;
  int32_t* table;
  int32_t* free_pages;
  int32_t* n_free;
  int32_t* cu;
  int32_t* pos0;
  int64_t* slots;
  int32_t* lacking;
  int B, page_size, max_pages, n_pages;
  int64_t T, cap;
  unsigned int* status;
};

struct Change {
  int old, now;             // positions before and after
  int have, want;           // pages
};
__device__ __forceinline__ int pages_of(const ResizeArgs& a, int n) {
  return (int)(((uint32_t)n + (uint32_t)a.page_size - 1) / (uint32_t)a.page_size);
}
__device__ __forceinline__ Change change_of(const ResizeArgs& a, int b, unsigned int* status) {
  Change c;
  c.old = a.lengths[b];
  c.now = a.new_lengths[b];
  if (c.old < 0 || c.old > a.cap || c.now < 0 || c.now > a.cap) {
    flag_device(status, kDevCheck);
    c.now = c.old;          // left as it is, and without pages to move
    c.have = c.want = 0;
    return c;
  }
  c.have = pages_of(a, c.old);
  c.want = pages_of(a, c.now);
  return c;
}
struct Sums {
  int64_t rel, take, add;   // pages released and taken, tokens added
  __device__ __forceinline__ void operator+=(const Sums& o) {
    rel += o.rel;
    take += o.take;
    add += o.add;
  }
};
__device__ __forceinline__ Sums sums_of(const Change& c) {
  return {max(c.have - c.want, 0), max(c.want - c.have, 0), max((int64_t)c.now - c.old, (int64_t)0)};
}

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__global__ void __launch_bounds__(kResizeThreads) paged_resize_kernel(const ResizeArgs a) {
  enum { kRel, kTake, kAdd };
  __shared__ Sums warp_sum[kResizeThreads / 32];
  __shared__ int ahead[3][kResizeThreads];         // released, taken, added in the rows in front of a thread's strip
  __shared__ int old_of[kResizeThreads], have_of[kResizeThreads], want_of[kResizeThreads];     // strips of one row
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = gridDim.x, cta = blockIdx.x;
  pdl_wait();
  pdl_trigger();
  // the scan of what rows release, take and add, every CTA for itself
  const int strip = (int)(((int64_t)a.B + kResizeThreads - 1) / kResizeThreads);
  const int b_lo = (int)min64(a.B, (int64_t)tid * strip), b_hi = (int)min64(a.B, (int64_t)b_lo + strip);
  const int nf = *a.n_free;
  Sums mine = {0, 0, 0};
  Change one = {};
  for (int b = b_lo; b < b_hi; ++b) {
    one = change_of(a, b, cta == 0 ? a.status : nullptr);
    mine += sums_of(one);
  }
  old_of[tid] = one.old;
  have_of[tid] = one.have;
  want_of[tid] = one.want;
  Sums inc = mine;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const Sums o = {__shfl_up_sync(0xffffffffu, inc.rel, m), __shfl_up_sync(0xffffffffu, inc.take, m),
                    __shfl_up_sync(0xffffffffu, inc.add, m)};
    if (lane >= m) inc += o;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  Sums before = {inc.rel - mine.rel, inc.take - mine.take, inc.add - mine.add}, total = {0, 0, 0};
#pragma unroll
  for (int w = 0; w < kResizeThreads / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  const bool broken = nf < 0 || nf > a.n_pages || nf + total.rel > a.n_pages;
  const int64_t lack = max64(0, total.take - total.rel - max(nf, 0)), over = max64(0, total.add - a.T);
  const bool none = broken || lack > 0 || over > 0;
  // (below 2^31 unless nothing is done)
  ahead[kRel][tid] = (int)before.rel;
  ahead[kTake][tid] = (int)before.take;
  ahead[kAdd][tid] = (int)before.add;
  cluster_sync_all();                    // every CTA has read what is written from here on
  if (cta == 0 && tid == 0) {
    if (broken) flag_device(a.status, kDevCheck);
    a.lacking[0] = (int)min64(lack, 0x7fffffff);
    a.lacking[1] = (int)min64(over, 0x7fffffff);
    if (!none) *a.n_free = (int)(nf + total.rel - total.take);
    a.cu[a.B] = none ? 0 : (int)total.add;
  }
  {
    Sums at = before;
    for (int b = b_lo; b < b_hi; ++b) {
      const Change c = strip == 1 ? one : change_of(a, b, nullptr);
      if (b % ctas == cta) {
        a.cu[b] = none ? 0 : (int)at.add;
        a.pos0[b] = c.old;
        if (strip == 1 && !none) a.lengths[b] = c.now;
      }
      at += sums_of(c);
    }
  }
  const uint32_t me = cta * kResizeThreads + tid, all = ctas * kResizeThreads;
  const uint32_t T = (uint32_t)a.T;
  if (none) {
    for (uint32_t t = me; t < T; t += all) a.slots[t] = -1;
    return;
  }
  // The strips that hold ranks r[k] of a sum, and the places in them.
  auto strips_of = [&](int what, const uint32_t (&r)[kResizeUnroll], int (&lo)[kResizeUnroll]) {
#pragma unroll
    for (int k = 0; k < kResizeUnroll; ++k) lo[k] = 0;
#pragma unroll
    for (int step = kResizeThreads / 2; step > 0; step >>= 1)
#pragma unroll
      for (int k = 0; k < kResizeUnroll; ++k)
        if (ahead[what][lo[k] + step] <= (int)r[k]) lo[k] += step;
  };
  // The row in a strip, its lengths before and the place in its share of the sum.
  auto row_of = [&](int what, int lo, uint32_t rank, int& off, Change& c) {
    off = (int)rank - ahead[what][lo];
    if (strip == 1) {
      c.old = old_of[lo];
      c.have = have_of[lo];
      c.want = want_of[lo];
      return lo;
    }
    for (int b = lo * strip;; ++b) {
      c = change_of(a, b, nullptr);
      const Sums s = sums_of(c);
      const int n = (int)(what == kRel ? s.rel : what == kTake ? s.take : s.add);
      if (off < n) return b;
      off -= n;
    }
  };
  // released pages: the first of them ends on top of the stack
  const int64_t top = nf + total.rel - 1;
  const uint32_t rel = (uint32_t)total.rel, take = (uint32_t)total.take, add = (uint32_t)total.add;
  auto moves = [&](int what, uint32_t count, auto f) {
    for (uint32_t r0 = me; r0 < count; r0 += all * kResizeUnroll) {
      uint32_t r[kResizeUnroll];
      int lo[kResizeUnroll];
#pragma unroll
      for (int k = 0; k < kResizeUnroll; ++k) r[k] = min(r0 + k * all, count - 1);
      strips_of(what, r, lo);
#pragma unroll
      for (int k = 0; k < kResizeUnroll; ++k) {
        if (r0 + k * all >= count) break;
        int off;
        Change c;
        const int b = row_of(what, lo[k], r[k], off, c);
        f(r[k], b, off, c);
      }
    }
  };
  moves(kRel, rel, [&](uint32_t r, int b, int off, const Change& c) {
    int32_t* e = a.table + (int64_t)b * a.max_pages + c.want + off;
    a.free_pages[top - r] = *e;
    *e = -1;
  });
  if (take > 0) {
    if (rel > 0) cluster_sync_all();
    moves(kTake, take, [&](uint32_t r, int b, int off, const Change& c) {
      a.table[(int64_t)b * a.max_pages + c.have + off] = a.free_pages[top - r];
    });
  }
  if (take > 0 || strip > 1) cluster_sync_all();
  const uint32_t ps = a.page_size;
  moves(kAdd, add, [&](uint32_t t, int b, int off, const Change& c) {
    const uint32_t x = (uint32_t)c.old + off, pg = x / ps;
    const int id = a.table[(int64_t)b * a.max_pages + pg];
    if (id < 0) flag_device(a.status, kDevCheck);           // and a slot that is not taken for none
    a.slots[t] = id < 0 ? -2 : (int64_t)id * ps + (x - pg * ps);
  });
  for (uint32_t t = add + me; t < T; t += all) a.slots[t] = -1;
  if (strip > 1) {
    cluster_sync_all();                  // nobody reads the old lengths any more
    for (int64_t b = me; b < a.B; b += all) a.lengths[b] = change_of(a, (int)b, nullptr).now;
  }
}

cudaLaunchConfig_t resize_config(int ctas, cudaLaunchAttribute (&attr)[2]) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kResizeThreads);
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}
// Asked for once per device: whether a cluster of 16 fits one.
int resize_ctas() {
  static std::atomic<int> known[64];
  int dev = 64;
  if (cudaGetDevice(&dev) != cudaSuccess) cudaGetLastError();
  int n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (n) return n;
  int fit = 0;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = resize_config(kResizeCtas, attr);
  if (allow_smem_once<paged_resize_kernel, true>(0) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&fit, paged_resize_kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    fit = 0;
  }
  n = fit > 0 ? kResizeCtas : kResizePortable;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// ---- the tree's masks and positions ---------------------------------------------
//
// A CTA to a sequence, a thread to a token.  In round r a token adds what the
// token 2^r above it has gathered, so a path of 256 takes eight rounds.  A
// token's own words stay in registers; W words, so that they are moved whole.
constexpr int kTreeThreads = kDraftMaxNew;

template <int W>
__global__ void __launch_bounds__(kTreeThreads) draft_tree_kernel(const int32_t* parents, const int32_t* cu, int64_t T,
                                                                  int max_new, const int32_t* pos0, int64_t* bits,
                                                                  int32_t* positions, unsigned int* status) {
  struct alignas(W % 2 ? 8 : 16) Words {
    unsigned long long w[W];
  };
  __shared__ Words words[2][64 * W];
  __shared__ int2 above[2][64 * W];                // the next one to ask, and the tokens in between
  const int b = blockIdx.x, i = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  const int lo = cu[b], hi = cu[b + 1], n = hi - lo, start = pos0 ? pos0[b] : 0;
  if (lo < 0 || hi < lo || hi > T || n > max_new) {
    if (i == 0) flag_device(status, kDevCheck);
    return;
  }
  if (b == gridDim.x - 1)                          // tokens that only fill up the batch (where the end is known)
    for (int64_t t = (int64_t)hi + i; t < T; t += blockDim.x) {
      if (positions) positions[t] = 0;
      for (int w = 0; w < W; ++w) bits[t * W + w] = 0;
    }
  Words mine;
  int2 up = make_int2(-1, 0);
  if (i < n) {
    up.x = parents[(int64_t)lo + i];
    if (up.x >= i || up.x < -1) {
      flag_device(status, kDevCheck);
      up.x = -1;
    }
    up.y = up.x >= 0;
  }
#pragma unroll
  for (int w = 0; w < W; ++w) mine.w[w] = w == i >> 6 ? 1ull << (i & 63) : 0;
  for (int reach = 1, at = 0; reach < n; reach <<= 1, at ^= 1) {
    words[at][i] = mine;
    above[at][i] = up;
    if (!__syncthreads_or(up.x >= 0)) break;       // (everybody has asked all the way up)
    if (up.x >= 0) {
      const Words theirs = words[at][up.x];
      const int2 next = above[at][up.x];
#pragma unroll
      for (int w = 0; w < W; ++w) mine.w[w] |= theirs.w[w];
      up = make_int2(next.x, up.y + next.y);
    }
  }
  if (i >= n) return;
  if (positions) positions[(int64_t)lo + i] = start + up.y;
  if constexpr (W % 2 == 0) {
    ulonglong2* to = reinterpret_cast<ulonglong2*>(bits + ((int64_t)lo + i) * W);
    if ((reinterpret_cast<uintptr_t>(bits) & 15) == 0) {
#pragma unroll
      for (int w = 0; w < W; w += 2) to[w / 2] = make_ulonglong2(mine.w[w], mine.w[w + 1]);
      return;
    }
  }
#pragma unroll
  for (int w = 0; w < W; ++w) bits[((int64_t)lo + i) * W + w] = (int64_t)mine.w[w];
}

// ---- the accepted tokens moved up ---------------------------------------------------
//
// Kept token i of a sequence goes from position pos0 + kept[i] to pos0 + i.
// The indices grow, so kept[i] >= i: a CTA that moves a run of tokens, all
// read before any is written, and then the next run, reads nothing that it
// has written.  CTAs have a sequence, a range of its heads and a side each; HBM
// bounds a large batch (256 sequences, 35 tokens each of 8 heads of 256 bytes: 84 MB
// in 17 us in a graph, four words in flight to a thread and 64 warps to an SM; eight
// and 32 took 20; as a call on cold inputs 19.3), the launch and four dependent loads a
// small one (16 sequences: 3.4).
constexpr int kKeepThreads = 256;
constexpr int kKeepUnroll = 4;

struct KeepArgs {
  uint8_t* pool[2];
  const int32_t* kept;
  const int32_t* cu;
  const int32_t* table;
  const int32_t* pos0;
  int64_t K;
  int n_pages, page_size, H, row_bytes, B, max_pages;
  int heads;                // of a CTA
  unsigned int* status;
};

__device__ __forceinline__ int64_t keep_offset(const KeepArgs& a, int b, int64_t x) {
  if (x < 0 || x >= (int64_t)a.max_pages * a.page_size) return -1;
  const int pg = (int)(x / a.page_size);
  const int id = a.table[(int64_t)b * a.max_pages + pg];
  if (id < 0 || id >= a.n_pages) return -1;
  return ((int64_t)id * a.H * a.page_size + (x - (int64_t)pg * a.page_size)) * a.row_bytes;
}

__global__ void __launch_bounds__(kKeepThreads, 8) paged_keep_kernel(const KeepArgs a) {
  __shared__ int64_t from[kKeepThreads], to[kKeepThreads];
  pdl_wait();
  pdl_trigger();
  const int side = blockIdx.y & 1, h0 = (int)(blockIdx.y >> 1) * a.heads, nh = min(a.heads, a.H - h0);
  uint8_t* const pool = side ? a.pool[1] : a.pool[0];
  const int words = a.row_bytes / 16, per = nh * words;            // 16-byte words of a token
  const int run = max(1, kKeepThreads * kKeepUnroll / per);        // tokens read before any is written
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    const int lo = a.cu[b], hi = a.cu[b + 1];
    if (lo < 0 || hi < lo || hi > a.K) {
      if (threadIdx.x == 0) flag_device(a.status, kDevCheck);
      continue;
    }
    const int64_t p0 = a.pos0[b];
    for (int i0 = lo; i0 < hi; i0 += kKeepThreads) {
      const int n = min(kKeepThreads, hi - i0);
      __syncthreads();
      if (threadIdx.x < n) {
        const int i = i0 + threadIdx.x, k = a.kept[i];
        int64_t s = -1, d = -1;
        if (k < i - lo || (i > lo && k <= a.kept[i - 1]) || p0 < 0) {
          flag_device(a.status, kDevCheck);
        } else if (k > i - lo) {
          s = keep_offset(a, b, p0 + k);
          d = keep_offset(a, b, p0 + i - lo);
          if (s < 0 || d < 0) flag_device(a.status, kDevCheck);
        }
        from[threadIdx.x] = d < 0 ? -1 : s;
        to[threadIdx.x] = d;
      }
      __syncthreads();
      for (int r = 0; r < n; r += run) {
        const int total = min(run, n - r) * per;
        for (int e0 = 0; e0 < total; e0 += kKeepThreads * kKeepUnroll) {   // one pass, but for very wide tokens
          uint4 v[kKeepUnroll];
          uint8_t* at[kKeepUnroll];
#pragma unroll
          for (int u = 0; u < kKeepUnroll; ++u) {
            const int e = e0 + u * kKeepThreads + threadIdx.x;
            at[u] = nullptr;
            if (e >= total) continue;
            const int t = r + e / per, w = e % per;
            if (from[t] < 0) continue;
            const int64_t off = ((int64_t)(h0 + w / words) * a.page_size) * a.row_bytes + (w % words) * 16;
            v[u] = *reinterpret_cast<const uint4*>(pool + from[t] + off);
            at[u] = pool + to[t] + off;
          }
          __syncthreads();
#pragma unroll
          for (int u = 0; u < kKeepUnroll; ++u)
            if (at[u]) *reinterpret_cast<uint4*>(at[u]) = v[u];
          __syncthreads();
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_paged_resize(const int32_t* new_lengths, int B, int page_size, int32_t* table, int max_pages,
                                int32_t* lengths, int32_t* free_pages, int n_pages, int32_t* n_free, int32_t* cu,
                                int32_t* pos0, int64_t* slots, int64_t T, int32_t* lacking, unsigned int* status,
                                cudaStream_t s) {
  ResizeArgs a;
  a.new_lengths = new_lengths;
  a.lengths = lengths;
  a.table = table;
  a.free_pages = free_pages;
  a.n_free = n_free;
  a.cu = cu;
  a.pos0 = pos0;
  a.slots = slots;
  a.lacking = lacking;
  a.B = B;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.n_pages = n_pages;
  a.T = T;
  a.cap = min64((int64_t)max_pages * page_size, 0x7fffffff);
  a.status = status;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = resize_config(resize_ctas(), attr);
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, paged_resize_kernel, a);
}

cudaError_t launch_draft_tree(const int32_t* parents, const int32_t* cu, int B, int64_t T, int max_new,
                              const int32_t* pos0, int64_t* bits, int32_t* positions, unsigned int* status,
                              cudaStream_t s) {
  if (B == 0 || T == 0) return cudaSuccess;
  const dim3 grid(B), block((max_new + 31) / 32 * 32);
  switch ((max_new + 63) / 64) {
    case 1: return launch_pdl(draft_tree_kernel<1>, grid, block, 0, s, parents, cu, T, max_new, pos0, bits, positions, status);
    case 2: return launch_pdl(draft_tree_kernel<2>, grid, block, 0, s, parents, cu, T, max_new, pos0, bits, positions, status);
    case 3: return launch_pdl(draft_tree_kernel<3>, grid, block, 0, s, parents, cu, T, max_new, pos0, bits, positions, status);
    default: return launch_pdl(draft_tree_kernel<4>, grid, block, 0, s, parents, cu, T, max_new, pos0, bits, positions, status);
  }
}

cudaError_t launch_paged_keep(const PagedPool& p, const int32_t* kept, int64_t K, const int32_t* cu, int B,
                              const int32_t* table, int max_pages, const int32_t* pos0, unsigned int* status,
                              cudaStream_t s) {
  if (B == 0 || K == 0) return cudaSuccess;
  KeepArgs a;
  a.pool[0] = static_cast<uint8_t*>(p.k);
  a.pool[1] = static_cast<uint8_t*>(p.v);
  a.kept = kept;
  a.cu = cu;
  a.table = table;
  a.pos0 = pos0;
  a.K = K;
  a.n_pages = p.n_pages;
  a.page_size = p.page_size;
  a.H = p.H;
  a.row_bytes = p.row_bytes;
  a.B = B;
  a.max_pages = max_pages;
  // Heads that make a run of what a sequence keeps on average: with fewer, short lists leave threads without work
  // (246 sequences that keep one token of 12 heads of 512 bytes: 19.6 -> 3.9 us), with more, a list takes several
  // runs.  Halved where that leaves SMs without a CTA.
  const int64_t run = min64(64, (K + B - 1) / B);
  const int64_t bytes = run * p.row_bytes;
  a.heads = max(1, (int)min64(p.H, (kKeepThreads * kKeepUnroll * 16 + bytes / 2) / bytes));
  while (a.heads > 1 && (int64_t)B * 2 * ((p.H + a.heads - 1) / a.heads) < 2 * sm_count()) a.heads = (a.heads + 1) / 2;
  while ((p.H + a.heads - 1) / a.heads > 32767) a.heads *= 2;
  a.status = status;
  const int groups = (p.H + a.heads - 1) / a.heads;
  return launch_pdl(paged_keep_kernel, dim3(min(B, 65536), 2 * groups), dim3(kKeepThreads), 0, s, a);
}

}  // namespace nt
