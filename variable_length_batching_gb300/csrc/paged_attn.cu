// Attention of one new token per sequence over a paged key/value cache on
// CUDA cores, and the join of its partial results.
//
//   o_h = sum_j softmax_j(scale q_h . k_j) v_j over the sequence's j < len,
// query head h reading key head h / G.  One pass over the keys with a running
// maximum and sum.
//
// This kernel takes any page size and both types; it serves fp32 and the
// shapes the tensor-core kernel does not take.  A warp loads a key's row
// across its lanes (D / 32 elements each) and works on batches of 32 / GP
// keys, GP the group's heads rounded up to a power of two, at most 8: the
// 32 lane-partial dot products of a batch are reduced together by a
// transposing butterfly (31 shuffles for 32 sums instead of 160), which
// leaves one (key, head) score per lane.  The warps of a CTA take batches in
// turn, each with its own running maximum, sum and output, merged in shared
// memory at the end of a segment (see paged_plan.cuh for the split).
#include "paged_plan.cuh"

namespace nt {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 64;           // keys per unit of the split
constexpr int kHeads = 8;           // query heads of one item, at most
constexpr int kExtra = 2;           // an item's cost beside its tiles, in tiles

template <int N>
__device__ __forceinline__ void load_row(const float* p, float* x) {
  if constexpr (N == 4) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  } else if constexpr (N == 2) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    x[0] = v.x; x[1] = v.y;
  } else {
    x[0] = *p;
  }
}
template <int N>
__device__ __forceinline__ void load_row(const bf16* p, float* x) {
  if constexpr (N == 4) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xffff0000u);
  } else if constexpr (N == 2) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
    x[0] = __uint_as_float(v << 16); x[1] = __uint_as_float(v & 0xffff0000u);
  } else {
    x[0] = __bfloat162float(*p);
  }
}

// v[i] summed over the lanes, for i = this lane: halves the array and the
// lane distance together.
__device__ __forceinline__ float butterfly(float (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) {
    const bool up = lane & m;
#pragma unroll
    for (int i = 0; i < m; ++i) {
      const float give = up ? v[i] : v[i + m];
      const float keep = up ? v[i + m] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, m);
    }
  }
  return v[0];
}

template <typename T, int D, int GP>
__global__ void __launch_bounds__(kThreads, 2) paged_attn_kernel(const PagedAttnProblem p, int items, int hgroups,
                                                              int G, bool whole_items, float scale_log2,
                                                              unsigned int* status) {
  constexpr int N = D / 32;          // elements of a row per lane
  constexpr int KB = 32 / GP;        // keys of a batch
  __shared__ PagedPlan plan;
  __shared__ float red_o[kWarps][GP][D];
  __shared__ float red_m[kWarps][GP], red_l[kWarps][GP];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t cap = min64((int64_t)p.max_pages * p.pool.page_size, 0x7fffffff);
  const int heads = min(kHeads, G);
  const PagedPartials part = paged_partials(p.workspace, gridDim.x, heads);
  pdl_wait();
  pdl_trigger();
  paged_plan(p.lengths, p.B, cap, items, kTile, kExtra, blockIdx.x, gridDim.x, &plan, status, kThreads);
  // sequences with no key: zeros
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (paged_length(p.lengths, b, cap, nullptr) != 0) continue;
    for (int e = threadIdx.x; e < p.H * D; e += kThreads)
      static_cast<T*>(p.o)[(int64_t)b * p.H * D + e] = from_f32<T>(0.f);
    if (p.lse)
      for (int h = threadIdx.x; h < p.H; h += kThreads) p.lse[(int64_t)h * p.B + b] = -INFINITY;
  }
  PagedWalk w;
  w.init(plan, p.lengths, p.B, cap, kTile, kExtra, whole_items);
  const int ps = p.pool.page_size;
  const int my_key = lane / GP;
  int64_t open_id = -1, open_parts = 0;      // the item left unfinished
  while (w.next(p.lengths, p.B, cap, items, kTile, kExtra)) {
    const int kvh = w.seg_item / hgroups, h0 = (w.seg_item % hgroups) * kHeads;
    const int nh = min(kHeads, G - h0);                      // query heads of the item
    const int64_t qh = (int64_t)kvh * G + h0;                // the first of them
    float q[GP][N];
#pragma unroll
    for (int g = 0; g < GP; ++g)
      if (g < nh) load_row<N>(static_cast<const T*>(p.q) + (int64_t)w.seg_b * p.q_stride + (qh + g) * D + lane * N, q[g]);
      else
#pragma unroll
        for (int c = 0; c < N; ++c) q[g][c] = 0.f;
    float o[GP][N] = {};
    float m = -INFINITY, l = 0.f;            // of head lane % GP
    const int k_end = (int)min64((int64_t)w.seg_len, w.t1 * kTile);
    const int32_t* table = p.table + (int64_t)w.seg_b * p.max_pages;
    for (int64_t kb = w.t0 * kTile + warp * KB; kb < k_end; kb += kWarps * KB) {
      float s[32], v[KB][N];
      int64_t off_mine = -1;                 // lanes 0..KB-1: the element offset of key kb + lane
      if (lane < KB && kb + lane < k_end) {
        const int key = (int)kb + lane;
        const int id = table[key / ps];
        if (id >= 0 && id < p.pool.n_pages)
          off_mine = (((int64_t)id * p.pool.H + kvh) * ps + key % ps) * D;
        else
          flag_device(status, kDevCheck);
      }
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        const int64_t off = __shfl_sync(0xffffffffu, off_mine, j);
        float k[N];
#pragma unroll
        for (int c = 0; c < N; ++c) k[c] = v[j][c] = 0.f;
        if (off >= 0) {
          load_row<N>(static_cast<const T*>(p.pool.k) + off + lane * N, k);
          load_row<N>(static_cast<const T*>(p.pool.v) + off + lane * N, v[j]);
        }
#pragma unroll
        for (int g = 0; g < GP; ++g) {
          float d = 0.f;
#pragma unroll
          for (int c = 0; c < N; ++c) d = fmaf(q[g][c], k[c], d);
          s[j * GP + g] = d;
        }
      }
      float sc = butterfly(s) * scale_log2;
      if (kb + my_key >= k_end) sc = -INFINITY;
      float mx = sc;
#pragma unroll
      for (int d = GP; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      const float mn = fmaxf(m, mx);
      const float base = mn == -INFINITY ? 0.f : mn;   // a batch of -inf scores alone adds nothing
      const float corr = exp2f(m - base), pr = exp2f(sc - base);
      float ps_ = pr;
#pragma unroll
      for (int d = GP; d < 32; d <<= 1) ps_ += __shfl_xor_sync(0xffffffffu, ps_, d);
      l = l * corr + ps_;
      m = mn;
#pragma unroll
      for (int g = 0; g < GP; ++g) {
        const float cg = __shfl_sync(0xffffffffu, corr, g);
#pragma unroll
        for (int c = 0; c < N; ++c) o[g][c] *= cg;
      }
#pragma unroll
      for (int j = 0; j < KB; ++j) {
#pragma unroll
        for (int g = 0; g < GP; ++g) {
          const float pj = __shfl_sync(0xffffffffu, pr, j * GP + g);
#pragma unroll
          for (int c = 0; c < N; ++c) o[g][c] = fmaf(pj, v[j][c], o[g][c]);
        }
      }
    }
    // merge the warps
#pragma unroll
    for (int g = 0; g < GP; ++g)
#pragma unroll
      for (int c = 0; c < N; ++c) red_o[warp][g][lane * N + c] = o[g][c];
    if (lane < GP) {
      red_m[warp][lane] = m;
      red_l[warp][lane] = l;
    }
    __syncthreads();
    const bool whole = w.begins && w.ends;
    const int slot = 2 * blockIdx.x + (w.begins ? 1 : 0);
    for (int e = threadIdx.x; e < nh * D; e += kThreads) {
      const int g = e / D, c = e % D;
      float mm = red_m[0][g];
#pragma unroll
      for (int x = 1; x < kWarps; ++x) mm = fmaxf(mm, red_m[x][g]);
      const float base = mm == -INFINITY ? 0.f : mm;
      float ll = 0.f, oo = 0.f;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        const float f = exp2f(red_m[x][g] - base);
        ll += f * red_l[x][g];
        oo += f * red_o[x][g][c];
      }
      if (whole) {
        const int64_t h = qh + g;
        static_cast<T*>(p.o)[((int64_t)w.seg_b * p.H + h) * D + c] = from_f32<T>(oo / ll);
        if (p.lse && c == 0) p.lse[h * p.B + w.seg_b] = (mm + log2f(ll)) * 0.6931471805599453f;
      } else {
        part.o[((int64_t)slot * heads + g) * D + c] = oo;
        if (c == 0) {
          part.ml[((int64_t)slot * heads + g) * 2] = mm;
          part.ml[((int64_t)slot * heads + g) * 2 + 1] = ll;
        }
      }
    }
    if (w.begins && !w.ends) {
      open_id = (int64_t)w.seg_b * items + w.seg_item;
      open_parts = w.parts(plan, kExtra, blockIdx.x, gridDim.x);
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    part.id[2 * blockIdx.x] = open_id;
    part.id[2 * blockIdx.x + 1] = open_parts;
  }
}

// One CTA per (CTA of the split, head of an item): joins the item that CTA
// began and left unfinished, whose rest is the slots 0 of the CTAs after it.
// Four columns per thread; a row of threads takes every rows-th partial with
// a running maximum, then the rows are joined in order, so the result does
// not depend on scheduling.
template <typename T, int D>
__global__ void __launch_bounds__(256) paged_join_kernel(const PagedAttnProblem p, int ctas, int items, int heads,
                                                         int hgroups, int G) {
  constexpr int kLanes = D / 4, kRows = 256 / kLanes;
  __shared__ float4 red[kRows][kLanes];
  __shared__ float red_m[kRows], red_l[kRows];
  pdl_trigger();                                  // the next call may set itself up; it waits for this one's end
  pdl_wait();
  const int stride = min(heads, G);
  const PagedPartials part = paged_partials(p.workspace, ctas, stride);
  const int c0 = blockIdx.x, g = blockIdx.y;
  const longlong2 open = *reinterpret_cast<const longlong2*>(part.id + 2 * c0);
  const int64_t id = open.x;
  if (id < 0) return;
  const int n = (int)open.y;                       // partial i: slot 1 of c0, then slot 0 of c0 + i
  const int b = (int)(id / items), item = (int)(id % items);
  const int h0 = (item % hgroups) * heads;
  if (h0 + g >= G) return;
  const int64_t h = (int64_t)(item / hgroups) * G + h0 + g;
  const int lane = threadIdx.x % kLanes, row = threadIdx.x / kLanes;
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  // kBatch partials' loads at a time: one latency for up to kBatch * kRows of them
  constexpr int kBatch = 4;
  for (int i0 = row; i0 < n; i0 += kBatch * kRows) {
    float2 ml[kBatch];
    float4 v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kRows;
      ml[k] = make_float2(-INFINITY, 0.f);
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) {
        const int64_t s = (int64_t)(i == 0 ? 2 * c0 + 1 : 2 * (c0 + i)) * stride + g;
        ml[k] = *reinterpret_cast<const float2*>(part.ml + s * 2);
        v[k] = *reinterpret_cast<const float4*>(part.o + s * D + 4 * lane);
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float mn = fmaxf(m, ml[k].x), base = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(m - base), fi = exp2f(ml[k].x - base);
      m = mn;
      l = l * f + ml[k].y * fi;
      o.x = o.x * f + v[k].x * fi;
      o.y = o.y * f + v[k].y * fi;
      o.z = o.z * f + v[k].z * fi;
      o.w = o.w * f + v[k].w * fi;
    }
  }
  red[row][lane] = o;
  if (lane == 0) {
    red_m[row] = m;
    red_l[row] = l;
  }
  __syncthreads();
  if (row != 0) return;
  const int rows = min(n, kRows);
  for (int r = 1; r < rows; ++r) m = fmaxf(m, red_m[r]);
  const float base = m == -INFINITY ? 0.f : m;
  l = 0.f;
  o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int r = 0; r < rows; ++r) {
    const float f = exp2f(red_m[r] - base);
    const float4 v = red[r][lane];
    l += red_l[r] * f;
    o.x += v.x * f;
    o.y += v.y * f;
    o.z += v.z * f;
    o.w += v.w * f;
  }
  T* out = static_cast<T*>(p.o) + ((int64_t)b * p.H + h) * D + 4 * lane;
  out[0] = from_f32<T>(o.x / l);
  out[1] = from_f32<T>(o.y / l);
  out[2] = from_f32<T>(o.z / l);
  out[3] = from_f32<T>(o.w / l);
  if (p.lse && lane == 0) p.lse[h * p.B + b] = (m + log2f(l)) * 0.6931471805599453f;
}

template <typename T>
cudaError_t join(const PagedAttnProblem& p, int ctas, int items, int heads, cudaStream_t s) {
  const int G = p.H / p.pool.H, hgroups = items / p.pool.H;
  const dim3 grid(ctas, min(heads, G)), block(256);
  switch (p.d) {
    case 32: return launch_pdl(paged_join_kernel<T, 32>, grid, block, 0, s, p, ctas, items, heads, hgroups, G);
    case 64: return launch_pdl(paged_join_kernel<T, 64>, grid, block, 0, s, p, ctas, items, heads, hgroups, G);
    default: return launch_pdl(paged_join_kernel<T, 128>, grid, block, 0, s, p, ctas, items, heads, hgroups, G);
  }
}

template <typename T, int D, int GP>
cudaError_t run(const PagedAttnProblem& p, unsigned int* status, cudaStream_t s) {
  const int G = p.H / p.pool.H, hgroups = (G + kHeads - 1) / kHeads, items = p.pool.H * hgroups;
  const int ctas = min(2 * sm_count(), kPagedMaxCtas);
  const bool whole = paged_whole_items(p, sizeof(T));
  cudaError_t e = launch_pdl(paged_attn_kernel<T, D, GP>, dim3(ctas), dim3(kThreads), 0, s, p, items, hgroups, G,
                             whole, p.scale * 1.4426950408889634f, status);
  if (e != cudaSuccess || whole) return e;
  return launch_paged_join(sizeof(T) == 2 ? NT_BF16 : NT_F32, p, ctas, items, kHeads, s);
}

template <typename T, int D>
cudaError_t run_g(const PagedAttnProblem& p, unsigned int* status, cudaStream_t s) {
  const int G = p.H / p.pool.H;
  if (G == 1) return run<T, D, 1>(p, status, s);
  if (G == 2) return run<T, D, 2>(p, status, s);
  if (G <= 4) return run<T, D, 4>(p, status, s);
  return run<T, D, 8>(p, status, s);
}

template <typename T>
cudaError_t run_d(const PagedAttnProblem& p, unsigned int* status, cudaStream_t s) {
  switch (p.d) {
    case 32: return run_g<T, 32>(p, status, s);
    case 64: return run_g<T, 64>(p, status, s);
    case 128: return run_g<T, 128>(p, status, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

size_t paged_attn_workspace_bytes(int G, int d) {
  const size_t heads = min(G, kPagedMaxHeads);
  return ((size_t)kPagedMaxCtas * 2 * (sizeof(int64_t) + heads * (2 + (size_t)d) * sizeof(float)) + 255) &
         ~(size_t)255;
}

cudaError_t launch_paged_join(nt_dtype dt, const PagedAttnProblem& p, int ctas, int items, int heads,
                              cudaStream_t s) {
  return dt == NT_BF16 ? join<bf16>(p, ctas, items, heads, s) : join<float>(p, ctas, items, heads, s);
}

cudaError_t launch_paged_attn(nt_dtype dt, const PagedAttnProblem& p, unsigned int* status, cudaStream_t s) {
  if (p.B == 0) return cudaSuccess;
  if (paged_attn_short_chosen(dt, p)) return launch_paged_attn_short(dt, p, status, s);
  if (paged_attn_tma_supported(p)) return launch_paged_attn_tma(dt, p, status, s);
  return dt == NT_BF16 ? run_d<bf16>(p, status, s) : run_d<float>(p, status, s);
}

}  // namespace nt
