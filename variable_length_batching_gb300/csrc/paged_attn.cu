// Attention of one new token per sequence over a paged key/value cache: which
// kernel a call takes, and the join of the tile kernel's partial results.
//
//   o_h = sum_j softmax_j(scale q_h . k_j) v_j over the sequence's j < len,
// query head h reading key head h / G, in one pass over the keys with a
// running maximum and sum.
#include "paged_plan.cuh"

namespace nt {
namespace {

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

// The kernel with the least estimated time, by the sizes of the tables.
cudaError_t launch_paged_attn(nt_dtype dt, const PagedAttnProblem& p, unsigned int* status, cudaStream_t s) {
  if (p.B == 0) return cudaSuccess;
  int cluster = 1;
  const double apart = paged_attn_short_us(dt, p), tiles = paged_attn_tma_us(dt, p);
  const double spread = paged_attn_spread_us(dt, p, &cluster);
  if (apart <= tiles && apart <= spread) return launch_paged_attn_short(dt, p, status, s);
  if (spread < tiles) return launch_paged_attn_spread(dt, p, cluster, status, s);
  return launch_paged_attn_tma(dt, p, status, s);
}

}  // namespace nt
