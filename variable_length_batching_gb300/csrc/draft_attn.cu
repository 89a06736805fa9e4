// Attention of drafted tokens over a paged cache: which kernel a call takes,
// and the join of partial results.
//
//   o_i,h = sum_x softmax_x(scale q_i,h . k_x) v_x
// over the positions x that new token i of a sequence sees: all before the new
// tokens, and of these the ones that the tree's mask names (without one:
// itself and those before it).
#include "draft_plan.cuh"

namespace nt {
namespace {

// One CTA per (CTA of the split, eight rows): joins the item that CTA began
// and left unfinished, whose rest is the slots 0 of the CTAs after it.  A warp
// has a row, a lane D / 32 columns of it; partials are added in order with a
// running maximum, eight loads at a time.
template <typename T, int D>
__global__ void __launch_bounds__(256) draft_join_kernel(const DraftBatch a, int ctas, int rows, void* workspace,
                                                         T* o, float* lse) {
  constexpr int kCols = D / 32, kBatch = 8;
  pdl_wait();
  pdl_trigger();
  const DraftPartials part = draft_partials(workspace, ctas, rows);
  const int c0 = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 open = part.open[c0];
  if (open.x < 0 || open.x >= a.B) return;
  const DraftSeq seq = draft_seq(a, open.x, nullptr);
  const DraftItem it = draft_item(a, seq.n, open.y, open.z);
  const int row = blockIdx.y * 8 + warp;
  if (row >= it.ni * it.nh) return;
  const int n = min(open.w, ctas - c0);            // partial i: slot 1 of c0, then slot 0 of c0 + i
  float m = -INFINITY, l = 0.f, acc[kCols] = {};
  for (int i0 = 0; i0 < n; i0 += kBatch) {
    float2 ml[kBatch];
    float v[kBatch][kCols];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k;
      ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int c = 0; c < kCols; ++c) v[k][c] = 0.f;
      if (i < n) {
        const int64_t s = (int64_t)(i == 0 ? 2 * c0 + 1 : 2 * (c0 + i)) * rows + row;
        ml[k] = *reinterpret_cast<const float2*>(part.ml + s * 2);
        const float* from = part.o + s * D + kCols * lane;
        if constexpr (kCols == 4) {
          const float4 x = *reinterpret_cast<const float4*>(from);
          v[k][0] = x.x, v[k][1] = x.y, v[k][2] = x.z, v[k][3] = x.w;
        } else if constexpr (kCols == 2) {
          const float2 x = *reinterpret_cast<const float2*>(from);
          v[k][0] = x.x, v[k][1] = x.y;
        } else {
          v[k][0] = *from;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float mn = fmaxf(m, ml[k].x), base = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(m - base), fi = exp2f(ml[k].x - base);
      m = mn;
      l = l * f + ml[k].y * fi;
#pragma unroll
      for (int c = 0; c < kCols; ++c) acc[c] = acc[c] * f + v[k][c] * fi;
    }
  }
  const int i = it.i0 + row / it.nh, h = it.kvh * a.G + it.h0 + row % it.nh;
  const int64_t t = (int64_t)seq.first + i;
  const bool any = draft_sees_any(a, seq, i);
  T* to = o + (t * a.H + h) * D + kCols * lane;
#pragma unroll
  for (int c = 0; c < kCols; ++c) to[c] = from_f32<T>(any ? acc[c] / l : 0.f);
  if (lse && lane == 0) lse[(int64_t)h * a.T + t] = any ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

template <typename T>
cudaError_t join(const DraftBatch& a, int d, int ctas, int rows, void* ws, void* o, float* lse, cudaStream_t s) {
  const int most = min(a.tokens, a.max_new) * a.heads;     // rows of any item
  const dim3 grid(ctas, (most + 7) / 8), block(256);
  T* out = static_cast<T*>(o);
  switch (d) {
    case 32: return launch_pdl(draft_join_kernel<T, 32>, grid, block, 0, s, a, ctas, rows, ws, out, lse);
    case 64: return launch_pdl(draft_join_kernel<T, 64>, grid, block, 0, s, a, ctas, rows, ws, out, lse);
    default: return launch_pdl(draft_join_kernel<T, 128>, grid, block, 0, s, a, ctas, rows, ws, out, lse);
  }
}

}  // namespace

size_t draft_workspace_bytes(int d) {
  constexpr size_t kRows = 256;
  return ((size_t)kPagedMaxCtas * (sizeof(int4) + 2 * kRows * (2 + (size_t)d) * sizeof(float)) + 255) & ~(size_t)255;
}

DraftBatch draft_batch(const DraftProblem& p, int rows, int groups, unsigned int* status) {
  DraftBatch a;
  a.cu = p.cu;
  a.lengths = p.lengths;
  a.table = p.table;
  a.bits = p.bits;
  a.B = p.B;
  a.max_new = p.max_new;
  a.words = max(1, (p.max_new + 63) / 64);
  a.T = p.T;
  a.cap = min64((int64_t)p.max_pages * p.pool.page_size, 0x7fffffff);
  a.max_pages = p.max_pages;
  a.page_size = p.pool.page_size;
  a.n_pages = p.pool.n_pages;
  a.H = p.H;
  a.G = p.H / p.pool.H;
  a.Hkv = p.pool.H;
  a.heads = min(a.G, rows);
  a.hgroups = (a.G + a.heads - 1) / a.heads;
  a.tokens = max(1, rows / a.heads) * groups;
  // units are counted in tiles of 32 keys at least, with at most 16 more to an item
  a.few = p.B <= kPlanFew && (double)p.B * draft_items_most(a) * ((double)a.cap / 32 + 17) < 2e9;
  a.status = status;
  return a;
}

cudaError_t launch_draft_join(nt_dtype dt, const DraftBatch& a, int d, int ctas, int rows, void* workspace, void* o,
                              float* lse, cudaStream_t s) {
  return dt == NT_BF16 ? join<bf16>(a, d, ctas, rows, workspace, o, lse, s)
                       : join<float>(a, d, ctas, rows, workspace, o, lse, s);
}

cudaError_t launch_draft_attn(nt_dtype dt, const DraftProblem& p, unsigned int* status, cudaStream_t s) {
  const int64_t rows = (int64_t)p.max_new * (p.H / p.pool.H);
  const bool tc = draft_tc_supported(dt, p);
  if (draft_slices_supported(dt, p) && (rows <= 64 || !tc)) return launch_draft_slices(p, status, s);
  return tc ? launch_draft_tc(p, status, s) : launch_draft_rows(dt, p, status, s);
}

}  // namespace nt
