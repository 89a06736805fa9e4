// Attention of drafted tokens over a paged cache: which kernel a call takes,
// and the join of partial results.
//
//   o_i,h = sum_x softmax_x(scale q_i,h . k_x) v_x
// over the positions x that new token i of a sequence sees: all before the new
// tokens, and of these the ones that the tree's mask names (without one:
// itself and those before it).
#include "draft_plan.cuh"
#include "tc_ptx.cuh"

namespace nt {
namespace {

// Joins the items that CTAs of the split began and left unfinished: the rest of
// CTA c0's is the slots 0 of the CTAs after it.  A lane has four columns of a
// row, so a warp takes 128 / D rows at once; partials are added in order with a
// running maximum, kBatch loads at a time.  L2's latency bounds it.  kShared:
// a CTA's warps share rows, each with an eighth of their partials, and
// blockIdx.x counts the unfinished items; for few rows of few items, which have
// many partials each.
constexpr int kJoinWarps = 8;

template <int D>
struct JoinRow {
  static constexpr int kBatch = 4;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  __device__ __forceinline__ void add(float mi, float li, const float4& v) {
    const float mn = fmaxf(m, mi), base = mn == -INFINITY ? 0.f : mn;
    const float f = exp2f(m - base), fi = exp2f(mi - base);
    m = mn;
    l = l * f + li * fi;
    acc.x = acc.x * f + v.x * fi;
    acc.y = acc.y * f + v.y * fi;
    acc.z = acc.z * f + v.z * fi;
    acc.w = acc.w * f + v.w * fi;
  }
  // Partials [from, to) of a row at these columns: partial i is slot 1 of c0, then slot 0 of c0 + i.
  __device__ __forceinline__ void partials(const DraftPartials& part, int c0, int rows, int row, int col, int from,
                                           int to) {
    for (int i0 = from; i0 < to; i0 += kBatch) {
      float2 ml[kBatch];
      float4 v[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k;
        ml[k] = make_float2(-INFINITY, 0.f);
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < to) {
          const int64_t s = (int64_t)(i == 0 ? 2 * c0 + 1 : 2 * (c0 + i)) * rows + row;
          ml[k] = *reinterpret_cast<const float2*>(part.ml + s * 2);
          v[k] = *reinterpret_cast<const float4*>(part.o + s * D + col);
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) add(ml[k].x, ml[k].y, v[k]);
    }
  }
};

template <typename T, int D, bool kShared>
__global__ void __launch_bounds__(kJoinWarps * 32, kShared ? 4 : 6)
    draft_join_kernel(const DraftBatch a, int ctas, int rows, void* workspace, T* o, float* lse) {
  constexpr int kLanes = D / 4, kAtOnce = 32 / kLanes;
  __shared__ int which;
  __shared__ float4 sv[kJoinWarps][32];
  __shared__ float2 sml[kJoinWarps][32];
  pdl_wait();
  pdl_trigger();
  const DraftPartials part = draft_partials(workspace, ctas, rows);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = lane % kLanes * 4;
  int c0 = blockIdx.x;
  if constexpr (kShared) {                          // the blockIdx.x-th CTA that left one
    constexpr int kMost = kPagedMaxCtas / (kJoinWarps * 32);
    __shared__ int counts[kMost * kJoinWarps];
    unsigned int left[kMost];
#pragma unroll
    for (int k = 0; k < kMost; ++k) {
      const int c = k * kJoinWarps * 32 + threadIdx.x;
      left[k] = __ballot_sync(0xffffffffu, c < ctas && part.open[c].x >= 0);
      if (lane == 0) counts[k * kJoinWarps + warp] = __popc(left[k]);
    }
    if (threadIdx.x == 0) which = -1;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMost; ++k) {
      int rank = __popc(left[k] & ((1u << lane) - 1));
      for (int w = 0; w < k * kJoinWarps + warp; ++w) rank += counts[w];
      if ((left[k] >> lane & 1) && rank == (int)blockIdx.x) which = k * kJoinWarps * 32 + threadIdx.x;
    }
    __syncthreads();
    c0 = which;
    if (c0 < 0) return;
  }
  const int4 open = part.open[c0];
  if (open.x < 0 || open.x >= a.B) return;
  const DraftSeq seq = draft_seq(a, open.x, nullptr);
  const DraftItem it = draft_item(a, seq.n, open.y, open.z);
  const int n = min(open.w, ctas - c0), all = it.ni * it.nh;
  const int row = (kShared ? blockIdx.y : blockIdx.y * kJoinWarps + warp) * kAtOnce + lane / kLanes;
  JoinRow<D> r;
  if constexpr (kShared) {
    const int share = (n + kJoinWarps - 1) / kJoinWarps;
    if (row < all) r.partials(part, c0, rows, row, col, min(n, warp * share), min(n, (warp + 1) * share));
    sv[warp][lane] = r.acc;
    sml[warp][lane] = make_float2(r.m, r.l);
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int w = 1; w < kJoinWarps; ++w) r.add(sml[w][lane].x, sml[w][lane].y, sv[w][lane]);
    }
    if (warp > 0) return;
  } else if (row < all) {
    r.partials(part, c0, rows, row, col, 0, n);
  }
  if (row >= all) return;
  const int i = it.i0 + row / it.nh, h = it.kvh * a.G + it.h0 + row % it.nh;
  const int64_t t = (int64_t)seq.first + i;
  const bool any = draft_sees_any(a, seq, i);
  T* to = o + (t * a.H + h) * D + col;
  const float out[4] = {any ? r.acc.x / r.l : 0.f, any ? r.acc.y / r.l : 0.f, any ? r.acc.z / r.l : 0.f,
                        any ? r.acc.w / r.l : 0.f};
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint2*>(to) = make_uint2(tc::pack_bf16x2(out[0], out[1]), tc::pack_bf16x2(out[2], out[3]));
  } else {
    *reinterpret_cast<float4*>(to) = make_float4(out[0], out[1], out[2], out[3]);
  }
  if (lse && col == 0) lse[(int64_t)h * a.T + t] = any ? (r.m + log2f(r.l)) * 0.6931471805599453f : -INFINITY;
}

template <typename T, int D>
cudaError_t join_d(const DraftBatch& a, int ctas, int rows, void* ws, void* o, float* lse, cudaStream_t s) {
  constexpr int kAtOnce = 128 / D;
  const int most = min(a.tokens, a.max_new) * a.heads;     // rows of any item
  const int64_t items = (int64_t)a.B * draft_items_most(a);
  T* out = static_cast<T*>(o);
  // Sixteen partials or more to an item, in rows that leave warps without one.
  // Two items of 48 and more partials, 53 rows of d = 128: the call 21.8 us,
  // 18.4 so; below sixteen the search for the item costs as much (12 items of 13: 0.8 us more).
  const int64_t shared = items * ((most + kAtOnce - 1) / kAtOnce);
  if (items * 16 <= ctas && shared <= 4 * ctas)
    return launch_pdl(draft_join_kernel<T, D, true>, dim3((unsigned)items, (most + kAtOnce - 1) / kAtOnce),
                      dim3(kJoinWarps * 32), 0, s, a, ctas, rows, ws, out, lse);
  const int y = (most + kAtOnce * kJoinWarps - 1) / (kAtOnce * kJoinWarps);
  return launch_pdl(draft_join_kernel<T, D, false>, dim3(ctas, y), dim3(kJoinWarps * 32), 0, s, a, ctas, rows, ws, out,
                    lse);
}
template <typename T>
cudaError_t join(const DraftBatch& a, int d, int ctas, int rows, void* ws, void* o, float* lse, cudaStream_t s) {
  switch (d) {
    case 32: return join_d<T, 32>(a, ctas, rows, ws, o, lse, s);
    case 64: return join_d<T, 64>(a, ctas, rows, ws, o, lse, s);
    default: return join_d<T, 128>(a, ctas, rows, ws, o, lse, s);
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
  a.light = groups > 1 ? a.tokens / groups : 0;
  // units are counted in tiles of 32 keys at least, with at most 16 more to an item
  a.few = p.B <= kPlanFew && (double)p.B * draft_items_most(a) * ((double)a.cap / 32 + 17) * draft_weight_most(a) < 2e9;
  a.status = status;
  return a;
}

cudaError_t launch_draft_join(nt_dtype dt, const DraftBatch& a, int d, int ctas, int rows, void* workspace, void* o,
                              float* lse, cudaStream_t s) {
  return dt == NT_BF16 ? join<bf16>(a, d, ctas, rows, workspace, o, lse, s)
                       : join<float>(a, d, ctas, rows, workspace, o, lse, s);
}

namespace {

// Rates of a kernel that deals tiles of keys out to `ctas` CTAs, and the
// estimated time (us) of a call: what it costs whatever it does, and a CTA's
// share of the tiles and of the items.
struct Rates {
  double first, tile, item;
};
double split_us(const DraftProblem& p, int rows, int groups, int keys, int ctas, const Rates& r) {
  const DraftBatch a = draft_batch(p, rows, groups, nullptr);
  const double items = p.B * draft_items_mean(p, a), tiles = items * (draft_mean_keys(p, a) / keys + 0.5);
  return r.first + fmax(tiles / ctas, 1) * r.tile + items / ctas * r.item;
}

}  // namespace

double draft_mean_keys(const DraftProblem& p, const DraftBatch& a) { return p.B == 1 ? a.cap : 0.4 * a.cap; }
double draft_items_mean(const DraftProblem& p, const DraftBatch& a) {
  const double heads = (double)a.Hkv * a.hgroups, n = (double)p.T / p.B, most = (p.max_new + a.tokens - 1) / a.tokens;
  return heads * (most <= 1 || n >= p.max_new ? most : fmin(most, fmax(1, n / a.tokens + 0.75)));
}

// The call takes the kernel with the least estimated time.  Lengths are on the
// device, so the estimates go by what the host knows: the tables' size (one
// sequence fills its table, several 0.4 of it), the tokens and the heads.  The
// rates were fitted to 4,000 random calls of up to 128 sequences whose tables are
// as wide as their longest sequence; there this choice cost 1 to 3% over the best
// kernel of each (geometric mean by type and width; without the spread kernel 6 to
// 16%, the tensor-memory kernel 10 to 12 at d = 64 and 128, the slices 1.5 at d = 32
// and 0.6 at 64, the rows kernel 6 to 11 in bf16 and 51 to 75 in fp32).  On 900
// other such calls the final kernels' choice costs 0.5%, at most 83%; on 300 of
// them with tables for 131,072 positions, as a table on the device may be, 13% and
// at most 89% (one context of 777 keys, eight tokens, 12 heads of 64: 6.6 us, and
// 10.5 in the wide table).
cudaError_t launch_draft_attn(nt_dtype dt, const DraftProblem& p, unsigned int* status, cudaStream_t s) {
  constexpr Rates kRowsBf16[3] = {{7.15, 1.47, 2.75}, {7.55, 2.0, 2.8}, {8.1, 3.1, 3.9}};
  constexpr Rates kRowsF32[3][3] = {{{7.65, 1.72, 3.8}, {7.65, 2.34, 3.8}, {7.65, 4.1, 3.8}},
                                    {{8.6, 2.74, 4.5}, {8.6, 4.0, 4.5}, {8.6, 7.4, 4.5}},
                                    {{10.6, 3.1, 5.8}, {10.6, 4.0, 5.8}, {10.6, 7.1, 5.8}}};
  constexpr Rates kTcRates[2][2] = {{{10.9, 1.06, 2.7}, {14.4, 2.2, 5.5}}, {{11.2, 1.66, 2.4}, {17.7, 3.1, 6.2}}};
  constexpr Rates kSliceRates[2][3] = {{{7.5, 0.525, 2.4}, {7.5, 0.93, 2.4}, {7.5, 1.64, 2.4}},
                                       {{8.45, 0.39, 2.6}, {8.45, 0.61, 2.6}, {8.45, 1.53, 2.6}}};
  const int sms = min(sm_count(), kPagedMaxCtas), w = p.d == 32 ? 0 : p.d == 64 ? 1 : 2;
  const int64_t rows = (int64_t)p.max_new * (p.H / p.pool.H);
  const int group = rows <= 16 ? 0 : rows <= 32 ? 1 : 2;
  int cluster;
  double best = draft_spread_us(dt, p, &cluster);
  enum { kSpread, kRows, kTc, kSlices } kernel = kSpread;
  auto consider = [&](decltype(kernel) k, double us) {
    if (us >= best) return;
    best = us;
    kernel = k;
  };
  if (dt == NT_BF16) consider(kRows, split_us(p, 64, 1, 64, 2 * sms, kRowsBf16[w]));
  else consider(kRows, split_us(p, 16 << group, 1, 64, p.d == 128 ? sms : 2 * sms, kRowsF32[w][group]));
  if (draft_tc_supported(dt, p)) {
    const bool wide = p.d == 128;
    Rates r = kTcRates[wide][rows > 128];
    // two row tiles: sequences that need but one, at most those whose tokens leave the average below it, take less
    // (draft_plan.cuh)
    if (rows > 128)
      r.tile *= 1 - (1 - (double)kLight / kHeavy) * fmax(0, 1 - (double)p.T / p.B / (128 / min(128, p.H / p.pool.H)));
    consider(kTc, split_us(p, 128, 1 + (rows > 128), 128, sms, r));
  }
  if (draft_slices_supported(dt, p))
    consider(kSlices, split_us(p, 16 << group, 1, w ? 64 : 128, sms, kSliceRates[w][group]));
  switch (kernel) {
    case kSpread: return launch_draft_spread(dt, p, cluster, status, s);
    case kTc: return launch_draft_tc(p, status, s);
    case kSlices: return launch_draft_slices(p, status, s);
    default: return launch_draft_rows(dt, p, status, s);
  }
}

}  // namespace nt
