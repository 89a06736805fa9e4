// Per-head RMS norm and rotary positions of packed queries and keys in one
// pass, and its backward.
//
// A token's position is its index within its cu_seqlens segment plus the
// segment's start (or is given).  The rotation angle of pair j at position p
// is 2 pi p u_j with u_j the pair's frequency in turns; u_j is held as a
// 64-bit fraction of a turn, so p * u_j modulo 2^64 is the exact fraction
// however far the position: no angle is ever formed in floating point before
// its whole turns are gone.  (An fp32 angle at p = 10^6 is off by 0.03 rad.)
//
//   y = x r gamma, r = 1 / sqrt(mean x^2 + eps)     (no gamma: y = x)
//   out_a = s (y_a cos - y_b sin),  out_b = s (y_a sin + y_b cos)
// and backward, with g the upstream gradient rotated back,
//   dgamma = sum g x r,  h = g gamma,  dx = r (h - x r mean(h x r)).
//
// Both directions are bound by HBM (about ten operations an element), so the
// layout is about keeping loads in flight.  A CTA serves q or k, for tb
// tokens.  Groups of LP lanes take one (token, head) row at a time, a lane
// two 8-element chunks: both halves of its eight pairs in either layout.  A
// group stays with one token and walks its heads, so the token's cosines and
// sines (formed once per CTA in shared memory), multiplied by gamma in the
// forward, stay in registers, and the rows of kBatch heads are requested
// before the first is used, in the forward before the table is even formed.
// Everything between the load and the one rounding of the store is fp32.
#include "nt_common.cuh"

namespace nt {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Device view of one side (q or k).
struct Side {
  const void* x;        // forward input; backward: the forward's input (norm only)
  const void* up;       // backward: upstream gradient
  void* out;            // forward output; backward: input gradient
  int64_t xs, us, os;   // token strides in elements
  const float* gamma;   // [d] or NULL (no norm)
  int H;
  int hg_log2;          // groups that share a token: 1 << hg_log2
  int ctas;             // CTAs that serve the side (the first side's come first)
};

struct Args {
  Side side[2];
  int64_t T;
  int d, rot, B;
  float inv_d, eps, scale;
  const int32_t* cu;
  const int32_t* pos0;
  const int32_t* positions;
  const uint64_t* turns;
  float* partial;       // backward: [CTAs][d] sums for dgamma
  unsigned int* status;
};

// Position of a token of segment b; false (flagged) if the offsets do not
// place the token there.
__device__ __forceinline__ bool position_in(const Args& a, int64_t t, int b, int64_t& pos) {
  const int start = a.cu[b];
  if (start > t || a.cu[b + 1] <= t || start < 0) {
    flag_device(a.status, kDevCheck);
    return false;
  }
  pos = t - start + (a.pos0 ? a.pos0[b] : 0);
  return true;
}

// Shared: pos[tb] (int64), ok[tb] (int), then the tile's table: pairs of
// (cos, sin) as float4 {c0, s0, c1, s1}, the four of a lane's eight pairs
// rot/16 apart, so that the lanes of a group read consecutive words.
struct Tile {
  int64_t* pos;
  int* ok;
  float4* cs;
};
__host__ __device__ __forceinline__ int table_offset(int tb) { return (tb * 12 + 15) & ~15; }
__device__ __forceinline__ Tile tile_of(unsigned char* smem, int tb) {
  Tile s;
  s.pos = reinterpret_cast<int64_t*>(smem);
  s.ok = reinterpret_cast<int*>(smem + tb * 8);
  s.cs = reinterpret_cast<float4*>(smem + table_offset(tb));
  return s;
}

// With nothing to rotate the positions are not read (and may be NULL).
__device__ void fill_tile(const Args& a, const Tile& s, int64_t t0, int n) {
  if (a.rot == 0 || a.positions) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
      s.ok[i] = 1;
      s.pos[i] = a.rot == 0 ? 0 : a.positions[t0 + i];
    }
  } else if (n <= kWarps) {
    // few tokens: one per warp, 32 probes a step (the latency of a search is
    // what a decoding step waits for: 2 steps instead of 8 for 256 segments)
    const int i = threadIdx.x >> 5;
    if (i < n) {
      const int b = segment_of_warp(a.cu, a.B, t0 + i);
      if ((threadIdx.x & 31) == 0) {
        int64_t p = 0;
        s.ok[i] = position_in(a, t0 + i, b, p);
        s.pos[i] = p;
      }
    }
  } else {
    for (int i = threadIdx.x; i < n; i += kThreads) {
      int64_t p = 0;
      s.ok[i] = position_in(a, t0 + i, segment_of_thread(a.cu, a.B, t0 + i), p);
      s.pos[i] = p;
    }
  }
  __syncthreads();
  const int quarter = a.rot >> 2;               // float4 words of one token
  const int lanes = a.rot >> 4;
  for (int e = threadIdx.x; e < n * quarter; e += kThreads) {
    const int tok = e / quarter, w = e - tok * quarter;
    const int q = w / lanes, i = w - q * lanes;  // word q of lane i: pairs 8 i + 2 q, + 1
    const uint64_t p = (uint64_t)s.pos[tok];
    float v[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint64_t frac = p * a.turns[8 * i + 2 * q + h];
      float sn, cn;
      sincospif((float)(int32_t)(frac >> 32) * 4.656612873077393e-10f, &sn, &cn);   // 2^-31: half turns
      v[2 * h] = cn * a.scale;
      v[2 * h + 1] = sn * a.scale;
    }
    s.cs[e] = make_float4(v[0], v[1], v[2], v[3]);
  }
  __syncthreads();
}

// A lane's place: its group's token within the tile and first head, and the
// columns of its two chunks.
template <int LP, bool kInter>
struct Lane {
  int i, tok, h0, hg, ca, cb;
  bool on, rotated;
  __device__ __forceinline__ Lane(const Args& a, const Side& p) {
    i = threadIdx.x % LP;
    const int g = threadIdx.x / LP;
    hg = 1 << p.hg_log2;
    tok = g >> p.hg_log2;
    h0 = g & (hg - 1);
    on = 16 * i < a.d;
    rotated = 16 * i < a.rot;
    if (!kInter && rotated) {
      ca = 8 * i;
      cb = (a.rot >> 1) + 8 * i;
    } else {
      ca = 16 * i;
      cb = 16 * i + 8;
    }
  }
  // cosines and sines of the lane's eight pairs (1 and 0 where nothing turns)
  __device__ __forceinline__ void angles(const Args& a, const Tile& s, float (&c)[8], float (&sn)[8]) const {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 w = rotated ? s.cs[tok * (a.rot >> 2) + q * (a.rot >> 4) + i] : make_float4(1.f, 0.f, 1.f, 0.f);
      c[2 * q] = w.x;
      sn[2 * q] = w.y;
      c[2 * q + 1] = w.z;
      sn[2 * q + 1] = w.w;
    }
  }
};
// Element indices (0..15: chunk a, then chunk b) of pair e's two parts.
template <bool kInter> __device__ constexpr int part_a(int e) { return kInter ? 2 * e : e; }
template <bool kInter> __device__ constexpr int part_b(int e) { return kInter ? 2 * e + 1 : e + 8; }

template <int LP>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int m = LP / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// One row's two chunks as loaded, and as fp32.
template <typename T> struct Raw;
template <> struct Raw<bf16> {
  uint4 a, b;
  __device__ __forceinline__ void load(const bf16* x, int ca, int cb) {
    a = *reinterpret_cast<const uint4*>(x + ca);
    b = *reinterpret_cast<const uint4*>(x + cb);
  }
  __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&v)[16]) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[2 * e] = __uint_as_float(w[e] << 16);
      v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  }
};
template <> struct Raw<float> {
  float4 a[4];
  __device__ __forceinline__ void load(const float* x, int ca, int cb) {
    a[0] = *reinterpret_cast<const float4*>(x + ca);
    a[1] = *reinterpret_cast<const float4*>(x + ca + 4);
    a[2] = *reinterpret_cast<const float4*>(x + cb);
    a[3] = *reinterpret_cast<const float4*>(x + cb + 4);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ void get(float (&v)[16]) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[4 * e] = a[e].x;
      v[4 * e + 1] = a[e].y;
      v[4 * e + 2] = a[e].z;
      v[4 * e + 3] = a[e].w;
    }
  }
};

template <typename T, int LP, bool kInter>
__global__ void __launch_bounds__(kThreads) rope_fwd_kernel(const Args a) {
  constexpr int kBatch = sizeof(T) == 2 ? 3 : 2;        // rows in flight per group
  extern __shared__ __align__(16) unsigned char smem[];
  const int sd = blockIdx.x >= a.side[0].ctas;
  const Side& p = a.side[sd];
  const Lane<LP, kInter> me(a, p);
  const int tb = kThreads / LP >> p.hg_log2;
  const int64_t t0 = (int64_t)(blockIdx.x - (sd ? a.side[0].ctas : 0)) * tb;
  const int n = (int)min64(tb, a.T - t0);
  const Tile s = tile_of(smem, tb);
  const bool here = me.on && me.tok < n;
  const T* x = static_cast<const T*>(p.x) + (t0 + me.tok) * p.xs;
  Raw<T> raw[kBatch];
  auto load = [&](int h) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      raw[k].zero();
      if (here && h + k * me.hg < p.H) raw[k].load(x + (int64_t)(h + k * me.hg) * a.d, me.ca, me.cb);
    }
  };
  pdl_wait();
  load(me.h0);
  fill_tile(a, s, t0, n);
  // pair e: out_a = r (x_a m[0] - x_b m[1]), out_b = r (x_a m[2] + x_b m[3])
  float m[8][4];
  const bool norm = p.gamma != nullptr;
  {
    float c[8], sn[8], gm[16];
    if (here) {
      me.angles(a, s, c, sn);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) c[e] = sn[e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) gm[e] = 1.f;
    if (norm && me.on) {
      Raw<float> g;
      g.load(p.gamma, me.ca, me.cb);
      g.get(gm);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float ga = gm[part_a<kInter>(e)], gb = gm[part_b<kInter>(e)];
      m[e][0] = ga * c[e];
      m[e][1] = gb * sn[e];
      m[e][2] = ga * sn[e];
      m[e][3] = gb * c[e];
    }
  }
  const bool write = here && s.ok[me.tok];
  T* o = static_cast<T*>(p.out) + (t0 + me.tok) * p.os;
  // the loop's bounds are the warp's: its groups may hold different first heads
  for (int hb = 0; hb < p.H; hb += kBatch * me.hg) {
    const int h = hb + me.h0;
    if (hb) load(h);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      float v[16];
      raw[k].get(v);
      float r = 1.f;
      if (norm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) ss = fmaf(v[e], v[e], ss);
        r = rsqrtf(group_sum<LP>(ss) * a.inv_d + a.eps);
      }
      float w[16];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int ia = part_a<kInter>(e), ib = part_b<kInter>(e);
        w[ia] = r * (v[ia] * m[e][0] - v[ib] * m[e][1]);
        w[ib] = r * (v[ia] * m[e][2] + v[ib] * m[e][3]);
      }
      if (write && h + k * me.hg < p.H) {
        T* y = o + (int64_t)(h + k * me.hg) * a.d;
        store8(y + me.ca, w);
        store8(y + me.cb, w + 8);
      }
    }
  }
}

template <typename T, int LP, bool kInter>
__global__ void __launch_bounds__(kThreads, 2) rope_bwd_kernel(const Args a) {
  constexpr int kBatch = sizeof(T) == 2 ? 2 : 1;
  extern __shared__ __align__(16) unsigned char smem[];
  const int sd = blockIdx.x >= a.side[0].ctas;
  const Side& p = a.side[sd];
  const Lane<LP, kInter> me(a, p);
  const int tb = kThreads / LP >> p.hg_log2;
  const Tile s = tile_of(smem, tb);
  const bool norm = p.gamma != nullptr;
  float gm[16], acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    gm[e] = 1.f;
    acc[e] = 0.f;
  }
  pdl_wait();
  pdl_trigger();
  if (norm && me.on) {
    Raw<float> g;
    g.load(p.gamma, me.ca, me.cb);
    g.get(gm);
  }
  for (int64_t t0 = (int64_t)(blockIdx.x - (sd ? a.side[0].ctas : 0)) * tb; t0 < a.T; t0 += (int64_t)p.ctas * tb) {
    const int n = (int)min64(tb, a.T - t0);
    const bool here = me.on && me.tok < n;
    const T* u = static_cast<const T*>(p.up) + (t0 + me.tok) * p.us;
    const T* x = static_cast<const T*>(p.x) + (t0 + me.tok) * p.xs;
    Raw<T> ru[kBatch], rx[kBatch];
    auto load = [&](int h) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        ru[k].zero();
        rx[k].zero();
        if (here && h + k * me.hg < p.H) {
          const int64_t at = (int64_t)(h + k * me.hg) * a.d;
          ru[k].load(u + at, me.ca, me.cb);
          if (norm) rx[k].load(x + at, me.ca, me.cb);
        }
      }
    };
    load(me.h0);
    __syncthreads();                         // the tile of the step before is read out
    fill_tile(a, s, t0, n);
    float c[8], sn[8];
    if (here) {
      me.angles(a, s, c, sn);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) c[e] = sn[e] = 0.f;
    }
    const bool write = here && s.ok[me.tok];
    T* o = static_cast<T*>(p.out) + (t0 + me.tok) * p.os;
    for (int hb = 0; hb < p.H; hb += kBatch * me.hg) {
      const int h = hb + me.h0;
      if (hb) load(h);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        float v[16], g[16];
        ru[k].get(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int ia = part_a<kInter>(e), ib = part_b<kInter>(e);
          g[ia] = v[ia] * c[e] + v[ib] * sn[e];
          g[ib] = v[ib] * c[e] - v[ia] * sn[e];
        }
        if (norm) {
          rx[k].get(v);
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 16; ++e) ss = fmaf(v[e], v[e], ss);
          const float r = rsqrtf(group_sum<LP>(ss) * a.inv_d + a.eps);
          float hx = 0.f;
          const float keep = write ? r : 0.f;        // a token in no segment adds nothing
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            v[e] *= keep;
            acc[e] = fmaf(g[e], v[e], acc[e]);
            g[e] *= gm[e];
            hx = fmaf(g[e], v[e], hx);
          }
          const float mean = group_sum<LP>(hx) * a.inv_d;
#pragma unroll
          for (int e = 0; e < 16; ++e) g[e] = r * (g[e] - v[e] * mean);
        }
        if (write && h + k * me.hg < p.H) {
          T* y = o + (int64_t)(h + k * me.hg) * a.d;
          store8(y + me.ca, g);
          store8(y + me.cb, g + 8);
        }
      }
    }
  }
  if (!a.partial) return;
  // dgamma: the groups of a warp by shuffle, the warps through shared memory
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);          // [kWarps][d]
  const int warp = threadIdx.x / 32;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float v = acc[e];
#pragma unroll
    for (int m = 16; m >= LP; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    if ((threadIdx.x & 31) < LP && me.on) red[warp * a.d + (e < 8 ? me.ca + e : me.cb + e - 8)] = v;
  }
  __syncthreads();
  for (int c = threadIdx.x; c < a.d; c += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += red[w * a.d + c];
    a.partial[(int64_t)blockIdx.x * a.d + c] = v;
  }
}

// dgamma of side blockIdx.y: the sum of its CTAs' partials, in CTA order
// within each of 32 strides, then across the strides.
__global__ void __launch_bounds__(1024) rope_dgamma_kernel(const float* partial, int parts_q, int parts_k, int d,
                                                           float* dq_gamma, float* dk_gamma) {
  __shared__ float red[32][33];
  const int col = threadIdx.x % 32, c = blockIdx.x * 32 + col, w = threadIdx.x / 32, sd = blockIdx.y;
  float* out = sd ? dk_gamma : dq_gamma;
  pdl_wait();
  if (!out) return;
  const int first = sd ? parts_q : 0, end = first + (sd ? parts_k : parts_q);
  float v = 0.f;
  if (c < d) {
#pragma unroll 4
    for (int p = first + w; p < end; p += 32) v += partial[(int64_t)p * d + c];
  }
  red[w][col] = v;
  __syncthreads();
  // warp w sums column w of the strides
  v = red[col][w];
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  if (col == 0 && blockIdx.x * 32 + w < d) out[blockIdx.x * 32 + w] = v;
}

int group_lanes(int d) {
  int lp = 1;
  while (16 * lp < d) lp <<= 1;
  return lp;
}

template <typename T, int LP, bool kInter>
cudaError_t run(const Args& a, bool bwd, int grid, size_t smem, cudaStream_t s) {
  return launch_pdl(bwd ? rope_bwd_kernel<T, LP, kInter> : rope_fwd_kernel<T, LP, kInter>, dim3(grid), dim3(kThreads),
                    smem, s, a);
}

template <typename T, bool kInter>
cudaError_t run_lp(const Args& a, bool bwd, int grid, size_t smem, cudaStream_t s) {
  switch (group_lanes(a.d)) {
    case 1: return run<T, 1, kInter>(a, bwd, grid, smem, s);
    case 2: return run<T, 2, kInter>(a, bwd, grid, smem, s);
    case 4: return run<T, 4, kInter>(a, bwd, grid, smem, s);
    case 8: return run<T, 8, kInter>(a, bwd, grid, smem, s);
    default: return run<T, 16, kInter>(a, bwd, grid, smem, s);
  }
}

}  // namespace

size_t qk_rope_bwd_workspace_bytes(int d) { return (size_t)kRopeMaxParts * (size_t)d * sizeof(float); }

cudaError_t launch_qk_rope(nt_dtype dt, const RopeProblem& p, bool bwd, float* workspace, unsigned int* status,
                           cudaStream_t s) {
  Args a = {};
  a.side[0] = {p.q, p.dq_out, p.q_out, p.q_stride, p.dq_out_stride, p.q_out_stride, p.q_gamma, p.H_q, 0, 0};
  a.side[1] = {p.k, p.dk_out, p.k_out, p.k_stride, p.dk_out_stride, p.k_out_stride, p.k_gamma, p.H_k, 0, 0};
  a.T = p.T;
  a.d = p.d;
  a.rot = p.rot_dim;
  a.inv_d = 1.f / p.d;
  a.B = p.B;
  a.eps = p.eps;
  a.scale = p.rot_scale;
  a.cu = p.cu;
  a.pos0 = p.pos0;
  a.positions = p.positions;
  a.turns = p.turns;
  a.status = status;
  const bool norm = p.q_gamma || p.k_gamma;
  a.partial = bwd && norm ? workspace : nullptr;
  const int groups = kThreads / group_lanes(p.d), sms = sm_count();
  size_t smem = bwd ? (size_t)kWarps * p.d * sizeof(float) : 0;
  for (Side& sd : a.side) {
    if (sd.H == 0 || p.T == 0) continue;
    // Groups per token: few, so that a group walks three heads or more with
    // one token's angles, unless the CTAs would then not fill the SMs twice.
    int lg = 0;
    while ((2 << lg) <= groups && (2 << lg) * 3 <= sd.H) ++lg;
    while ((2 << lg) <= groups && (1 << lg) < sd.H && p.T < (int64_t)2 * sms * (groups >> lg)) ++lg;
    const int tb = groups >> lg;
    const int64_t tiles = (p.T + tb - 1) / tb;
    sd.hg_log2 = lg;
    // The backward's CTAs stay (their sums of dgamma are what is added up at
    // the end): four per SM between the sides, by their heads.
    sd.ctas = (int)(bwd ? max64(1, min64(tiles, (int64_t)sms * 4 * sd.H / (p.H_q + p.H_k))) : tiles);
    const size_t need = (size_t)table_offset(tb) + (size_t)tb * (p.rot_dim / 4) * 16;
    if (smem < need) smem = need;
  }
  const int grid = a.side[0].ctas + a.side[1].ctas;
  cudaError_t e = cudaSuccess;
  if (grid > 0) {
    if (dt == NT_BF16)
      e = p.interleaved ? run_lp<bf16, true>(a, bwd, grid, smem, s) : run_lp<bf16, false>(a, bwd, grid, smem, s);
    else
      e = p.interleaved ? run_lp<float, true>(a, bwd, grid, smem, s) : run_lp<float, false>(a, bwd, grid, smem, s);
  }
  if (e != cudaSuccess || !bwd || !norm) return e;
  return launch_pdl(rope_dgamma_kernel, dim3((p.d + 31) / 32, 2), dim3(1024), 0, s, (const float*)workspace,
                    a.side[0].ctas, a.side[1].ctas, p.d, p.dq_gamma, p.dk_gamma);
}

}  // namespace nt
