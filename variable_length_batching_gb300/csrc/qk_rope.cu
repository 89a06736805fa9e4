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
// A CTA takes TB tokens: it forms their cosines and sines once in shared
// memory for all heads of q and k, then groups of LP lanes (two 8-element
// chunks each, so that a lane holds both halves of its pairs in either
// layout) take one (token, head) row at a time.  Everything between the load
// and the one rounding of the store is fp32.
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
};

struct Args {
  Side side[2];
  int64_t T;
  int d, rot, interleaved, B, tb;
  float eps, scale;
  const int32_t* cu;
  const int32_t* pos0;
  const int32_t* positions;
  const uint64_t* turns;
  float* partial;       // backward: [grid][2][d] sums for dgamma
  unsigned int* status;
};

// Position of token t; false (flagged) if the offsets do not place it.
__device__ bool token_position(const Args& a, int64_t t, int64_t& pos) {
  if (a.positions) {
    pos = a.positions[t];
    return true;
  }
  int lo = 0, hi = a.B - 1;          // last segment that starts at or before t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.cu[mid] <= t) lo = mid; else hi = mid - 1;
  }
  const int start = a.cu[lo];
  if (start > t || a.cu[lo + 1] <= t || start < 0) {
    flag_device(a.status, kDevCheck);
    return false;
  }
  pos = t - start + (a.pos0 ? a.pos0[lo] : 0);
  return true;
}

// Shared: ok[tb] (int), pos[tb] (int64), then the tile's table: pairs of
// (cos, sin) as float4 {c0, s0, c1, s1}, the four of a lane's eight pairs
// rot/16 apart, so that the lanes of a group read consecutive words.
struct Tile {
  int64_t* pos;
  int* ok;
  float4* cs;
};
__device__ __forceinline__ Tile tile_of(unsigned char* smem, const Args& a) {
  Tile s;
  s.pos = reinterpret_cast<int64_t*>(smem);
  s.ok = reinterpret_cast<int*>(smem + a.tb * 8);
  s.cs = reinterpret_cast<float4*>(smem + ((a.tb * 12 + 15) & ~15));
  return s;
}

// With nothing to rotate the positions are not read (and may be NULL).
__device__ void fill_tile(const Args& a, const Tile& s, int64_t t0, int n) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    int64_t p = 0;
    s.ok[i] = a.rot == 0 || token_position(a, t0 + i, p);
    s.pos[i] = p;
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

// Rotate a lane's two chunks (dir = 1 forward, -1 transposed).
__device__ __forceinline__ void rotate(float* xa, float* xb, const float4* cs, int lanes, int i, bool interleaved,
                                       float dir) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float4 w = cs[q * lanes + i];
    const float c0 = w.x, s0 = w.y * dir, c1 = w.z, s1 = w.w * dir;
    if (interleaved) {     // pairs 2q and 2q + 1 of the lane: chunk a holds the first four, chunk b the rest
      float* x = (q < 2 ? xa : xb) + (q & 1) * 4;
      const float a0 = x[0], b0 = x[1], a1 = x[2], b1 = x[3];
      x[0] = a0 * c0 - b0 * s0;
      x[1] = a0 * s0 + b0 * c0;
      x[2] = a1 * c1 - b1 * s1;
      x[3] = a1 * s1 + b1 * c1;
    } else {
      const float a0 = xa[2 * q], b0 = xb[2 * q], a1 = xa[2 * q + 1], b1 = xb[2 * q + 1];
      xa[2 * q] = a0 * c0 - b0 * s0;
      xb[2 * q] = a0 * s0 + b0 * c0;
      xa[2 * q + 1] = a1 * c1 - b1 * s1;
      xb[2 * q + 1] = a1 * s1 + b1 * c1;
    }
  }
}

template <int LP>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int m = LP / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// Columns of lane i's two chunks.
__device__ __forceinline__ void lane_columns(const Args& a, int i, int& ca, int& cb) {
  if (!a.interleaved && 16 * i < a.rot) {
    ca = 8 * i;
    cb = (a.rot >> 1) + 8 * i;
  } else {
    ca = 16 * i;
    cb = 16 * i + 8;
  }
}

template <typename T, int LP>
__global__ void __launch_bounds__(kThreads) rope_fwd_kernel(const Args a) {
  extern __shared__ __align__(16) unsigned char smem[];
  const Tile s = tile_of(smem, a);
  const int64_t t0 = (int64_t)blockIdx.x * a.tb;
  const int n = (int)min64(a.tb, a.T - t0);
  fill_tile(a, s, t0, n);
  const int i = threadIdx.x % LP, g = threadIdx.x / LP;
  const bool lane_on = 16 * i < a.d, rotated = 16 * i < a.rot;
  const int lanes = a.rot >> 4;
  int ca, cb;
  lane_columns(a, i, ca, cb);
#pragma unroll 1
  for (int sd = 0; sd < 2; ++sd) {
    const Side& p = a.side[sd];
    if (p.H == 0) continue;
    float ga[8], gb[8];
    const bool norm = p.gamma != nullptr;
    if (norm && lane_on) {
      load8(p.gamma + ca, ga);
      load8(p.gamma + cb, gb);
    }
    const int items = n * p.H;
    // whole warps stay in the loop together (the group sums are shuffles)
    for (int it0 = 0; it0 < items; it0 += kThreads / LP) {
      const int it = it0 + g;
      const int tok = it / p.H, h = it - tok * p.H;
      const bool on = it < items && lane_on && s.ok[tok];
      float xa[8] = {}, xb[8] = {};
      const T* x = static_cast<const T*>(p.x) + (t0 + tok) * p.xs + (int64_t)h * a.d;
      if (on) {
        load8(x + ca, xa);
        load8(x + cb, xb);
      }
      if (norm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += xa[e] * xa[e] + xb[e] * xb[e];
        const float r = rsqrtf(group_sum<LP>(ss) / (float)a.d + a.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          xa[e] *= r * ga[e];
          xb[e] *= r * gb[e];
        }
      }
      if (on) {
        if (rotated) rotate(xa, xb, s.cs + tok * (a.rot >> 2), lanes, i, a.interleaved, 1.f);
        T* o = static_cast<T*>(p.out) + (t0 + tok) * p.os + (int64_t)h * a.d;
        store8(o + ca, xa);
        store8(o + cb, xb);
      }
    }
  }
}

template <typename T, int LP>
__global__ void __launch_bounds__(kThreads) rope_bwd_kernel(const Args a) {
  extern __shared__ __align__(16) unsigned char smem[];
  const Tile s = tile_of(smem, a);
  const int i = threadIdx.x % LP, g = threadIdx.x / LP;
  const bool lane_on = 16 * i < a.d, rotated = 16 * i < a.rot;
  const int lanes = a.rot >> 4;
  int ca, cb;
  lane_columns(a, i, ca, cb);
  float acc[2][16] = {};
  for (int64_t t0 = (int64_t)blockIdx.x * a.tb; t0 < a.T; t0 += (int64_t)gridDim.x * a.tb) {
    const int n = (int)min64(a.tb, a.T - t0);
    __syncthreads();                         // the tile of the step before is read out
    fill_tile(a, s, t0, n);
#pragma unroll
    for (int sd = 0; sd < 2; ++sd) {
      const Side& p = a.side[sd];
      if (p.H == 0) continue;
      const bool norm = p.gamma != nullptr;
      const int items = n * p.H;
      for (int it0 = 0; it0 < items; it0 += kThreads / LP) {
        const int it = it0 + g;
        const int tok = it / p.H, h = it - tok * p.H;
        const bool on = it < items && lane_on && s.ok[tok];
        float ga[8] = {}, gb[8] = {};        // upstream, then rotated back
        if (on) {
          const T* u = static_cast<const T*>(p.up) + (t0 + tok) * p.us + (int64_t)h * a.d;
          load8(u + ca, ga);
          load8(u + cb, gb);
          if (rotated) rotate(ga, gb, s.cs + tok * (a.rot >> 2), lanes, i, a.interleaved, -1.f);
        }
        if (norm) {
          float xa[8] = {}, xb[8] = {};
          if (on) {
            const T* x = static_cast<const T*>(p.x) + (t0 + tok) * p.xs + (int64_t)h * a.d;
            load8(x + ca, xa);
            load8(x + cb, xb);
          }
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss += xa[e] * xa[e] + xb[e] * xb[e];
          const float r = rsqrtf(group_sum<LP>(ss) / (float)a.d + a.eps);
          float hx = 0.f;
          if (on) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              xa[e] *= r;
              xb[e] *= r;
              acc[sd][e] += ga[e] * xa[e];
              acc[sd][8 + e] += gb[e] * xb[e];
              ga[e] *= p.gamma[ca + e];
              gb[e] *= p.gamma[cb + e];
              hx += ga[e] * xa[e] + gb[e] * xb[e];
            }
          }
          const float m = group_sum<LP>(hx) / (float)a.d;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            ga[e] = r * (ga[e] - xa[e] * m);
            gb[e] = r * (gb[e] - xb[e] * m);
          }
        }
        if (on) {
          T* o = static_cast<T*>(p.out) + (t0 + tok) * p.os + (int64_t)h * a.d;
          store8(o + ca, ga);
          store8(o + cb, gb);
        }
      }
    }
  }
  if (!a.partial) return;
  // dgamma: the groups of a warp by shuffle, the warps through shared memory
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);          // [kWarps][d], one side at a time
  const int warp = threadIdx.x / 32;
#pragma unroll
  for (int sd = 0; sd < 2; ++sd) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float v = acc[sd][e];
#pragma unroll
      for (int m = 16; m >= LP; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
      if ((threadIdx.x & 31) < LP && lane_on) red[warp * a.d + (e < 8 ? ca + e : cb + e - 8)] = v;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.d; c += kThreads) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += red[w * a.d + c];
      a.partial[((int64_t)blockIdx.x * 2 + sd) * a.d + c] = v;
    }
    __syncthreads();
  }
}

// dgamma[side][c] = the sum of the CTAs' partials, in CTA order within each
// of eight strides, then across the strides.
__global__ void __launch_bounds__(256) rope_dgamma_kernel(const float* partial, int parts, int d, float* dq_gamma,
                                                          float* dk_gamma) {
  __shared__ float red[8][32];
  const int c = blockIdx.x * 32 + threadIdx.x % 32, w = threadIdx.x / 32, sd = blockIdx.y;
  float* out = sd ? dk_gamma : dq_gamma;
  if (!out) return;
  float v = 0.f;
  if (c < d)
    for (int p = w; p < parts; p += 8) v += partial[((int64_t)p * 2 + sd) * d + c];
  red[w][threadIdx.x % 32] = v;
  __syncthreads();
  if (w == 0 && c < d) {
    for (int k = 1; k < 8; ++k) v += red[k][threadIdx.x];
    out[c] = v;
  }
}

int group_lanes(int d) {
  int lp = 1;
  while (16 * lp < d) lp <<= 1;
  return lp;
}

template <typename T, int LP>
cudaError_t run(const Args& a, bool bwd, int grid, size_t smem, cudaStream_t s) {
  if (bwd) rope_bwd_kernel<T, LP><<<grid, kThreads, smem, s>>>(a);
  else rope_fwd_kernel<T, LP><<<grid, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t run_lp(const Args& a, bool bwd, int grid, size_t smem, cudaStream_t s) {
  switch (group_lanes(a.d)) {
    case 1: return run<T, 1>(a, bwd, grid, smem, s);
    case 2: return run<T, 2>(a, bwd, grid, smem, s);
    case 4: return run<T, 4>(a, bwd, grid, smem, s);
    case 8: return run<T, 8>(a, bwd, grid, smem, s);
    default: return run<T, 16>(a, bwd, grid, smem, s);
  }
}

}  // namespace

size_t qk_rope_bwd_workspace_bytes(int d) { return (size_t)kRopeMaxParts * 2 * (size_t)d * sizeof(float); }

cudaError_t launch_qk_rope(nt_dtype dt, const RopeProblem& p, bool bwd, float* workspace, unsigned int* status,
                           cudaStream_t s) {
  const int LP = group_lanes(p.d);
  Args a = {};
  a.side[0] = {p.q, p.dq_out, p.q_out, p.q_stride, p.dq_out_stride, p.q_out_stride, p.q_gamma, p.H_q};
  a.side[1] = {p.k, p.dk_out, p.k_out, p.k_stride, p.dk_out_stride, p.k_out_stride, p.k_gamma, p.H_k};
  a.T = p.T;
  a.d = p.d;
  a.rot = p.rot_dim;
  a.interleaved = p.interleaved;
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
  // tokens per CTA: one while the tokens do not fill the SMs, at most 16
  const int sms = sm_count();
  int tb = 1;
  while (tb < 16 && p.T >= (int64_t)sms * 8 * tb * 2) tb <<= 1;
  a.tb = tb;
  const int64_t tiles = (p.T + tb - 1) / tb;
  size_t smem = (size_t)((tb * 12 + 15) & ~15) + (size_t)tb * (p.rot_dim / 4) * 16;
  int64_t grid = tiles;
  if (bwd) {
    grid = min64(tiles, min64(kRopeMaxParts, (int64_t)sms * 4));
    const size_t red = (size_t)kWarps * p.d * sizeof(float);
    if (smem < red) smem = red;
  }
  (void)LP;
  cudaError_t e = cudaSuccess;
  if (p.T > 0)
    e = dt == NT_BF16 ? run_lp<bf16>(a, bwd, (int)grid, smem, s) : run_lp<float>(a, bwd, (int)grid, smem, s);
  if (e != cudaSuccess || !bwd || !norm) return e;
  rope_dgamma_kernel<<<dim3((p.d + 31) / 32, 2), 256, 0, s>>>(workspace, p.T > 0 ? (int)grid : 0, p.d, p.dq_gamma,
                                                            p.dk_gamma);
  return cudaGetLastError();
}

}  // namespace nt
