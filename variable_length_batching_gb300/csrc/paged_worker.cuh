// What a warp does with 16 keys of a paged cache and up to HP query heads of
// one key head: scores, a running softmax, outputs.  Used by the kernels of
// paged attention, which differ in how the keys come to shared memory.
#pragma once

#include "tc_ptx.cuh"

namespace nt {
namespace paged {

using namespace tc;

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// v[i] summed over the lanes, for i = this lane: halves the array and the
// lane distance together (31 shuffles for 32 sums).
__device__ __forceinline__ float butterfly32(float (&v)[32]) {
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

template <int N>
__device__ __forceinline__ void load_row(const float* p, float (&x)[N]) {
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

// A warp's query rows, running maxima, sums and outputs.  Its keys lie in a
// stage: rows of kRow bytes, the values `side` bytes behind the keys; bf16
// rows in boxes of `box` keys by 64 columns with the 128-byte swizzle (64-byte
// for D = 32), fp32 rows plain.
template <typename T, int D, int HP>
struct Worker;

// bf16: matrix products.
template <int D, int HP>
struct Worker<bf16, D, HP> {
  static constexpr int NT = HP / 8;
  static constexpr uint32_t kRow = D * 2;
  static constexpr int kRedStride = D + 4;      // floats: keeps the result's writes conflict-free
  static constexpr uint32_t kBoxRow = D < 64 ? D * 2 : 128;   // bytes of a key in a box's columns
  uint32_t qa[D / 16][4];
  float m[NT], l[NT], o[NT][D / 16][4];
  int g, tq;                       // accumulator row (head) and column pair
  uint32_t hs, row_off, xr;        // a box's next 64 columns; this lane's row in the matrix loads; its swizzle
  int box, slice;

  __device__ __forceinline__ uint32_t row_at(int r) const {
    return (uint32_t)(r / box) * box * kRow + r % box * kBoxRow;
  }
  __device__ __forceinline__ Worker(int box_, int slice_) {
    const int lane = threadIdx.x & 31;
    g = lane >> 2;
    tq = lane & 3;
    box = box_;
    slice = slice_;
    hs = box * 128;
    const int mrow = slice * 16 + ((lane >> 4) << 3) + (lane & 7);
    row_off = row_at(mrow);
    const int sw = D < 64 ? (mrow >> 1) & 3 : mrow & 7;
    xr = (((lane >> 3) & 1) ^ sw) << 4;
  }
  // nh query rows, contiguous, in shared or global memory
  __device__ __forceinline__ void load_q(const void* rows, int nh) {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(rows);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      qa[ks][0] = g < nh ? q[(g * D + ks * 16) / 2 + tq] : 0u;
      qa[ks][2] = g < nh ? q[(g * D + ks * 16 + 8) / 2 + tq] : 0u;
      qa[ks][1] = NT == 2 && g + 8 < nh ? q[((g + 8) * D + ks * 16) / 2 + tq] : 0u;
      qa[ks][3] = NT == 2 && g + 8 < nh ? q[((g + 8) * D + ks * 16 + 8) / 2 + tq] : 0u;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n] = -INFINITY;
      l[n] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[n][i][c] = 0.f;
    }
  }
  // the first `left` of the slice's keys
  __device__ __forceinline__ void tile(uint8_t* stage, uint32_t side, int left, float scale_log2) {
    const int lane = threadIdx.x & 31;
    const uint32_t kbase = smem_u32(stage), vbase = kbase + side;
    if (left < 16) {
      // rows behind the last key may hold anything: zeros instead, so that a probability of 0 adds 0
      for (int e = lane; e < (16 - left) * (D / 8); e += 32) {
        const int row = slice * 16 + left + e / (D / 8), ch = e % (D / 8);
        *reinterpret_cast<uint4*>(stage + side + row_at(row) + (ch >> 3) * hs + (ch & 7) * 16) =
            make_uint4(0, 0, 0, 0);
      }
      __syncwarp();
    }
    // two chains for each eight keys
    float s[2][4] = {}, s2[2][4] = {};
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t kb[4];
      ldsm4(kbase + (ks >> 2) * hs + row_off + ((((uint32_t)ks & 3) << 5) ^ xr), kb);
      mma16816(ks & 1 ? s2[0] : s[0], qa[ks], kb[0], kb[1]);
      mma16816(ks & 1 ? s2[1] : s[1], qa[ks], kb[2], kb[3]);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      s[0][c] += s2[0][c];
      s[1][c] += s2[1][c];
    }
    uint32_t pb[NT][2];
    float corr[NT];
    bool moved = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float v[4] = {s[0][2 * n] * scale_log2, s[0][2 * n + 1] * scale_log2, s[1][2 * n] * scale_log2,
                    s[1][2 * n + 1] * scale_log2};
      if (left < 16) {
        if (2 * tq >= left) v[0] = -INFINITY;
        if (2 * tq + 1 >= left) v[1] = -INFINITY;
        if (8 + 2 * tq >= left) v[2] = -INFINITY;
        if (9 + 2 * tq >= left) v[3] = -INFINITY;
      }
      float mx = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m[n], mx);
      const float base = mn == -INFINITY ? 0.f : mn;
      moved |= mn > m[n];
      corr[n] = ex2_approx(m[n] - base);
      m[n] = mn;
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = ex2_approx(v[c] - base);
      l[n] = l[n] * corr[n] + (v[0] + v[1]) + (v[2] + v[3]);
      pb[n][0] = pack_bf16x2(v[0], v[1]);
      pb[n][1] = pack_bf16x2(v[2], v[3]);
    }
    if (__any_sync(0xffffffffu, moved)) {
      // the output's columns are heads 2 tq and 2 tq + 1: their factors sit in those rows' lanes
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float c0 = __shfl_sync(0xffffffffu, corr[n], 8 * tq);
        const float c1 = __shfl_sync(0xffffffffu, corr[n], 8 * tq + 4);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          o[n][i][0] *= c0;
          o[n][i][1] *= c1;
          o[n][i][2] *= c0;
          o[n][i][3] *= c1;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      uint32_t va[4];
      ldsm4_t(vbase + (i >> 2) * hs + row_off + ((((uint32_t)i & 3) << 5) ^ xr), va);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma16816(o[n][i], va, pb[n][0], pb[n][1]);
    }
    if (left < 16) fence_async_shared();       // the zeros, before the next copy into this stage
  }
  // The whole item's output from this warp alone: rows [nh][D] at o, gathered
  // in `rows` (shared, HP x D); and, after it, the heads' log-sum-exps: this
  // lane's head (lanes with tq = 0), and head + 8.
  __device__ __forceinline__ void finish(bf16* rows, bf16* o_, int nh) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      l[n] += __shfl_xor_sync(0xffffffffu, l[n], 1);
      l[n] += __shfl_xor_sync(0xffffffffu, l[n], 2);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float inv = 1.f / __shfl_sync(0xffffffffu, l[n], 8 * tq + 4 * c);
        bf16* r = rows + (n * 8 + 2 * tq + c) * D + g;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          r[i * 16] = __float2bfloat16_rn(o[n][i][c] * inv);
          r[i * 16 + 8] = __float2bfloat16_rn(o[n][i][c + 2] * inv);
        }
      }
    }
    __syncwarp();
    for (int e = lane; e < nh * (D / 8); e += 32)
      reinterpret_cast<uint4*>(o_)[e] = reinterpret_cast<const uint4*>(rows)[e];
    __syncwarp();
  }
  __device__ __forceinline__ int head_of_lane() const { return tq == 0 ? g : -1; }
  __device__ __forceinline__ float head_lse() const { return (m[0] + log2f(l[0])) * 0.6931471805599453f; }
  __device__ __forceinline__ float head_lse1() const { return (m[NT - 1] + log2f(l[NT - 1])) * 0.6931471805599453f; }
  // the warp's result: maxima and sums (-1: no keys, nothing to add), outputs [HP][kRedStride]
  __device__ __forceinline__ void result(float* rm, float* rl, float* ro, int nh, bool active) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      l[n] += __shfl_xor_sync(0xffffffffu, l[n], 1);
      l[n] += __shfl_xor_sync(0xffffffffu, l[n], 2);
      if (tq == 0) {
        rm[n * 8 + g] = m[n];
        rl[n * 8 + g] = active ? l[n] : -1.f;
      }
    }
    if (!active) return;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int h = n * 8 + 2 * tq + c;
        if (h >= nh) continue;
        float* r = ro + h * kRedStride + g;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          r[i * 16] = o[n][i][c];
          r[i * 16 + 8] = o[n][i][c + 2];
        }
      }
  }
};

// fp32: D / 32 elements of a row per lane, batches of KB keys x HP heads.
template <int D, int HP>
struct Worker<float, D, HP> {
  static constexpr uint32_t kRow = D * 4;
  static constexpr int kRedStride = D + 4;
  static constexpr int N = D / 32, KB = 32 / HP < 16 ? 32 / HP : 16;
  float q[HP][N], o[HP][N];
  float m, l;                      // of head lane % HP
  int slice;

  __device__ __forceinline__ Worker(int, int slice_) : slice(slice_) {}
  __device__ __forceinline__ void load_q(const void* rows, int nh) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 0; h < HP; ++h) {
#pragma unroll
      for (int c = 0; c < N; ++c) q[h][c] = o[h][c] = 0.f;
      if (h < nh) load_row<N>(reinterpret_cast<const float*>(rows) + h * D + lane * N, q[h]);
    }
    m = -INFINITY;
    l = 0.f;
  }
  __device__ __forceinline__ void tile(const uint8_t* stage, uint32_t side, int left, float scale_log2) {
    const int lane = threadIdx.x & 31;
    const float* k = reinterpret_cast<const float*>(stage) + slice * 16 * D + lane * N;
    const float* v = k + side / 4;
#pragma unroll
    for (int b = 0; b < 16; b += KB) {
      if (b >= left) break;
      float s[32];
#pragma unroll
      for (int j = 0; j < 32 / HP; ++j) {
        float x[N];
#pragma unroll
        for (int c = 0; c < N; ++c) x[c] = 0.f;
        if (j < KB && b + j < left) load_row<N>(k + (b + j) * D, x);
#pragma unroll
        for (int h = 0; h < HP; ++h) {
          float d = 0.f;
#pragma unroll
          for (int c = 0; c < N; ++c) d = fmaf(q[h][c], x[c], d);
          s[j * HP + h] = d;
        }
      }
      float sc = butterfly32(s) * scale_log2;        // of key b + lane / HP, head lane % HP
      if (lane / HP >= KB || b + lane / HP >= left) sc = -INFINITY;
      float mx = sc;
#pragma unroll
      for (int d = HP; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      const float mn = fmaxf(m, mx);
      const float base = mn == -INFINITY ? 0.f : mn;
      const float corr = exp2f(m - base), pr = exp2f(sc - base);
      float sum = pr;
#pragma unroll
      for (int d = HP; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      const bool moved = mn > m;
      l = l * corr + sum;
      m = mn;
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int h = 0; h < HP; ++h) {
          const float ch = __shfl_sync(0xffffffffu, corr, h);
#pragma unroll
          for (int c = 0; c < N; ++c) o[h][c] *= ch;
        }
      }
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        if (b + j >= left) break;                    // rows behind the last key may hold anything
        float x[N];
        load_row<N>(v + (b + j) * D, x);
#pragma unroll
        for (int h = 0; h < HP; ++h) {
          const float pj = __shfl_sync(0xffffffffu, pr, j * HP + h);
#pragma unroll
          for (int c = 0; c < N; ++c) o[h][c] = fmaf(pj, x[c], o[h][c]);
        }
      }
    }
  }
  __device__ __forceinline__ void finish(float*, float* o_, int nh) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 0; h < HP; ++h) {
      const float inv = 1.f / __shfl_sync(0xffffffffu, l, h);
      if (h < nh) {
#pragma unroll
        for (int c = 0; c < N; ++c) o_[h * D + lane * N + c] = o[h][c] * inv;
      }
    }
  }
  __device__ __forceinline__ int head_of_lane() const {
    const int lane = threadIdx.x & 31;
    return lane < HP ? lane : -1;
  }
  __device__ __forceinline__ float head_lse() const { return (m + log2f(l)) * 0.6931471805599453f; }
  __device__ __forceinline__ void result(float* rm, float* rl, float* ro, int nh, bool active) {
    const int lane = threadIdx.x & 31;
    if (lane < HP) {
      rm[lane] = m;
      rl[lane] = active ? l : -1.f;
    }
    if (!active) return;
#pragma unroll
    for (int h = 0; h < HP; ++h)
      if (h < nh)
#pragma unroll
        for (int c = 0; c < N; ++c) ro[h * kRedStride + lane * N + c] = o[h][c];
  }
};

__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}

// A warp copies 16 keys and their values into a slot that its Worker (box 16)
// reads, row by row with cp.async, so any page size will do.  `row`: of lane
// i < 16 the pool's row of key i, negative for zeros.
template <typename T, int D>
__device__ __forceinline__ void copy_slice(uint32_t dst, const void* k, const void* v, int64_t row) {
  constexpr uint32_t kRow = D * sizeof(T);
  constexpr int kChunks = kRow / 16;                                // 16-byte words of a row
  constexpr int kRowsAt = 32 / kChunks < 1 ? 1 : 32 / kChunks;      // rows a warp copies at once
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int r0 = 0; r0 < 16; r0 += kRowsAt) {
    const int r = r0 + (kRowsAt > 1 ? lane / kChunks : 0), c = lane % kChunks;
    const int64_t at = __shfl_sync(0xffffffffu, row, r);
    // bf16: 64-column halves of 16 rows, swizzled as the worker reads them
    uint32_t to;
    if constexpr (sizeof(T) == 4) to = r * kRow + c * 16;
    else if constexpr (D == 32) to = r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    else to = (c >> 3) * 2048 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    const int64_t from = at < 0 ? 0 : at * kRow + c * 16;
    copy16_or_zero(dst + to, static_cast<const uint8_t*>(k) + from, at >= 0);
    copy16_or_zero(dst + 16 * kRow + to, static_cast<const uint8_t*>(v) + from, at >= 0);
  }
}

}  // namespace paged
}  // namespace nt
