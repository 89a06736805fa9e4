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

__device__ __forceinline__ float4 lds4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// A warp's query rows, running maxima, sums and outputs.  Its keys lie in a
// stage, the values `side` bytes behind the keys, in boxes of `box` keys by
// 128 bytes of their rows (64 for bf16 rows of 32) with the 128-byte (64-byte)
// swizzle.  kScratch: bytes of shared memory a warp needs beside the stage.
// kKeepsQ: whether the query rows stay where they are read from (then in
// shared memory) until the item's end.
template <typename T, int D, int HP>
struct Worker;

// bf16: matrix products.
template <int D, int HP>
struct Worker<bf16, D, HP> {
  static constexpr uint32_t kScratch = 0;
  static constexpr bool kKeepsQ = false;
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
  __device__ __forceinline__ Worker(int box_, int slice_, void*) {
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
  // Probabilities x, y >= 0 as the sums of two bf16, off by 2^-15 of them at
  // most (one bf16 would be off by 2^-8, which shows in the output).  The upper
  // part is the largest bf16 below the value, so that both are positive: an
  // infinite value in the cache gives the infinity that x times it is, and a
  // lower part of 0 or below would make it NaN.
  static __device__ __forceinline__ void split(float x, float y, uint32_t& hi, uint32_t& lo) {
    const uint32_t a = (max(__float_as_uint(x), 1u) - 1) & 0xffff0000u;
    const uint32_t b = (max(__float_as_uint(y), 1u) - 1) & 0xffff0000u;
    hi = __byte_perm(a, b, 0x7632);
    lo = pack_bf16x2(x - __uint_as_float(a), y - __uint_as_float(b));
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
    uint32_t pb[NT][2], pl[NT][2];
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
      split(v[0], v[1], pb[n][0], pl[n][0]);
      split(v[2], v[3], pb[n][1], pl[n][1]);
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
    // two column blocks at a time: a product does not wait for the one before it
#pragma unroll
    for (int i = 0; i < D / 16; i += 2) {
      uint32_t va[2][4];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        ldsm4_t(vbase + ((i + k) >> 2) * hs + row_off + ((((uint32_t)(i + k) & 3) << 5) ^ xr), va[k]);
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma16816(o[n][i + k], va[k], part ? pl[n][0] : pb[n][0], part ? pl[n][1] : pb[n][1]);
    }
    if (left < 16) fence_async_shared();       // the zeros, before the next copy into this stage
  }
  // The whole item's output from this warp alone: rows [nh][D] at o, gathered
  // in `rows` (shared, HP x D).
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
  // the heads' log-sum-exps, after finish
  __device__ __forceinline__ void store_lse(float* lse, int64_t stride, int nh) const {
#pragma unroll
    for (int n = 0; n < NT; ++n)
      if (tq == 0 && n * 8 + g < nh) lse[(n * 8 + g) * stride] = (m[n] + log2f(l[n])) * 0.6931471805599453f;
  }
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

// fp32, on the CUDA cores, in packed pairs.  Scores: a lane has one key and
// half of its columns against all heads, whose rows it reads as broadcasts;
// the halves are added, and each half of the warp keeps every other head.
// Outputs: a lane has four columns of all heads and every kGroups-th key, the
// probabilities read as broadcasts from the warp's scratch.  (Columns across the
// lanes and sums by shuffles take 31 shuffles for 32 scores, and one more for
// every probability and head: the ragged batch of 64 with 8 key heads of 64 and
// eight heads to each takes 102 us that way, 64 this, with d = 32 and one 49
// and 32.)
template <int D, int HP>
struct Worker<float, D, HP> {
  static constexpr uint32_t kScratch = 16 * HP * 4;
  static constexpr bool kKeepsQ = true;
  static constexpr uint32_t kRow = D * 4;
  static constexpr int kRedStride = D + 4;
  static constexpr int kMine = HP > 1 ? HP / 2 : 1;      // heads whose softmax this lane keeps: 2 i + half
  static constexpr int kGroups = 128 / D;                // keys side by side in the output's product
  static constexpr int kAcc = D == 128 ? 8 : 4;          // sums a dot product is split into
  float m[kMine], l[kMine], o[HP][4];                    // l: of this lane's keys
  const float* q;
  float* p;                                              // probabilities [16][HP]
  int slice, half, grp;
  uint32_t hs, k_off, k_x, v_off, v_x, v_jump;

  __device__ __forceinline__ Worker(int box, int slice_, void* scratch) : p(static_cast<float*>(scratch)), slice(slice_) {
    const int lane = threadIdx.x & 31, c = lane % (D / 4);
    half = lane >> 4;
    grp = lane / (D / 4);
    hs = box * 128;                                      // to a box's next 32 columns
    auto row_at = [&](int r) { return (uint32_t)(r / box) * box * kRow + r % box * 128; };
    k_off = row_at(slice * 16 + (lane & 15)) + half * (D / 64) * hs;
    k_x = ((D == 32 ? half * 4 : 0) ^ (lane & 7)) << 4;
    v_off = row_at(slice * 16) + (c >> 3) * hs + grp * 128;
    v_x = ((c & 7) ^ grp) << 4;
    v_jump = box == 8 ? 8 * kRow : 1024;                 // to the slice's second eight rows
  }
  // HP query rows (those behind the item's heads may hold anything)
  __device__ __forceinline__ void load_q(const void* rows, int) {
    q = static_cast<const float*>(rows);
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
#pragma unroll
    for (int h = 0; h < HP; ++h)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[h][c] = 0.f;
  }
  // kMasked: `see` has a bit for each key of the slice that rows 2 i + half see
  template <bool kMasked = false>
  __device__ __forceinline__ void tile(const uint8_t* stage, uint32_t side, int left, float scale_log2,
                                       const uint32_t* see = nullptr) {
    const int lane = threadIdx.x & 31, key = lane & 15;
    const uint32_t k = smem_u32(stage) + k_off, v = smem_u32(stage) + side + v_off, qs = smem_u32(q + half * (D / 2));
    float acc[HP][kAcc] = {};
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      const float4 x = lds4(k + (i >> 3) * hs + (((i & 7) << 4) ^ k_x));
      const int a = kAcc == 8 ? (i & 1) * 4 : 0;
#pragma unroll
      for (int h = 0; h < HP; ++h) {
        const float4 y = lds4(qs + (h * D + 4 * i) * 4);
        ffma2(x.x, x.y, y.x, y.y, acc[h][a], acc[h][a + 1], acc[h][a], acc[h][a + 1]);
        ffma2(x.z, x.w, y.z, y.w, acc[h][a + 2], acc[h][a + 3], acc[h][a + 2], acc[h][a + 3]);
      }
    }
    float s[HP];
#pragma unroll
    for (int h = 0; h < HP; ++h) {
      s[h] = (acc[h][0] + acc[h][1]) + (acc[h][2] + acc[h][3]);
      if constexpr (kAcc == 8) s[h] += (acc[h][4] + acc[h][5]) + (acc[h][6] + acc[h][7]);
    }
    float corr[kMine];
    bool moved = false;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      float t;
      if constexpr (HP == 1) t = s[0] + __shfl_xor_sync(0xffffffffu, s[0], 16);
      else t = (half ? s[2 * i + 1] : s[2 * i]) + __shfl_xor_sync(0xffffffffu, half ? s[2 * i] : s[2 * i + 1], 16);
      const bool seen = kMasked ? see[i] >> key & 1 : key < left;
      t = seen ? t * scale_log2 : -INFINITY;             // rows behind the last key may hold anything
      float mx = t;
#pragma unroll
      for (int x = 1; x < 16; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      const float mn = fmaxf(m[i], mx), base = mn == -INFINITY ? 0.f : mn;
      moved |= mn > m[i];
      corr[i] = exp2f(m[i] - base);
      m[i] = mn;
      const float pr = exp2f(t - base);
      l[i] = l[i] * corr[i] + pr;
      if (HP > 1 || half == 0) p[key * HP + (HP > 1 ? 2 * i + half : 0)] = pr;
    }
    __syncwarp();
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int h = 0; h < HP; ++h) {
        const float c = __shfl_sync(0xffffffffu, corr[h / 2], (h & 1) * 16);
        fmul2(o[h][0], o[h][1], c, c, o[h][0], o[h][1]);
        fmul2(o[h][2], o[h][3], c, c, o[h][2], o[h][3]);
      }
    }
#pragma unroll
    for (int j = 0; j < 16; j += kGroups) {              // key j + grp
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (j + grp < left) x = lds4(v + (j >> 3) * v_jump + (j & 7) * 128 + (v_x ^ ((j & 7) << 4)));
      float pr[HP];
      const float* pk = p + (j + grp) * HP;
      if constexpr (HP == 1) {
        pr[0] = *pk;
      } else if constexpr (HP == 2) {
        const float2 y = *reinterpret_cast<const float2*>(pk);
        pr[0] = y.x;
        pr[1] = y.y;
      } else {
#pragma unroll
        for (int h = 0; h < HP; h += 4) {
          const float4 y = *reinterpret_cast<const float4*>(pk + h);
          pr[h] = y.x;
          pr[h + 1] = y.y;
          pr[h + 2] = y.z;
          pr[h + 3] = y.w;
        }
      }
#pragma unroll
      for (int h = 0; h < HP; ++h) {
        ffma2(x.x, x.y, pr[h], pr[h], o[h][0], o[h][1], o[h][0], o[h][1]);
        ffma2(x.z, x.w, pr[h], pr[h], o[h][2], o[h][3], o[h][2], o[h][3]);
      }
    }
    __syncwarp();                                        // the scratch is free again
  }
  // the sums over all keys, in every lane that keeps or holds them
  __device__ __forceinline__ void gather() {
#pragma unroll
    for (int i = 0; i < kMine; ++i)
#pragma unroll
      for (int x = 1; x < 16; x <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
#pragma unroll
    for (int x = D / 4; x < 32; x <<= 1)
#pragma unroll
      for (int h = 0; h < HP; ++h)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[h][c] += __shfl_xor_sync(0xffffffffu, o[h][c], x);
  }
  __device__ __forceinline__ void finish(float*, float* o_, int nh) {
    const int lane = threadIdx.x & 31;
    gather();
#pragma unroll
    for (int h = 0; h < HP; ++h) {
      const float inv = 1.f / __shfl_sync(0xffffffffu, l[h / 2], (h & 1) * 16);
      if (h < nh && lane < D / 4)
        *reinterpret_cast<float4*>(o_ + h * D + 4 * lane) =
            make_float4(o[h][0] * inv, o[h][1] * inv, o[h][2] * inv, o[h][3] * inv);
    }
  }
  __device__ __forceinline__ void store_lse(float* lse, int64_t stride, int nh) const {
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int h = 2 * i + half;
      if ((threadIdx.x & 15) == 0 && h < nh) lse[h * stride] = (m[i] + log2f(l[i])) * 0.6931471805599453f;
    }
  }
  __device__ __forceinline__ void result(float* rm, float* rl, float* ro, int nh, bool active) {
    const int lane = threadIdx.x & 31;
    gather();
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int h = 2 * i + half;
      if ((lane & 15) == 0 && h < HP) {
        rm[h] = m[i];
        rl[h] = active ? l[i] : -1.f;
      }
    }
    if (!active || lane >= D / 4) return;
#pragma unroll
    for (int h = 0; h < HP; ++h)
      if (h < nh)
        *reinterpret_cast<float4*>(ro + h * kRedStride + 4 * lane) = make_float4(o[h][0], o[h][1], o[h][2], o[h][3]);
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
    uint32_t to;
    if constexpr (kRow == 64) to = r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    else to = (c >> 3) * 2048 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    const int64_t from = at < 0 ? 0 : at * kRow + c * 16;
    copy16_or_zero(dst + to, static_cast<const uint8_t*>(k) + from, at >= 0);
    copy16_or_zero(dst + 16 * kRow + to, static_cast<const uint8_t*>(v) + from, at >= 0);
  }
}

}  // namespace paged
}  // namespace nt
