// What the threads of the general kernel for drafted tokens do with a tile of
// 64 keys and up to 64 rows: scores, a running softmax, outputs.
#pragma once

#include "draft_plan.cuh"
#include "paged_worker.cuh"

namespace nt {
namespace draft {

using namespace paged;

__device__ __forceinline__ void cp_async16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait0() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait1() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

// Place of 16-byte chunk c of row r, so that eight rows' equal chunks, and a
// row's eight neighbouring ones, lie in different banks.
template <uint32_t kRow>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
  const int x = kRow >= 128 ? r & 7 : (r >> 1) & 3;
  return (uint32_t)r * kRow + ((c ^ x) << 4);
}

// Values of a chunk that are not finite become 0; true if there were any.
template <typename T>
__device__ __forceinline__ bool clear_bad(uint8_t* chunk) {
  uint4 v = *reinterpret_cast<const uint4*>(chunk);
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (sizeof(T) == 4) {
      if ((w[i] & 0x7f800000u) == 0x7f800000u) any = true, w[i] = 0;
    } else {
      if ((w[i] & 0x7f80u) == 0x7f80u) any = true, w[i] &= 0xffff0000u;
      if ((w[i] & 0x7f800000u) == 0x7f800000u) any = true, w[i] &= 0x0000ffffu;
    }
  }
  if (any) *reinterpret_cast<uint4*>(chunk) = make_uint4(w[0], w[1], w[2], w[3]);
  return any;
}
__device__ __forceinline__ float if_bad(float v) { return fabsf(v) <= 3.402823466e38f ? 0.f : v; }

// The value of a row that sees no key is 0, its log-sum-exp -infinity.
__device__ __forceinline__ float row_lse(float m, float l, bool any) {
  return any ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

template <typename T, int D>
struct Rows;

// bf16: warp w has rows 16 w to 16 w + 15; a lane two of them, g and g + 8.
template <int D>
struct Rows<bf16, D> {
  uint32_t qa[D / 16][4];
  float m[2], l[2], o[D / 8][4];
  int g, tq, row0;

  __device__ __forceinline__ explicit Rows(void*) {
    const int lane = threadIdx.x & 31;
    g = lane >> 2;
    tq = lane & 3;
    row0 = (threadIdx.x >> 5) * 16;
  }
  __device__ __forceinline__ void load_q(const bf16* q, int64_t stride, int64_t token, int head, int ni, int nh) {
    const uint32_t* at[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = row0 + g + 8 * r;
      at[r] = row < ni * nh ? reinterpret_cast<const uint32_t*>(q + (token + row / nh) * stride +
                                                               (int64_t)(head + row % nh) * D)
                            : nullptr;
      m[r] = -INFINITY;
      l[r] = 0.f;
    }
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      qa[ks][0] = at[0] ? at[0][ks * 8 + tq] : 0u;
      qa[ks][1] = at[1] ? at[1][ks * 8 + tq] : 0u;
      qa[ks][2] = at[0] ? at[0][ks * 8 + 4 + tq] : 0u;
      qa[ks][3] = at[1] ? at[1][ks * 8 + 4 + tq] : 0u;
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[i][c] = 0.f;
  }
  __device__ __forceinline__ void tile(const DraftBatch& a, const DraftSeq& seq, const DraftItem& it,
                                       const uint8_t* ks_, const uint8_t* vs_, int64_t x0, bool all, float scale_log2) {
    if (row0 >= it.ni * it.nh) return;
    const int lane = threadIdx.x & 31;
    const uint32_t kb_ = smem_u32(ks_), vb_ = smem_u32(vs_);
    float s[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) s[j][c] = 0.f;
    const int krow = ((lane >> 4) << 3) + (lane & 7), kc = (lane >> 3) & 1;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t b[4];
        ldsm4(kb_ + swizzled<D * 2>(j * 16 + krow, 2 * ks + kc), b);
        mma16816(s[2 * j], qa[ks], b[0], b[1]);
        mma16816(s[2 * j + 1], qa[ks], b[2], b[3]);
      }
    uint64_t see[2] = {~0ull, ~0ull};
    if (!all) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = row0 + g + 8 * r;
        see[r] = row < it.ni * it.nh ? draft_sees(a, seq, it.i0 + row / it.nh, x0) : 0;
      }
    }
    uint32_t hi[8][2], lo[8][2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float& x = s[j][2 * r + c];
          x = all || (see[r] >> (j * 8 + 2 * tq + c) & 1) ? x * scale_log2 : -INFINITY;
          mx = fmaxf(mx, x);
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m[r], mx), base = mn == -INFINITY ? 0.f : mn;
      const float corr = ex2_approx(m[r] - base);
      m[r] = mn;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float x[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          x[c] = ex2_approx(s[j][2 * r + c] - base);
          sum += x[c];
        }
        Worker<bf16, D, 8>::split(x[0], x[1], hi[j][r], lo[j][r]);
      }
      l[r] = l[r] * corr + sum;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][2 * r] *= corr;
        o[i][2 * r + 1] *= corr;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t ph[4] = {hi[2 * j][0], hi[2 * j][1], hi[2 * j + 1][0], hi[2 * j + 1][1]};
      const uint32_t pl[4] = {lo[2 * j][0], lo[2 * j][1], lo[2 * j + 1][0], lo[2 * j + 1][1]};
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t b[4];
        ldsm4_t(vb_ + swizzled<D * 2>(j * 16 + (lane & 15), 2 * i + (lane >> 4)), b);
        mma16816(o[2 * i], ph, b[0], b[1]);
        mma16816(o[2 * i + 1], ph, b[2], b[3]);
        mma16816(o[2 * i], pl, b[0], b[1]);
        mma16816(o[2 * i + 1], pl, b[2], b[3]);
      }
    }
  }
  __device__ __forceinline__ void add_bad(const DraftBatch& a, const DraftSeq& seq, const DraftItem& it, int64_t x0,
                                       uint64_t bad, const uint8_t* v, const int64_t* off) {
    for (int r = 0; r < 2; ++r) {
      const int row = row0 + g + 8 * r;
      if (row >= it.ni * it.nh) continue;
      uint64_t todo = bad & draft_sees(a, seq, it.i0 + row / it.nh, x0);
      for (; todo; todo &= todo - 1) {
        const uint32_t* vr = reinterpret_cast<const uint32_t*>(v + off[__ffsll(todo) - 1]);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint32_t x = vr[i * 4 + tq];
          o[i][2 * r] += if_bad(bf16lo(x));
          o[i][2 * r + 1] += if_bad(bf16hi(x));
        }
      }
    }
  }
  __device__ __forceinline__ void sum_up() {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
  }
  __device__ __forceinline__ void store(const DraftBatch& a, const DraftSeq& seq, const DraftItem& it, bf16* out,
                                        float* lse) {
    sum_up();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = row0 + g + 8 * r;
      if (row >= it.ni * it.nh) continue;
      const int i = row / it.nh, h = it.kvh * a.G + it.h0 + row % it.nh;
      const int64_t t = (int64_t)seq.first + it.i0 + i;
      const bool any = draft_sees_any(a, seq, it.i0 + i);
      const float inv = any ? 1.f / l[r] : 0.f;
      uint32_t* to = reinterpret_cast<uint32_t*>(out + (t * a.H + h) * D);
#pragma unroll
      for (int c = 0; c < D / 8; ++c)
        to[c * 4 + tq] = any ? pack_bf16x2(o[c][2 * r] * inv, o[c][2 * r + 1] * inv) : 0u;
      if (lse && tq == 0) lse[(int64_t)h * a.T + t] = row_lse(m[r], l[r], any);
    }
  }
  __device__ __forceinline__ void store_part(float* ml, float* po) {
    sum_up();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = row0 + g + 8 * r;
      if (tq == 0) *reinterpret_cast<float2*>(ml + row * 2) = make_float2(m[r], l[r]);
#pragma unroll
      for (int c = 0; c < D / 8; ++c)
        *reinterpret_cast<float2*>(po + row * D + c * 8 + 2 * tq) = make_float2(o[c][2 * r], o[c][2 * r + 1]);
    }
  }
};

// fp32: thread (y, x) of 16 x 16 has rows 4 y to 4 y + 3, of the scores the
// keys x + 16 j, of the outputs the columns kVec x + 16 kVec i.
template <int D>
struct Rows<float, D> {
  static constexpr int kVec = D == 32 ? 2 : 4, kParts = D / (16 * kVec), kStride = 68;
  float m[4], l[4], o[4][D / 16];
  float *qs, *ps;
  int y, x;

  __device__ __forceinline__ explicit Rows(void* scratch) {
    qs = static_cast<float*>(scratch);
    ps = qs + 64 * D;
    y = threadIdx.x >> 4;
    x = threadIdx.x & 15;
  }
  __device__ __forceinline__ void load_q(const float* q, int64_t stride, int64_t token, int head, int ni, int nh) {
    for (int e = threadIdx.x; e < 64 * (D / 4); e += 256) {
      const int row = e / (D / 4), c = e % (D / 4);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < ni * nh)
        v = *reinterpret_cast<const float4*>(q + (token + row / nh) * stride + (int64_t)(head + row % nh) * D + 4 * c);
      *reinterpret_cast<float4*>(qs + row * D + 4 * c) = v;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[r][c] = 0.f;
    }
  }
  __device__ __forceinline__ void tile(const DraftBatch& a, const DraftSeq& seq, const DraftItem& it,
                                       const uint8_t* ks_, const uint8_t* vs_, int64_t x0, bool all, float scale_log2) {
    const int rows = it.ni * it.nh;
    if ((y & ~1) * 4 >= rows) return;                       // the whole warp's rows
    float2 s2[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) s2[r][j] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int c = 0; c < D / 4; ++c) {
      float4 kq[4], qq[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = x + 16 * j;
        kq[j] = *reinterpret_cast<const float4*>(ks_ + swizzled<D * 4>(key, c));
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) qq[r] = *reinterpret_cast<const float4*>(qs + (4 * y + r) * D + 4 * c);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          ffma2(qq[r].x, qq[r].y, kq[j].x, kq[j].y, s2[r][j].x, s2[r][j].y, s2[r][j].x, s2[r][j].y);
          ffma2(qq[r].z, qq[r].w, kq[j].z, kq[j].w, s2[r][j].x, s2[r][j].y, s2[r][j].x, s2[r][j].y);
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 4 * y + r;
      uint64_t see = ~0ull;
      if (!all) see = row < rows ? draft_sees(a, seq, it.i0 + row / it.nh, x0) : 0;
      float s[4], mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[j] = all || (see >> (x + 16 * j) & 1) ? (s2[r][j].x + s2[r][j].y) * scale_log2 : -INFINITY;
        mx = fmaxf(mx, s[j]);
      }
#pragma unroll
      for (int k = 1; k < 16; k <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
      const float mn = fmaxf(m[r], mx), base = mn == -INFINITY ? 0.f : mn;
      const float corr = ex2_approx(m[r] - base);
      m[r] = mn;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[j] = ex2_approx(s[j] - base);
        sum += s[j];
        ps[row * kStride + x + 16 * j] = s[j];
      }
      l[r] = l[r] * corr + sum;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[r][c] *= corr;
    }
    __syncwarp();                                           // a warp reads the rows that it wrote
#pragma unroll 2
    for (int k4 = 0; k4 < 16; ++k4) {
      float4 pr[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) pr[r] = *reinterpret_cast<const float4*>(ps + (4 * y + r) * kStride + 4 * k4);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int key = 4 * k4 + k;
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
          const int col = kVec * x + 16 * kVec * i;
          const float* vp = reinterpret_cast<const float*>(vs_ + swizzled<D * 4>(key, col / 4)) + col % 4;
          float v[kVec];
          if constexpr (kVec == 4) {
            const float4 t = *reinterpret_cast<const float4*>(vp);
            v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
          } else {
            const float2 t = *reinterpret_cast<const float2*>(vp);
            v[0] = t.x, v[1] = t.y;
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float pk = k == 0 ? pr[r].x : k == 1 ? pr[r].y : k == 2 ? pr[r].z : pr[r].w;
#pragma unroll
            for (int c = 0; c < kVec; c += 2)
              ffma2(pk, pk, v[c], v[c + 1], o[r][kVec * i + c], o[r][kVec * i + c + 1], o[r][kVec * i + c],
                    o[r][kVec * i + c + 1]);
          }
        }
      }
    }
  }
  __device__ __forceinline__ void add_bad(const DraftBatch& a, const DraftSeq& seq, const DraftItem& it, int64_t x0,
                                       uint64_t bad, const uint8_t* v, const int64_t* off) {
    for (int r = 0; r < 4; ++r) {
      const int row = 4 * y + r;
      if (row >= it.ni * it.nh) continue;
      uint64_t todo = bad & draft_sees(a, seq, it.i0 + row / it.nh, x0);
      for (; todo; todo &= todo - 1) {
        const float* vr = reinterpret_cast<const float*>(v + off[__ffsll(todo) - 1]);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) o[r][c] += if_bad(vr[kVec * x + 16 * kVec * (c / kVec) + c % kVec]);
      }
    }
  }
  __device__ __forceinline__ void sum_up() {
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int k = 1; k < 16; k <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], k);
  }
  __device__ __forceinline__ void put(float* row, int r, float f) const {
#pragma unroll
    for (int c = 0; c < D / 16; ++c) row[kVec * x + 16 * kVec * (c / kVec) + c % kVec] = o[r][c] * f;
  }
  __device__ __forceinline__ void store(const DraftBatch& a, const DraftSeq& seq, const DraftItem& it, float* out,
                                        float* lse) {
    sum_up();
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 4 * y + r;
      if (row >= it.ni * it.nh) continue;
      const int i = row / it.nh, h = it.kvh * a.G + it.h0 + row % it.nh;
      const int64_t t = (int64_t)seq.first + it.i0 + i;
      const bool any = draft_sees_any(a, seq, it.i0 + i);
      if (!any)
#pragma unroll
        for (int c = 0; c < D / 16; ++c) o[r][c] = 0.f;
      put(out + (t * a.H + h) * D, r, any ? 1.f / l[r] : 0.f);
      if (lse && x == 0) lse[(int64_t)h * a.T + t] = row_lse(m[r], l[r], any);
    }
  }
  __device__ __forceinline__ void store_part(float* ml, float* po) {
    sum_up();
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 4 * y + r;
      if (x == 0) *reinterpret_cast<float2*>(ml + row * 2) = make_float2(m[r], l[r]);
      put(po + row * D, r, 1.f);
    }
  }
};

}  // namespace draft
}  // namespace nt
