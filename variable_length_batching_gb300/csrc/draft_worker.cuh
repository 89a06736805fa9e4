// What the threads of the kernels for drafted tokens do with keys and rows:
// scores, a running softmax, outputs.  Rows: 64 keys and up to 64 rows to a CTA
// (the general kernel).  Slice: 16 keys and 16 rows to a warp.
#pragma once

#include "draft_plan.cuh"
#include "paged_worker.cuh"

namespace nt {
namespace draft {

using namespace paged;

// 16 bytes, or zeros (nothing is read) where `there` is false.
__device__ __forceinline__ void cp_async16(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait0() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait1() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

// Place of 16-byte chunk c of row r: rows lie 16 bytes further apart than they
// are long, so that eight rows' equal chunks lie in different banks.
template <uint32_t kRow>
__device__ __forceinline__ uint32_t padded(int r, int c) {
  return (uint32_t)r * (kRow + 16) + (c << 4);
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
template <typename T>
__device__ __forceinline__ bool has_bad(const uint4& v) {
  if (sizeof(T) == 4) {
    const uint32_t m = 0x7fffffffu;
    return max(max(v.x & m, v.y & m), max(v.z & m, v.w & m)) >= 0x7f800000u;
  }
  bool any = false;
  for (uint32_t w : {v.x, v.y, v.z, v.w}) any |= (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
  return any;
}
__device__ __forceinline__ float if_bad(float v) { return fabsf(v) <= 3.402823466e38f ? 0.f : v; }

// The value of a row that sees no key is 0, its log-sum-exp -infinity.
__device__ __forceinline__ float row_lse(float m, float l, bool any) {
  return any ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// kGroups groups of threads have the same 64 / kGroups rows and as many of the tile's keys each.
template <typename T, int D, int kGroups = 1>
struct Rows;

// bf16: warp w has rows 16 w to 16 w + 15; a lane two of them, g and g + 8.
template <int D>
struct Rows<bf16, D, 1> {
  uint32_t qa[D / 16][4];
  float m[2], l[2], o[D / 8][4];
  int g, tq, row0;

  __device__ __forceinline__ explicit Rows(void*) {
    const int lane = threadIdx.x & 31;
    g = lane >> 2;
    tq = lane & 3;
    row0 = (threadIdx.x >> 5) * 16;
  }
  __device__ __forceinline__ void merge(float*) {}
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
        ldsm4(kb_ + padded<D * 2>(j * 16 + krow, 2 * ks + kc), b);
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
        ldsm4_t(vb_ + padded<D * 2>(j * 16 + (lane & 15), 2 * i + (lane >> 4)), b);
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

// fp32 on the tensor cores: a value is the sum of two tf32 (11 bits each), and
// a product the sum of three, upper by upper and upper by lower both ways.  Of
// the two factors the one with fewer uses, q or p, is rounded to its upper part, so
// that its lower part has either sign and what is left out, lower by lower, is
// 2^-21 at most and 0 on average; k and v are cut.  A matrix instruction cuts
// its sums to fp32 as well, a step each, so only 16 columns or one tile's keys are
// summed in it, the lower products apart, and fp32 adds do the rest.
struct Tf32 {
  uint32_t hi, lo;
};
__device__ __forceinline__ Tf32 tf32_cut(float x) {
  Tf32 t;
  t.hi = __float_as_uint(x) & 0xffffe000u;
  t.lo = __float_as_uint(x - __uint_as_float(t.hi)) + 0x1000u;
  return t;
}
__device__ __forceinline__ Tf32 tf32_round(float x) {      // |x| below 2^127
  Tf32 t;
  t.hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  t.lo = __float_as_uint(x - __uint_as_float(t.hi)) + 0x1000u;
  return t;
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// fp32: warp w has rows 16 (w % kRowGroups) to + 15 and the tile's keys of its
// group; a lane two of the rows, g and g + 8, of the scores the keys 8 n + 2 tq
// and + 1, of the outputs those columns.
template <int D, int kGroups>
struct Rows<float, D, kGroups> {
  static constexpr int kM = 64 / kGroups, kRowGroups = kM / 16, kKeyGroups = 8 / kRowGroups, kN = 64 / kKeyGroups / 8;
  float m[2], l[2], o[D / 8][4];
  float4 *qh, *ql;                 // upper and lower parts of the queries, as the instruction takes them
  int g, tq, lane, row0, group, key0;

  __device__ __forceinline__ explicit Rows(void* scratch) {
    lane = threadIdx.x & 31;
    g = lane >> 2;
    tq = lane & 3;
    const int warp = threadIdx.x >> 5;
    row0 = warp % kRowGroups * 16;
    group = warp / kRowGroups;
    key0 = group * 8 * kN;
    qh = static_cast<float4*>(scratch);
    ql = qh + kM * D / 4;
  }
  __device__ __forceinline__ void load_q(const float* q, int64_t stride, int64_t token, int head, int ni, int nh) {
    constexpr int kAll = kM * D / 4, kTurns = (kAll + 255) / 256, kAtOnce = kTurns < 4 ? kTurns : 4;
    for (int e0 = threadIdx.x; e0 < kAll; e0 += 256 * kAtOnce) {
      float v[kAtOnce][4];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int at = (e0 >> 5) + 8 * k, ks = at % (D / 8);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = at / (D / 8) * 16 + g + 8 * r;
          const bool there = row < ni * nh;
          const float* from = q + (token + row / nh) * stride + (int64_t)(head + row % nh) * D + 8 * ks + tq;
          v[k][r] = there ? from[0] : 0.f;
          v[k][2 + r] = there ? from[4] : 0.f;
        }
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        float hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = v[k][i];
          const Tf32 t = fabsf(x) < 1.7014118e38f ? tf32_round(x) : tf32_cut(x);
          hi[i] = __uint_as_float(t.hi);
          lo[i] = __uint_as_float(t.lo);
          if (!(fabsf(x) <= 3.402823466e38f)) hi[i] = x, lo[i] = 0.f;
        }
        const int e = e0 + 256 * k;
        if (kAll % 256 == 0 || e < kAll) {
          qh[e] = make_float4(hi[0], hi[1], hi[2], hi[3]);
          ql[e] = make_float4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) m[r] = -INFINITY, l[r] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 8; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[c][i] = 0.f;
  }
  // A score by plain multiply-adds, where that of the parts is not finite: the parts of an infinite key make NaN of it,
  // and a NaN whose payload is all in the bits that the upper part has lost is an infinity there.
  static __device__ __noinline__ float score(const float* q_hi, const float* q_lo, const uint8_t* ks_, int row,
                                             int key) {
    float s = 0.f;
    for (int c = 0; c < D; ++c) {
      const int e = ((c / 8) * 32 + (row & 7) * 4 + (c & 3)) * 4 + (row >> 3) + (c & 4) / 2;
      s = fmaf(q_hi[e] + q_lo[e], *reinterpret_cast<const float*>(ks_ + padded<D * 4>(key, c / 4) + (c & 3) * 4), s);
    }
    return s;
  }
  __device__ __forceinline__ void tile(const DraftBatch& a, const DraftSeq& seq, const DraftItem& it,
                                       const uint8_t* ks_, const uint8_t* vs_, int64_t x0, bool all, float scale_log2) {
    const int rows = it.ni * it.nh;
    if (row0 >= rows) return;                               // the whole warp's rows
    uint64_t see[2];                                        // read while the scores are computed
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = row0 + g + 8 * r;
      see[r] = all ? ~0ull : row < rows ? draft_sees(a, seq, it.i0 + row / it.nh, x0) >> key0 : 0;
    }
    float s[kN][4], sl[kN][4];
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[n][i] = sl[n][i] = 0.f;
    const float4 *qhi = qh + row0 * D / 4 + lane, *qlo = ql + row0 * D / 4 + lane;
#pragma unroll 2
    for (int k2 = 0; k2 < D / 16; ++k2) {
      uint32_t ah[2][4], al[2][4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float4 h = qhi[(2 * k2 + k) * 32], w = qlo[(2 * k2 + k) * 32];
        ah[k][0] = __float_as_uint(h.x), ah[k][1] = __float_as_uint(h.y), ah[k][2] = __float_as_uint(h.z),
        ah[k][3] = __float_as_uint(h.w);
        al[k][0] = __float_as_uint(w.x), al[k][1] = __float_as_uint(w.y), al[k][2] = __float_as_uint(w.z),
        al[k][3] = __float_as_uint(w.w);
      }
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        uint32_t kr[4];
        ldsm4(smem_u32(ks_ + padded<D * 4>(key0 + 8 * n + (lane & 7), 4 * k2 + (lane >> 3))), kr);
        Tf32 b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = tf32_cut(__uint_as_float(kr[i]));
        float t[4] = {};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          mma_tf32(sl[n], al[k], b[2 * k].hi, b[2 * k + 1].hi);
          mma_tf32(sl[n], ah[k], b[2 * k].lo, b[2 * k + 1].lo);
          mma_tf32(t, ah[k], b[2 * k].hi, b[2 * k + 1].hi);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[n][i] += t[i];
      }
    }
    bool odd = false;
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[n][i] += sl[n][i];
        odd |= !(fabsf(s[n][i]) <= 3.402823466e38f) && (see[i >> 1] >> (8 * n + 2 * tq + (i & 1)) & 1);
      }
    if (odd) {
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!(fabsf(s[n][i]) <= 3.402823466e38f))
            s[n][i] = score(reinterpret_cast<const float*>(qh + row0 * D / 4),
                            reinterpret_cast<const float*>(ql + row0 * D / 4), ks_, g + 8 * (i >> 1),
                            key0 + 8 * n + 2 * tq + (i & 1));
    }
    float corr[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float mx = -INFINITY;
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float& x = s[n][2 * r + j];
          x = all || (see[r] >> (8 * n + 2 * tq + j) & 1) ? x * scale_log2 : -INFINITY;
          mx = fmaxf(mx, x);
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m[r], mx), base = mn == -INFINITY ? 0.f : mn;
      corr[r] = ex2_approx(m[r] - base);
      m[r] = mn;
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          s[n][2 * r + j] = ex2_approx(s[n][2 * r + j] - base);
          sum += s[n][2 * r + j];
        }
      l[r] = l[r] * corr[r] + sum;
    }
    uint32_t ph[kN][4], pl[kN][4];           // the keys' order in the instruction: 2 tq as column tq, 2 tq + 1 as tq + 4
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Tf32 t = tf32_round(s[n][i]);
        const int at = (i & 1) * 2 + (i >> 1);
        ph[n][at] = t.hi;
        pl[n][at] = t.lo;
      }
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
      float t[4] = {}, tl[4] = {};
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        const int key = key0 + 8 * n + 2 * tq, chunk = 2 * c + (g >> 2), at = (g & 3) * 4;
        const Tf32 b0 = tf32_cut(*reinterpret_cast<const float*>(vs_ + padded<D * 4>(key, chunk) + at));
        const Tf32 b1 = tf32_cut(*reinterpret_cast<const float*>(vs_ + padded<D * 4>(key + 1, chunk) + at));
        mma_tf32(tl, pl[n], b0.hi, b1.hi);
        mma_tf32(tl, ph[n], b0.lo, b1.lo);
        mma_tf32(t, ph[n], b0.hi, b1.hi);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) o[c][i] = o[c][i] * corr[i >> 1] + (t[i] + tl[i]);
    }
  }
  __device__ __forceinline__ void add_bad(const DraftBatch& a, const DraftSeq& seq, const DraftItem& it, int64_t x0,
                                       uint64_t bad, const uint8_t* v, const int64_t* off) {
    bad &= (kN == 8 ? ~0ull : (1ull << 8 * kN) - 1) << key0;
    for (int r = 0; r < 2; ++r) {
      const int row = row0 + g + 8 * r;
      if (row >= it.ni * it.nh) continue;
      uint64_t todo = bad & draft_sees(a, seq, it.i0 + row / it.nh, x0);
      for (; todo; todo &= todo - 1) {
        const float* vr = reinterpret_cast<const float*>(v + off[__ffsll(todo) - 1]);
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const float2 x = *reinterpret_cast<const float2*>(vr + 8 * c + 2 * tq);
          const float y0 = if_bad(x.x), y1 = if_bad(x.y);
          if (r == 0) o[c][0] += y0, o[c][1] += y1;
          else o[c][2] += y0, o[c][3] += y1;
        }
      }
    }
  }
  // The groups' results into the first one's; `red` has room for 128 rows of D and two.
  __device__ __forceinline__ void merge(float* red) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
    float2* ml = reinterpret_cast<float2*>(red + 128 * D);
    if (group > 0) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int at = group * kM + row0 + g + 8 * r;
        put(red + at * D, r, 1.f);
        if (tq == 0) ml[at] = make_float2(m[r], l[r]);
      }
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int r = 0; r < 2; ++r)
      for (int k = 1; k < kKeyGroups; ++k) {
        const int at = k * kM + row0 + g + 8 * r;
        const float2 other = ml[at];
        const float mn = fmaxf(m[r], other.x), base = mn == -INFINITY ? 0.f : mn;
        const float f = ex2_approx(m[r] - base), fo = ex2_approx(other.x - base);
        m[r] = mn;
        l[r] = l[r] * f + other.y * fo;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const float2 x = *reinterpret_cast<const float2*>(red + at * D + 8 * c + 2 * tq);
          o[c][2 * r] = o[c][2 * r] * f + x.x * fo;
          o[c][2 * r + 1] = o[c][2 * r + 1] * f + x.y * fo;
        }
      }
  }
  __device__ __forceinline__ void put(float* row, int r, float f) const {
#pragma unroll
    for (int c = 0; c < D / 8; ++c)
      *reinterpret_cast<float2*>(row + 8 * c + 2 * tq) = make_float2(o[c][2 * r] * f, o[c][2 * r + 1] * f);
  }
  __device__ __forceinline__ void store(const DraftBatch& a, const DraftSeq& seq, const DraftItem& it, float* out,
                                        float* lse) {
    if (group > 0) return;
    bool sees_any[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = row0 + g + 8 * r;
      sees_any[r] = row < it.ni * it.nh && draft_sees_any(a, seq, it.i0 + row / it.nh);
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = row0 + g + 8 * r;
      if (row >= it.ni * it.nh) continue;
      const int i = row / it.nh, h = it.kvh * a.G + it.h0 + row % it.nh;
      const int64_t t = (int64_t)seq.first + it.i0 + i;
      if (!sees_any[r])
#pragma unroll
        for (int c = 0; c < D / 8; ++c) o[c][2 * r] = o[c][2 * r + 1] = 0.f;
      put(out + (t * a.H + h) * D, r, sees_any[r] ? 1.f / l[r] : 0.f);
      if (lse && tq == 0) lse[(int64_t)h * a.T + t] = row_lse(m[r], l[r], sees_any[r]);
    }
  }
  __device__ __forceinline__ void store_part(float* ml, float* po) {
    if (group > 0) return;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = row0 + g + 8 * r;
      if (tq == 0) *reinterpret_cast<float2*>(ml + row * 2) = make_float2(m[r], l[r]);
      put(po + row * D, r, 1.f);
    }
  }
};

// ---- slices of 16 keys -------------------------------------------------------------

constexpr int kWords = kDraftMaxNew / 64;
constexpr int kBadWords = 10;               // new tokens, from the 16 keys that the first of them is in

// Keys [x, x + 16) that a row sees, from its mask words in shared memory.
__device__ __forceinline__ uint32_t sees16(const DraftBatch& a, const DraftSeq& s, int i, const unsigned long long* words,
                                           int x) {
  const int left = s.len - x, j = x - (s.len - s.n);
  const uint32_t there = left >= 16 ? 0xffffu : (1u << max(left, 0)) - 1;
  if (j <= -16) return there;
  if (!a.bits) {
    const int upto = i - j;                         // the last one seen, from x
    return upto < 0 ? 0 : upto >= 15 ? there : there & ((2u << upto) - 1);
  }
  if (j < 0) return there & ((1u << -j) - 1 | (uint32_t)(words[0] << -j));
  const int k = j >> 6, sh = j & 63;
  uint64_t m = k < a.words ? words[k] >> sh : 0;
  if (sh && k + 1 < a.words) m |= words[k + 1] << (64 - sh);
  return there & (uint32_t)m;
}

// A warp's 16 rows and their running statistics; a lane has two, g and g + 8.
// The warp's keys lie in a stage as those of paged_worker.cuh, the values kSide bytes behind them.
template <int D, uint32_t kSide>
struct Slice {
  static constexpr uint32_t kRow = D * 2;
  static constexpr int kRedStride = D + 4;      // floats: keeps the results' writes conflict-free
  static constexpr uint32_t kBoxRow = D < 64 ? D * 2 : 128;   // bytes of a key in a box's columns
  uint32_t qa[D / 16][4];
  float m[2], l[2], o[D / 8][4];
  int g, tq;
  uint32_t hs;                     // to a box's next 64 columns
  int box;                         // a power of two

  __device__ __forceinline__ explicit Slice(int box_) : box(box_) {
    const int lane = threadIdx.x & 31;
    g = lane >> 2;
    tq = lane & 3;
    hs = box * 128;
  }
  __device__ __forceinline__ uint32_t row_at(int r) const {
    return (uint32_t)(r & -box) * kRow + (r & (box - 1)) * kBoxRow;
  }
  __device__ __forceinline__ static int swizzle(int r) { return D < 64 ? (r >> 1) & 3 : r & 7; }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[i][c] = 0.f;
  }
  // rows `first` to first + 15 of the item's, as TMA laid them down, 64 columns `part` bytes behind the 64 before (rows
  // behind the item's last hold anything)
  __device__ __forceinline__ void load_q(uint32_t rows, int first, int part) {
    const int lane = threadIdx.x & 31, row = first + (lane & 15);
    const uint32_t at = rows + row * kBoxRow, x = ((lane >> 4) ^ swizzle(row)) << 4;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
      ldsm4(at + (ks >> 2) * part + ((((uint32_t)ks & 3) << 5) ^ x), qa[ks]);
    clear();
  }
  // the same from two rows in memory, NULL for none
  __device__ __forceinline__ void load_q(const bf16* row0, const bf16* row1) {
    const uint32_t *q0 = reinterpret_cast<const uint32_t*>(row0), *q1 = reinterpret_cast<const uint32_t*>(row1);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      qa[ks][0] = q0 ? q0[ks * 8 + tq] : 0u;
      qa[ks][1] = q1 ? q1[ks * 8 + tq] : 0u;
      qa[ks][2] = q0 ? q0[ks * 8 + 4 + tq] : 0u;
      qa[ks][3] = q1 ? q1[ks * 8 + 4 + tq] : 0u;
    }
    clear();
  }
  // Slice `slice` of the stage; `all`: every row sees every key, else the rows' masks in `see`.
  __device__ __forceinline__ void tile(uint32_t kbase, int slice, bool all, const uint32_t (&see)[2], float scale_log2) {
    const int lane = threadIdx.x & 31;
    const uint32_t vbase = kbase + kSide;
    const int krow = slice * 16 + ((lane >> 4) << 3) + (lane & 7), vrow = slice * 16 + (lane & 15);
    const uint32_t k_at = kbase + row_at(krow), v_at = vbase + row_at(vrow);
    const uint32_t kx = (((lane >> 3) & 1) ^ swizzle(krow)) << 4, vx = ((lane >> 4) ^ swizzle(vrow)) << 4;
    // two chains for each eight keys
    float s[2][4] = {}, s2[2][4] = {};
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t b[4];
      ldsm4(k_at + (ks >> 2) * hs + ((((uint32_t)ks & 3) << 5) ^ kx), b);
      mma16816(ks & 1 ? s2[0] : s[0], qa[ks], b[0], b[1]);
      mma16816(ks & 1 ? s2[1] : s[1], qa[ks], b[2], b[3]);
    }
    uint32_t ph[4], pl[4];
    float corr[2];
    bool moved = false;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        v[c] = (s[c >> 1][2 * r + (c & 1)] + s2[c >> 1][2 * r + (c & 1)]) * scale_log2;
        if (!all && !(see[r] >> ((c >> 1) * 8 + 2 * tq + (c & 1)) & 1)) v[c] = -INFINITY;
      }
      float mx = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m[r], mx), base = mn == -INFINITY ? 0.f : mn;
      moved |= mn > m[r];
      corr[r] = ex2_approx(m[r] - base);
      m[r] = mn;
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = ex2_approx(v[c] - base);
      l[r] = l[r] * corr[r] + (v[0] + v[1]) + (v[2] + v[3]);
      Worker<bf16, D, 8>::split(v[0], v[1], ph[r], pl[r]);
      Worker<bf16, D, 8>::split(v[2], v[3], ph[2 + r], pl[2 + r]);
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][0] *= corr[0];
        o[i][1] *= corr[0];
        o[i][2] *= corr[1];
        o[i][3] *= corr[1];
      }
    }
    // two column blocks at a time: a product does not wait for the one before it
#pragma unroll
    for (int i = 0; i < D / 16; i += 2) {
      uint32_t b[2][4];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        ldsm4_t(v_at + ((i + k) >> 2) * hs + ((((uint32_t)(i + k) & 3) << 5) ^ vx), b[k]);
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          mma16816(o[2 * (i + k)], part ? pl : ph, b[k][0], b[k][1]);
          mma16816(o[2 * (i + k) + 1], part ? pl : ph, b[k][2], b[k][3]);
        }
    }
  }
  // V of a slice as the products may read it: rows behind the last key become zeros, values that are not finite are
  // taken out (their keys in `found`).
  __device__ __forceinline__ uint32_t clean(uint8_t* stage, int slice, int left) const {
    const int lane = threadIdx.x & 31;
    uint32_t found = 0;
    for (int e = lane; e < 16 * (D / 8); e += 32) {
      const int key = e / (D / 8), ch = e % (D / 8);
      uint8_t* at = stage + kSide + row_at(slice * 16 + key) + (ch >> 3) * hs + (ch & 7) * 16;
      if (key >= left) *reinterpret_cast<uint4*>(at) = make_uint4(0, 0, 0, 0);
      else if (clear_bad<bf16>(at)) found |= 1u << key;
    }
    __syncwarp();
    return __reduce_or_sync(0xffffffffu, found);
  }
  // the warp's results: maxima and sums (-1: no keys, nothing to add), outputs [16][kRedStride]
  __device__ __forceinline__ void result(float* rm, float* rl, float* ro, bool active) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (tq == 0) {
        rm[g + 8 * r] = m[r];
        rl[g + 8 * r] = active ? l[r] : -1.f;
      }
      if (!active) continue;
      float* to = ro + (g + 8 * r) * kRedStride + 2 * tq;
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<float2*>(to + i * 8) = make_float2(o[i][2 * r], o[i][2 * r + 1]);
    }
  }
};

}  // namespace draft
}  // namespace nt
