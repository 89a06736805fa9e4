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
// Both directions are bound by HBM (65,536 tokens of 12 + 12 heads of 64 in
// bf16: forward 66 to 69 us, 86 to 90% of the measured copy rate, backward 96,
// 93%; 16,384 of 32 + 8 of 128: 53.3 and 78.9, 93% and 94%; in fp32 forward 110,
// 90%, and 30,000 of 12 + 12 of 64 67.8, 80%), and at about ten
// operations an element not by much, so the layout keeps loads in flight
// without holding registers or waiting at barriers.  A row (one head of one
// token) is a group of LP lanes, 16 elements to a lane in 16-byte words spread
// over the row so that the words of neighbouring lanes are neighbours, and so
// that a lane holds both columns of its eight pairs in either layout.  A warp
// takes units of some tokens and consecutive heads of q or of k, one row per
// group and step.  Units are dealt out in order, a round at a time:
// all warps work in one region of memory (giving each warp a range of its own
// costs a tenth of the bandwidth), and the unit's heads are chosen so that
// the rounds come out even.  Each thread copies its own words of the rows
// kSlots steps ahead into its own words of shared memory (cp.async), so
// nothing but its own copies is ever waited for.  A warp forms its tokens'
// cosines and sines itself and keeps them, in the forward multiplied by
// gamma, in registers.  Everything between the load and the one rounding of
// the store is fp32, in packed pairs.
#include "tc_ptx.cuh"

namespace nt {
namespace {

using tc::ffma2;
using tc::fmul2;

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
  uint32_t units[2];         // of each side: token groups x parts of its heads
  int parts[2], unit_heads;  // parts of a side's heads, heads of a part
  int d, rot, B;
  float inv_d, eps, scale;
  const int32_t* cu;
  const int32_t* pos0;
  const int32_t* positions;
  const uint64_t* turns;
  float* partial;            // backward: [CTAs][2][d] sums for dgamma
  unsigned int* status;
};

// Position of this lane's token t; the warp's tokens are t_first, ...,
// t_last (consecutive, clipped to T).  False (flagged) if the offsets place
// it in no segment.  The warp searches its first token's segment together, 32
// probes a step (two dependent loads for up to 1,024 segments), and finds the
// others among the 32 boundaries that follow; a token behind those (tokens
// separated by many empty segments) is searched by itself.
__device__ __forceinline__ bool lane_position(const Args& a, int64_t t, int64_t t_first, int n_tok, int64_t& pos) {
  const int lane = threadIdx.x & 31;
  pos = 0;
  if (a.rot == 0) return true;
  if (a.positions) {
    pos = a.positions[t];
    return true;
  }
  const int b0 = segment_of_warp(a.cu, a.B, t_first);
  const int first_start = a.cu[b0];
  const int bound = a.cu[min((int64_t)b0 + 1 + lane, (int64_t)a.B)];     // repeats cu[B] past the end
  int mine = 0;
  for (int k = 0; k < n_tok; ++k) {
    const int c = __popc(__ballot_sync(0xffffffffu, bound <= t_first + k));
    if (t_first + k == t) mine = c;
  }
  int start = __shfl_sync(0xffffffffu, bound, max(mine - 1, 0)), end = __shfl_sync(0xffffffffu, bound, min(mine, 31));
  int seg = b0 + mine;
  if (mine == 0) start = first_start;
  if (mine == 32) {
    seg = segment_of_thread(a.cu, a.B, t);
    start = a.cu[seg];
    end = a.cu[seg + 1];
  }
  if (seg >= a.B || start > t || end <= t || start < 0) {
    flag_device(a.status, kDevCheck);
    return false;
  }
  pos = t - start + (a.pos0 ? a.pos0[seg] : 0);
  return true;
}

// A lane's columns: element e of 16 is column col(e / V) + e % V, V the
// elements of a 16-byte word.  The lanes of the rotated part come first.
template <typename T, int LP, bool kInter>
struct Lane {
  static constexpr int V = 16 / sizeof(T), W = 16 / V;
  static constexpr int kGroups = 32 / LP;                         // a warp's (lanes behind the last one idle)
  static constexpr int kRow = LP * 16 * sizeof(T);                // bytes of a row, at most
  static constexpr int kSide = kRow >= 128 ? 1 : 128 / kRow;      // rows of one token in a step, side by side
  static constexpr int kTok = kGroups / kSide;                    // tokens of a step
  int i, tok, h_off, col0, step;
  bool on, rotated;
  __device__ __forceinline__ Lane(const Args& a) {
    const int lane = threadIdx.x & 31;
    const bool idle = lane >= kGroups * LP;
    const int g = idle ? 0 : lane / LP;
    i = lane % LP;
    tok = g / kSide;
    h_off = g % kSide;
    on = !idle && 16 * i < a.d;
    rotated = !idle && 16 * i < a.rot;
    const int first = rotated ? 0 : a.rot, width = rotated ? a.rot : a.d - a.rot;
    col0 = first + V * (i - first / 16);
    step = width / W;
  }
  __device__ __forceinline__ int col(int w) const { return col0 + w * step; }
  // cosines and sines of the lane's eight pairs at pos (1 and 0 where nothing turns)
  __device__ __forceinline__ void angles(const Args& a, int64_t pos, float (&c)[8], float (&s)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      c[e] = 1.f;
      s[e] = 0.f;
    }
    if (!rotated) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // the pair's first column: element e (half), element 2 e (interleaved)
      const int j = kInter ? (col(2 * e / V) + 2 * e % V) / 2 : col(e / V) + e % V;
      const float frac = (float)(int32_t)(((uint64_t)pos * a.turns[j]) >> 32);     // in 2^-32 turns, [-1/2, 1/2)
      // For bf16 the hardware's sine and cosine do: within [-pi, pi] they are
      // off by 2^-21, with the angle's rounding by 2^-20 at most, a 4,096th of
      // the half step (2^-8) that an output as large as its pair is rounded by,
      // and cost an eighth of the exact ones, which fp32 takes.
      if constexpr (sizeof(T) == 2) __sincosf(frac * 1.4629180792671596e-9f, &s[e], &c[e]);    // 2 pi 2^-32
      else sincospif(frac * 4.656612873077393e-10f, &s[e], &c[e]);                            // 2^-31: half turns
      c[e] *= a.scale;
      s[e] *= a.scale;
    }
  }
  __device__ __forceinline__ void gamma(const float* p, float (&v)[16]) const {
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = 1.f;
    if (!p || !on) return;
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
      const float4 x = *reinterpret_cast<const float4*>(p + col(e / V) + e % V);
      v[e] = x.x;
      v[e + 1] = x.y;
      v[e + 2] = x.z;
      v[e + 3] = x.w;
    }
  }
  // copy the lane's words of a row into its ring words, 16 bytes each; x and
  // y point at its first column
  __device__ __forceinline__ void copy(uint32_t dst, const T* x) const {
#pragma unroll
    for (int w = 0; w < W; ++w)
      asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;"
                   ::"r"(dst + w * kThreads * 16), "l"(x + w * step) : "memory");
  }
  __device__ __forceinline__ void store(T* y, const float (&v)[16]) const {
#pragma unroll
    for (int w = 0; w < W; ++w) {
      uint4 x;
      if constexpr (sizeof(T) == 2) {
        x = make_uint4(tc::pack_bf16x2(v[8 * w], v[8 * w + 1]), tc::pack_bf16x2(v[8 * w + 2], v[8 * w + 3]),
                       tc::pack_bf16x2(v[8 * w + 4], v[8 * w + 5]), tc::pack_bf16x2(v[8 * w + 6], v[8 * w + 7]));
      } else {
        x = make_uint4(__float_as_uint(v[4 * w]), __float_as_uint(v[4 * w + 1]), __float_as_uint(v[4 * w + 2]),
                       __float_as_uint(v[4 * w + 3]));
      }
      *reinterpret_cast<uint4*>(y + w * step) = x;
    }
  }
};

// v summed over a row's lanes, in one order for all of them.
template <int LP>
__device__ __forceinline__ float group_sum(float v) {
  if constexpr ((LP & (LP - 1)) == 0) {
#pragma unroll
    for (int m = LP / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
  } else {
    const int first = (threadIdx.x & 31) / LP * LP;
    float s = 0.f;
#pragma unroll
    for (int m = 0; m < LP; ++m) s += __shfl_sync(0xffffffffu, v, min(first + m, 31));
    return s;
  }
}
// v summed over a warp's rows, for lanes below LP.
template <int LP>
__device__ __forceinline__ float rows_sum(float v) {
  if constexpr ((LP & (LP - 1)) == 0) {
#pragma unroll
    for (int m = 16; m >= LP; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
  } else {
    float s = v;
#pragma unroll
    for (int g = 1; g < 32 / LP; ++g) s += __shfl_sync(0xffffffffu, v, ((threadIdx.x & 31) + g * LP) & 31);
    return s;
  }
}

// The thread's own words of the ring: 16-byte word w of slot s at
// (s * words + w) * kThreads + thread, so that a warp's accesses are
// consecutive.
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <typename T>
__device__ __forceinline__ void read_row(const uint4* src, float (&v)[16]) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint4 x = src[w * kThreads];
      const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[8 * w + 2 * e] = tc::bf16lo(u[e]);
        v[8 * w + 2 * e + 1] = tc::bf16hi(u[e]);
      }
    }
  } else {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint4 x = src[w * kThreads];
      v[4 * w] = __uint_as_float(x.x);
      v[4 * w + 1] = __uint_as_float(x.y);
      v[4 * w + 2] = __uint_as_float(x.z);
      v[4 * w + 3] = __uint_as_float(x.w);
    }
  }
}

// sum of v[e]^2, or of u[e] v[e]
__device__ __forceinline__ float dot16(const float (&u)[16], const float (&v)[16]) {
  float s0 = 0.f, s1 = 0.f;
#pragma unroll
  for (int e = 0; e < 16; e += 2) ffma2(u[e], u[e + 1], v[e], v[e + 1], s0, s1, s0, s1);
  return s0 + s1;
}

// out = the rotation of v by per-pair factors: for pair (a, b) of eight,
// out_a = v_a f[.] + v_b f[.], in packed pairs.  m holds, for the half layout
// and the two pairs e, e + 1 at a time: {aa, aa'}, {ab, ab'}, {ba, ba'},
// {bb, bb'}; for the interleaved one and pair e: {aa, bb}, {ab, ba}.
template <bool kInter>
__device__ __forceinline__ void turn(const float (&v)[16], const float (&m)[32], float (&w)[16]) {
  if constexpr (kInter) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float x, y;
      fmul2(v[2 * e + 1], v[2 * e], m[4 * e + 2], m[4 * e + 3], x, y);
      ffma2(v[2 * e], v[2 * e + 1], m[4 * e], m[4 * e + 1], x, y, w[2 * e], w[2 * e + 1]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      float x, y;
      fmul2(v[8 + e], v[9 + e], m[4 * e + 2], m[4 * e + 3], x, y);
      ffma2(v[e], v[e + 1], m[4 * e], m[4 * e + 1], x, y, w[e], w[e + 1]);
      fmul2(v[e], v[e + 1], m[4 * e + 4], m[4 * e + 5], x, y);
      ffma2(v[8 + e], v[9 + e], m[4 * e + 6], m[4 * e + 7], x, y, w[8 + e], w[9 + e]);
    }
  }
}

// The same for a lane behind the rotated columns: each value by its own
// factor, so that an infinity stays in its column.
template <bool kInter>
__device__ __forceinline__ void pass(const float (&v)[16], const float (&m)[32], float (&w)[16]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (kInter) {
      w[2 * e] = v[2 * e] * m[4 * e];
      w[2 * e + 1] = v[2 * e + 1] * m[4 * e + 1];
    } else {
      const int b = 4 * (e & ~1) + (e & 1);
      w[e] = v[e] * m[b];
      w[8 + e] = v[8 + e] * m[b + 6];
    }
  }
}

// The warp's place among its units: warp w of n takes units w, w + n, ... of
// the line (q's units, then k's).
struct Place {
  uint32_t u, n;         // unit, warps
  int sd, h, h_end;      // side; head, end of the unit's heads
  uint32_t tg;           // token group
  bool more;
  __device__ __forceinline__ Place(const Args& a) {
    n = gridDim.x * kWarps;
    u = blockIdx.x * kWarps + (threadIdx.x >> 5);
    set(a);
  }
  __device__ __forceinline__ void set(const Args& a) {
    more = u < a.units[0] + a.units[1];
    if (!more) return;
    sd = u >= a.units[0];
    const uint32_t v = u - (sd ? a.units[0] : 0);
    tg = v / (uint32_t)a.parts[sd];
    h = (int)(v - tg * a.parts[sd]) * a.unit_heads;
    h_end = min(h + a.unit_heads, a.side[sd].H);
  }
  __device__ __forceinline__ void next(const Args& a) {
    u += n;
    set(a);
  }
};

// How many steps ahead rows are copied: few.  More than about 48 KB in flight
// on an SM is slower, not faster (the stream's forward with four slots 72 us,
// three 69; its backward with three 101, two 98).
template <typename T> struct Ring {          // forward: one row a step
  static constexpr int kWords = sizeof(T);   // 16-byte words of a row per lane
  static constexpr int kSlots = sizeof(T) == 2 ? 3 : 2;
  static constexpr size_t kBytes = (size_t)kSlots * kWords * 16 * kThreads;
};

// The inner loops hold everything of a unit in registers and step pointers:
// with four warps a scheduler, instructions are the next bound (157 a row and
// lane; 240 with the addresses formed anew each step).
template <typename T, int LP, bool kInter>
__global__ void __launch_bounds__(kThreads, 2) rope_fwd_kernel(const Args a) {
  using R = Ring<T>;
  constexpr uint32_t kSlotWords = R::kWords * kThreads;
  extern __shared__ __align__(16) uint4 ring[];
  using L = Lane<T, LP, kInter>;
  constexpr int kTok = L::kTok;
  const L me(a);
  Place at(a), ahead(a);                     // the unit in hand, and the unit to copy, kSlots rows further
  pdl_wait();
  pdl_trigger();
  const T* px = nullptr;                     // the next row to copy, and how many the unit has left
  int pn = 0;
  bool pon = false;
  auto enter = [&] {
    if (!ahead.more) return;
    const Side& p = a.side[ahead.sd];
    const int64_t t = (int64_t)ahead.tg * kTok + me.tok;
    pon = me.on && t < a.T;
    px = static_cast<const T*>(p.x) + t * p.xs + (int64_t)(ahead.h + me.h_off) * a.d + me.col0;
    pn = ahead.h_end - ahead.h;
  };
  enter();
  uint32_t so = threadIdx.x;                 // this thread's first word of the slot in hand
  auto copy = [&] {
    if (pn > 0) {
      if (pon && me.h_off < pn) me.copy(tc::smem_u32(ring + so), px);
      px += a.d * L::kSide;
      if ((pn -= L::kSide) <= 0) {
        ahead.next(a);
        enter();
      }
    }
    copy_commit();
    so = so + kSlotWords >= R::kSlots * kSlotWords ? threadIdx.x : so + kSlotWords;
  };
#pragma unroll
  for (int s = 0; s < R::kSlots; ++s) {
    // lanes beyond the head's columns copy nothing and add zeros to its sums
    if (!me.on)
#pragma unroll
      for (int w = 0; w < R::kWords; ++w) ring[so + w * kThreads] = make_uint4(0, 0, 0, 0);
    copy();
  }
  while (at.more) {
    const Side& p = a.side[at.sd];
    const int64_t first = (int64_t)at.tg * kTok, t = first + me.tok;
    int64_t pos;
    const bool write = lane_position(a, min64(t, a.T - 1), first, (int)min64(kTok, a.T - first), pos) && me.on &&
                       t < a.T;
    const bool norm = p.gamma != nullptr;
    T* y = static_cast<T*>(p.out) + t * p.os + (int64_t)(at.h + me.h_off) * a.d + me.col0;
    float m[32];
    {
      float c[8], sn[8], gm[16];
      me.angles(a, pos, c, sn);
      me.gamma(p.gamma, gm);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float ga = gm[kInter ? 2 * e : e], gb = gm[kInter ? 2 * e + 1 : 8 + e];
        if constexpr (kInter) {
          m[4 * e] = ga * c[e];
          m[4 * e + 1] = gb * c[e];
          m[4 * e + 2] = -gb * sn[e];
          m[4 * e + 3] = ga * sn[e];
        } else {
          const int b = 4 * (e & ~1) + (e & 1);
          m[b] = ga * c[e];
          m[b + 2] = -gb * sn[e];
          m[b + 4] = ga * sn[e];
          m[b + 6] = gb * c[e];
        }
      }
    }
    for (int n = at.h_end - at.h; n > 0; n -= L::kSide) {
      copy_wait<R::kSlots - 1>();
      float v[16], w[16];
      read_row<T>(ring + so, v);
      if (me.rotated) turn<kInter>(v, m, w);
      else pass<kInter>(v, m, w);
      if (norm) {
        const float r = rsqrtf(fmaf(group_sum<LP>(dot16(v, v)), a.inv_d, a.eps));
#pragma unroll
        for (int e = 0; e < 16; e += 2) fmul2(w[e], w[e + 1], r, r, w[e], w[e + 1]);
      }
      copy();
      if (write && me.h_off < n) me.store(y, w);
      y += a.d * L::kSide;
    }
    at.next(a);
  }
}

template <typename T> struct RingBwd {       // backward: the upstream row and the input's
  static constexpr int kWords = 2 * sizeof(T);
  static constexpr int kSlots = 2;
  static constexpr size_t kBytes = (size_t)kSlots * kWords * 16 * kThreads;
};

// A warp comes to k's units after its last of q: it sums dgamma of one side
// in registers and puts it away when it comes to the other.
template <typename T, int LP, bool kInter>
__global__ void __launch_bounds__(kThreads, 2) rope_bwd_kernel(const Args a) {
  using R = RingBwd<T>;
  extern __shared__ __align__(16) uint4 ring[];
  using L = Lane<T, LP, kInter>;
  constexpr int kTok = L::kTok;
  float* red = reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(ring) + R::kBytes);   // [kWarps][2][d]
  constexpr uint32_t kSlotWords = R::kWords * kThreads;
  const L me(a);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Place at(a), ahead(a);
  pdl_wait();
  pdl_trigger();
  const T *px = nullptr, *pu = nullptr;      // the next rows to copy, and how many the unit has left
  int pn = 0;
  bool pon = false, pnorm = false;
  auto enter = [&] {
    if (!ahead.more) return;
    const Side& p = a.side[ahead.sd];
    const int64_t t = (int64_t)ahead.tg * kTok + me.tok, in = (int64_t)(ahead.h + me.h_off) * a.d + me.col0;
    pon = me.on && t < a.T;
    pnorm = p.gamma != nullptr;
    pu = static_cast<const T*>(p.up) + t * p.us + in;
    px = static_cast<const T*>(p.x) + t * p.xs + in;
    pn = ahead.h_end - ahead.h;
  };
  enter();
  uint32_t so = threadIdx.x;
  auto copy = [&] {
    if (pn > 0) {
      if (pon && me.h_off < pn) {
        const uint32_t dst = tc::smem_u32(ring + so);
        me.copy(dst, pu);
        if (pnorm) me.copy(dst + R::kWords / 2 * kThreads * 16, px);
      }
      pu += a.d * L::kSide;
      px += a.d * L::kSide;
      if ((pn -= L::kSide) <= 0) {
        ahead.next(a);
        enter();
      }
    }
    copy_commit();
    so = so + kSlotWords >= R::kSlots * kSlotWords ? threadIdx.x : so + kSlotWords;
  };
#pragma unroll
  for (int s = 0; s < R::kSlots; ++s) {
    // lanes beyond the head's columns copy nothing and add zeros to its sums
#pragma unroll
    for (int w = 0; w < R::kWords; ++w) ring[so + w * kThreads] = make_uint4(0, 0, 0, 0);
    copy();
  }
  if (a.partial) {
    for (int e = lane; e < 2 * a.d; e += 32) red[warp * 2 * a.d + e] = 0.f;
    __syncwarp();
  }
  float acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  auto put_away = [&](int sd) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float v = rows_sum<LP>(acc[e]);
      if (lane < LP && me.on) red[(warp * 2 + sd) * a.d + me.col(e / me.V) + e % me.V] = v;
      acc[e] = 0.f;
    }
  };
  float gm[16];
  int sd = -1;                               // the side acc and gm are of
  while (at.more) {
    const Side& p = a.side[at.sd];
    const int64_t first = (int64_t)at.tg * kTok, t = first + me.tok;
    int64_t pos;
    const bool write = lane_position(a, min64(t, a.T - 1), first, (int)min64(kTok, a.T - first), pos) && me.on &&
                       t < a.T;
    const bool norm = p.gamma != nullptr;
    T* y = static_cast<T*>(p.out) + t * p.os + (int64_t)(at.h + me.h_off) * a.d + me.col0;
    float c[8], sn[8];
    me.angles(a, pos, c, sn);
    if (sd != at.sd) {
      if (sd >= 0 && a.partial) put_away(sd);
      sd = at.sd;
      me.gamma(p.gamma, gm);
    }
    for (int n = at.h_end - at.h; n > 0; n -= L::kSide) {
      copy_wait<R::kSlots - 1>();
      const bool live = write && me.h_off < n;
      float v[16], g[16];
      read_row<T>(ring + so, v);
      // the transposed rotation
      if (!me.rotated) {
#pragma unroll
        for (int e = 0; e < 16; ++e) g[e] = v[e];
      } else if constexpr (kInter) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float x, z;
          fmul2(v[2 * e + 1], v[2 * e], sn[e], -sn[e], x, z);
          ffma2(v[2 * e], v[2 * e + 1], c[e], c[e], x, z, g[2 * e], g[2 * e + 1]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          float x, z;
          fmul2(v[8 + e], v[9 + e], sn[e], sn[e + 1], x, z);
          ffma2(v[e], v[e + 1], c[e], c[e + 1], x, z, g[e], g[e + 1]);
          fmul2(v[e], v[e + 1], -sn[e], -sn[e + 1], x, z);
          ffma2(v[8 + e], v[9 + e], c[e], c[e + 1], x, z, g[8 + e], g[9 + e]);
        }
      }
      if (norm) {
        read_row<T>(ring + so + R::kWords / 2 * kThreads, v);
        // A row that is not there (a token beyond the last, a head beyond the unit's: its words are an earlier
        // row's, the other side's perhaps), or that the offsets place nowhere, adds nothing.  Zeros, not a factor
        // of zero, which would let NaN and infinities through.
        if (__any_sync(0xffffffffu, me.on && !live)) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            v[e] = live ? v[e] : 0.f;
            g[e] = live ? g[e] : 0.f;
          }
        }
        const float r = rsqrtf(fmaf(group_sum<LP>(dot16(v, v)), a.inv_d, a.eps));
        // eps 0 and a row of zeros: r is infinite, and a row that is not there has nothing to multiply by it
        const float keep = live ? r : 0.f;
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          fmul2(v[e], v[e + 1], keep, keep, v[e], v[e + 1]);
          ffma2(g[e], g[e + 1], v[e], v[e + 1], acc[e], acc[e + 1], acc[e], acc[e + 1]);
          fmul2(g[e], g[e + 1], gm[e], gm[e + 1], g[e], g[e + 1]);
        }
        const float mean = -group_sum<LP>(dot16(g, v)) * a.inv_d;
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          ffma2(v[e], v[e + 1], mean, mean, g[e], g[e + 1], g[e], g[e + 1]);
          fmul2(g[e], g[e + 1], r, r, g[e], g[e + 1]);
        }
      }
      copy();
      if (live) me.store(y, g);
      y += a.d * L::kSide;
    }
    at.next(a);
  }
  if (!a.partial) return;
  if (sd >= 0) put_away(sd);
  __syncthreads();
  for (int e = threadIdx.x; e < 2 * a.d; e += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += red[w * 2 * a.d + e];
    a.partial[(int64_t)blockIdx.x * 2 * a.d + e] = v;
  }
}

// dgamma of side blockIdx.y: the sum of the CTAs' partials, in CTA order
// within each of 32 strides, then across the strides.
__global__ void __launch_bounds__(1024) rope_dgamma_kernel(const float* partial, int parts, int d, float* dq_gamma,
                                                           float* dk_gamma) {
  __shared__ float red[32][33];
  const int col = threadIdx.x % 32, c = blockIdx.x * 32 + col, w = threadIdx.x / 32, sd = blockIdx.y;
  float* out = sd ? dk_gamma : dq_gamma;
  pdl_wait();
  if (!out) return;
  float v = 0.f;
  if (c < d) {
#pragma unroll 8
    for (int p = w; p < parts; p += 32) v += partial[((int64_t)p * 2 + sd) * d + c];
  }
  red[w][col] = v;
  __syncthreads();
  // warp w sums column w of the strides
  v = red[col][w];
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  if (col == 0 && blockIdx.x * 32 + w < d) out[blockIdx.x * 32 + w] = v;
}

// Lanes of a row: those that leave the fewest of a warp's idle (d = 80: five,
// 30 lanes of 32 at work instead of 20 with eight, 38.5 -> 33.1 us for 30,000
// tokens of 15 heads; d = 160: ten, 71.7 -> 54.3 for 25,000 of 18).
int group_lanes(int d) {
  int best = 16;
  for (int lp : {10, 8, 6, 5, 4, 2, 1})
    if (16 * lp >= d && 32 / lp > 32 / best) best = lp;
  return best;
}

template <typename T, int LP, bool kInter>
cudaError_t run(const Args& a, bool bwd, int grid, cudaStream_t s) {
  static_assert(Ring<T>::kBytes <= 48 * 1024, "needs no opt-in");
  if (!bwd) return launch_pdl(rope_fwd_kernel<T, LP, kInter>, dim3(grid), dim3(kThreads), Ring<T>::kBytes, s, a);
  const size_t sums = (size_t)kWarps * 2 * sizeof(float);         // per column
  const cudaError_t e = allow_smem_once<rope_bwd_kernel<T, LP, kInter>>(RingBwd<T>::kBytes + sums * 16 * LP);
  if (e != cudaSuccess) return e;
  return launch_pdl(rope_bwd_kernel<T, LP, kInter>, dim3(grid), dim3(kThreads),
                    RingBwd<T>::kBytes + (a.partial ? sums * a.d : 0), s, a);
}

template <typename T, bool kInter>
cudaError_t run_lp(const Args& a, bool bwd, int grid, cudaStream_t s) {
  switch (group_lanes(a.d)) {
    case 1: return run<T, 1, kInter>(a, bwd, grid, s);
    case 2: return run<T, 2, kInter>(a, bwd, grid, s);
    case 4: return run<T, 4, kInter>(a, bwd, grid, s);
    case 5: return run<T, 5, kInter>(a, bwd, grid, s);
    case 6: return run<T, 6, kInter>(a, bwd, grid, s);
    case 10: return run<T, 10, kInter>(a, bwd, grid, s);
    case 8: return run<T, 8, kInter>(a, bwd, grid, s);
    default: return run<T, 16, kInter>(a, bwd, grid, s);
  }
}

}  // namespace

size_t qk_rope_bwd_workspace_bytes(int d) { return (size_t)kRopeMaxCtas * 2 * (size_t)d * sizeof(float); }

cudaError_t launch_qk_rope(nt_dtype dt, const RopeProblem& p, bool bwd, float* workspace, unsigned int* status,
                           cudaStream_t s) {
  Args a = {};
  a.side[0] = {p.q, p.dq_out, p.q_out, p.q_stride, p.dq_out_stride, p.q_out_stride, p.q_gamma, p.H_q};
  a.side[1] = {p.k, p.dk_out, p.k_out, p.k_stride, p.dk_out_stride, p.k_out_stride, p.k_gamma, p.H_k};
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
  // as in Lane
  const int LP = group_lanes(p.d), row = LP * 16 * (dt == NT_BF16 ? 2 : 4), side = row >= 128 ? 1 : 128 / row;
  const int tok = 32 / LP / side;
  const int64_t groups = (p.T + tok - 1) / tok, warps = min64((int64_t)2 * sm_count(), kRopeMaxCtas) * kWarps;
  // The heads of a unit, a multiple of the rows side by side: the number that
  // gives the fewest steps, the rounds of units times a unit's steps and about
  // three steps' worth of work for its tokens' angles.  (Unit counts stay
  // below 2^31: a unit is 512 bytes of q or k at least, and 2^31 of those are
  // 1 TB.)
  const int most = (max(p.H_q, p.H_k) + side - 1) / side;          // steps of a token group, at most
  const bool one_round = groups * ((p.H_q + side - 1) / side + (p.H_k + side - 1) / side) <= warps;
  int64_t best = 0;
  for (int st = 1; st <= (one_round ? min(most, 1) : most); st = st == 64 ? max(most, 65) : st + 1) {
    const int hu = st * side;
    const int64_t units = groups * ((p.H_q + hu - 1) / hu + (p.H_k + hu - 1) / hu);
    const int64_t cost = (units + warps - 1) / warps * (st + 3);
    if (units > 0x7fffffffLL || (best && cost >= best)) continue;
    best = cost;
    a.unit_heads = hu;
  }
  int64_t total = 0;
  for (int sd = 0; sd < 2 && best; ++sd) {
    a.parts[sd] = max(1, (a.side[sd].H + a.unit_heads - 1) / a.unit_heads);
    a.units[sd] = a.side[sd].H ? (uint32_t)(groups * a.parts[sd]) : 0;
    total += a.units[sd];
  }
  if (total == 0 && p.T > 0 && most > 0) return cudaErrorInvalidValue;
  const int grid = (int)min64((total + kWarps - 1) / kWarps, warps / kWarps);
  cudaError_t e = cudaSuccess;
  if (grid > 0) {
    if (dt == NT_BF16)
      e = p.interleaved ? run_lp<bf16, true>(a, bwd, grid, s) : run_lp<bf16, false>(a, bwd, grid, s);
    else
      e = p.interleaved ? run_lp<float, true>(a, bwd, grid, s) : run_lp<float, false>(a, bwd, grid, s);
  }
  if (e != cudaSuccess || !bwd || !norm) return e;
  return launch_pdl(rope_dgamma_kernel, dim3((p.d + 31) / 32, 2), dim3(1024), 0, s, (const float*)workspace, grid, p.d,
                    p.dq_gamma, p.dk_gamma);
}

}  // namespace nt
