// The pages of a key/value cache: new keys and values of packed tokens
// written to their sequences' pages, and whole pages copied.
//
// A pool holds pages [n_pages][H_kv][page_size][d]: the rows of one head in a
// page are contiguous, so that attention over the cache reads blocks of
// page_size * d elements.  Both kernels move 16 bytes per thread and access
// and compute nothing: their floor is the bytes read and written (65,536
// tokens of 12 heads of 64 in bf16 written in 66.7 us, 89% of the measured
// copy rate; 2,048 pages of 64 positions copied in 118.5 us, 100%).
#include "nt_common.cuh"

namespace nt {
namespace {

constexpr int kThreads = 256;
constexpr int kWriteTokens = 32;      // tokens a CTA of the write takes, at most

// Division of x < 2^22 by a constant: floor(x m / 2^s), m = ceil(2^s / d), is
// exact while x (m d - 2^s) < 2^s, and m d - 2^s < d <= 2^21.
struct Divisor {
  uint32_t d, m;
  int s;
  __host__ explicit Divisor(uint32_t d_ = 1) : d(d_), m(0), s(0) {
    if (d > (1u << 21)) return;          // m = 0: divide
    while ((1u << s) < d) ++s;
    s += 22;                             // d 2^22 <= 2^s: x (m d - 2^s) < 2^22 d <= 2^s
    m = (uint32_t)(((1ull << s) + d - 1) / d);
  }
  __device__ __forceinline__ uint32_t div(uint32_t x) const {
    return m && x < (1u << 22) ? (uint32_t)((uint64_t)x * m >> s) : x / d;
  }
};

struct WriteArgs {
  const uint8_t* src[2];              // k, v
  uint8_t* pool[2];
  int64_t stride[2];                  // bytes between tokens
  int64_t T;
  int n_pages, page_size, H, row_bytes, B, max_pages;
  int tokens;                         // tokens a CTA takes
  Divisor by_words, by_row;           // 16-byte words of a token's keys, of a row
  const int32_t* cu;
  const int32_t* pos0;
  const int32_t* table;
  const int64_t* slots;               // the tokens' places, where they are given
  unsigned int* status;
};

// Byte offset in the pool of token t's row of head 0, or -1 (flagged).
__device__ __forceinline__ int64_t write_offset(const WriteArgs& a, int64_t t, int b) {
  const int start = a.cu[b];
  int64_t off = -1;
  if (start >= 0 && start <= t && a.cu[b + 1] > t) {
    const int64_t pos = t - start + (a.pos0 ? a.pos0[b] : 0);
    if (pos >= 0 && pos < (int64_t)a.max_pages * a.page_size) {
      const int pg = (int)(pos / a.page_size);
      const int id = a.table[(int64_t)b * a.max_pages + pg];
      if (id >= 0 && id < a.n_pages)
        off = ((int64_t)id * a.H * a.page_size + (pos - (int64_t)pg * a.page_size)) * a.row_bytes;
    }
  }
  if (off < 0) flag_device(a.status, kDevCheck);
  return off;
}

// The same of a token whose place is given; -1 (not flagged) for none.
__device__ __forceinline__ int64_t slot_offset(const WriteArgs& a, int64_t t) {
  const int64_t slot = a.slots[t];
  if (slot < 0 || slot >= (int64_t)a.n_pages * a.page_size) {
    if (slot != -1) flag_device(a.status, kDevCheck);
    return -1;
  }
  const int64_t id = slot / a.page_size;
  return (id * a.H * a.page_size + (slot - id * a.page_size)) * a.row_bytes;
}

// The rows of a token are contiguous at the source; each head's row goes to
// its own place in the page.  The CTA's keys, then its values, are one run of
// 16-byte words over its threads, kUnroll loads in flight: 24 KB per CTA.
// kSlots: the places are given; a kernel of its own (as a branch of one it cost
// the other 0.1 us of 3.1).  Calls among others, 8 heads of 128: 512 tokens 2.5 us by
// slots, 3.1 by offsets and table; 64,000 81.8 and 85.3, the bytes 77.3.
template <bool kSlots>
__global__ void __launch_bounds__(kThreads) paged_write_kernel(const WriteArgs a) {
  constexpr int kUnroll = 6;
  __shared__ int64_t dst[kWriteTokens];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
  const int n = (int)min64(a.tokens, a.T - t0);
  pdl_wait();
  pdl_trigger();
  if constexpr (kSlots) {
    if (threadIdx.x < n) dst[threadIdx.x] = slot_offset(a, t0 + threadIdx.x);
  } else if (n <= kThreads / 32) {
    if (warp < n) {
      const int b = segment_of_warp(a.cu, a.B, t0 + warp);
      if (lane == 0) dst[warp] = write_offset(a, t0 + warp, b);
    }
  } else {
    for (int i = threadIdx.x; i < n; i += kThreads)
      dst[i] = write_offset(a, t0 + i, segment_of_thread(a.cu, a.B, t0 + i));
  }
  __syncthreads();
  const uint32_t words = a.H * (a.row_bytes / 16), total = 2 * n * words;
  const int64_t head_bytes = (int64_t)a.page_size * a.row_bytes;
  for (uint32_t e0 = threadIdx.x; e0 < total; e0 += kThreads * kUnroll) {
    uint4 x[kUnroll];
    uint8_t* to[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const uint32_t e = e0 + k * kThreads;
      to[k] = nullptr;
      if (e >= total) continue;
      const int sd = e >= total / 2;
      const uint32_t r = e - (sd ? total / 2 : 0);
      const uint32_t tok = a.by_words.div(r), w = r - tok * words;
      const uint32_t h = a.by_row.div(w), c = w - h * (a.row_bytes / 16);
      if (dst[tok] < 0) continue;
      x[k] = *reinterpret_cast<const uint4*>(a.src[sd] + (t0 + tok) * a.stride[sd] + (int64_t)w * 16);
      to[k] = a.pool[sd] + dst[tok] + h * head_bytes + c * 16;
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k)
      if (to[k]) *reinterpret_cast<uint4*>(to[k]) = x[k];
  }
}

// The copy's page list travels in the launch's arguments: nothing is copied
// to the device first, and a captured launch keeps its list.  Short lists go
// in short arguments: 32 KB of them take 1.2 us more to launch (16 pages: 2.8
// us of host time, 4.0).
template <int N>
struct CopyArgs {
  uint8_t* pool[2];
  int64_t page_bytes;
  int32_t src[N], dst[N];
};

constexpr int kCopyFew = 448, kCopyMany = 4000;
constexpr int kCopyBytes = 16384;      // bytes of a page a CTA moves

template <int N>
__global__ void __launch_bounds__(kThreads) paged_copy_kernel(const __grid_constant__ CopyArgs<N> a) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.y;
  uint8_t* pool = a.pool[blockIdx.z];
  const int64_t lo = (int64_t)blockIdx.x * kCopyBytes, hi = min64(lo + kCopyBytes, a.page_bytes);
  const uint8_t* s = pool + a.src[i] * a.page_bytes;
  uint8_t* d = pool + a.dst[i] * a.page_bytes;
  for (int64_t o = lo + threadIdx.x * 16; o < hi; o += kThreads * 16)
    *reinterpret_cast<uint4*>(d + o) = *reinterpret_cast<const uint4*>(s + o);
}

template <int N>
cudaError_t copy_pages(const PagedPool& p, const int32_t* src, const int32_t* dst, int n, cudaStream_t s) {
  static_assert(sizeof(CopyArgs<N>) <= 32764, "kernel arguments");
  CopyArgs<N> a;
  a.pool[0] = static_cast<uint8_t*>(p.k);
  a.pool[1] = static_cast<uint8_t*>(p.v);
  a.page_bytes = (int64_t)p.H * p.page_size * p.row_bytes;
  for (int i = 0; i < n; ++i) {
    a.src[i] = src[i];
    a.dst[i] = dst[i];
  }
  const dim3 grid((unsigned)((a.page_bytes + kCopyBytes - 1) / kCopyBytes), n, 2);
  return launch_pdl(paged_copy_kernel<N>, grid, dim3(kThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_paged_write(const PagedPool& p, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                               int64_t T, const int32_t* cu, int B, const int32_t* pos0, const int32_t* table,
                               int max_pages, const int64_t* slots, unsigned int* status, cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  WriteArgs a = {};
  a.src[0] = static_cast<const uint8_t*>(k);
  a.src[1] = static_cast<const uint8_t*>(v);
  a.pool[0] = static_cast<uint8_t*>(p.k);
  a.pool[1] = static_cast<uint8_t*>(p.v);
  a.stride[0] = k_stride;
  a.stride[1] = v_stride;
  a.T = T;
  a.n_pages = p.n_pages;
  a.page_size = p.page_size;
  a.H = p.H;
  a.row_bytes = p.row_bytes;
  a.B = B;
  a.max_pages = max_pages;
  a.cu = cu;
  a.pos0 = pos0;
  a.table = table;
  a.slots = slots;
  a.status = status;
  a.by_words = Divisor(p.H * (p.row_bytes / 16));
  a.by_row = Divisor(p.row_bytes / 16);
  // one token per CTA until that fills the SMs four times (8 heads of 128: 24
  // tokens 2.4 us, with 32 in a CTA 8.5; 65,536 76.5 us, with one 176); at most 2^22 words
  a.tokens = 1;
  while (a.tokens < kWriteTokens && T >= (int64_t)sm_count() * 4 * a.tokens * 2 &&
         (int64_t)a.by_words.d * a.tokens * 4 <= (1 << 22))
    a.tokens <<= 1;
  const auto kernel = slots ? paged_write_kernel<true> : paged_write_kernel<false>;
  return launch_pdl(kernel, dim3((unsigned)((T + a.tokens - 1) / a.tokens)), dim3(kThreads), 0, s, a);
}

cudaError_t launch_paged_copy(const PagedPool& p, const int32_t* src, const int32_t* dst, int64_t n, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  for (int64_t i = 0; i < n && e == cudaSuccess;) {
    const int64_t left = n - i;
    const int c = (int)min64(left, left <= kCopyFew ? kCopyFew : kCopyMany);
    e = left <= kCopyFew ? copy_pages<kCopyFew>(p, src + i, dst + i, c, s)
                         : copy_pages<kCopyMany>(p, src + i, dst + i, c, s);
    i += c;
  }
  return e;
}

}  // namespace nt
