// The pages of a key/value cache: new keys and values of packed tokens
// written to their sequences' pages, and whole pages copied.
//
// A pool holds pages [n_pages][H_kv][page_size][d]: the rows of one head in a
// page are contiguous, so that attention over the cache reads blocks of
// page_size * d elements.  Both kernels move 16 bytes per thread and access
// and compute nothing: their floor is the bytes read and written.
#include "nt_common.cuh"

namespace nt {
namespace {

constexpr int kThreads = 256;
constexpr int kWriteTokens = 32;      // tokens a CTA of the write takes, at most

struct WriteArgs {
  const uint8_t* src[2];              // k, v
  uint8_t* pool[2];
  int64_t stride[2];                  // bytes between tokens
  int64_t T;
  int n_pages, page_size, H, row_bytes, B, max_pages;
  int tokens;                         // tokens a CTA takes
  const int32_t* cu;
  const int32_t* pos0;
  const int32_t* table;
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

// A warp copies a token's keys, then its values: 16 bytes a lane, kUnroll
// loads in flight.  The rows of a token are contiguous at the source; each
// head's row goes to its own place in the page.
__global__ void __launch_bounds__(kThreads) paged_write_kernel(const WriteArgs a) {
  constexpr int kUnroll = 4;
  __shared__ int64_t dst[kWriteTokens];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
  const int n = (int)min64(a.tokens, a.T - t0);
  pdl_wait();
  pdl_trigger();
  if (n <= kThreads / 32) {
    if (warp < n) {
      const int b = segment_of_warp(a.cu, a.B, t0 + warp);
      if (lane == 0) dst[warp] = write_offset(a, t0 + warp, b);
    }
  } else {
    for (int i = threadIdx.x; i < n; i += kThreads)
      dst[i] = write_offset(a, t0 + i, segment_of_thread(a.cu, a.B, t0 + i));
  }
  __syncthreads();
  const int row_words = a.row_bytes / 16, words = a.H * row_words;
  const int64_t head_bytes = (int64_t)a.page_size * a.row_bytes;
  // units of kUnroll x 32 words of one side of one token, over the warps
  const int per = (words + 32 * kUnroll - 1) / (32 * kUnroll), units = n * 2 * per;
  for (int u = warp; u < units; u += kThreads / 32) {
    const int tok = u / (2 * per), rest = u - tok * 2 * per;
    const int sd = rest >= per, w0 = (rest - sd * per) * 32 * kUnroll + lane;
    const int64_t off = dst[tok];
    if (off < 0) continue;
    const uint8_t* src = a.src[sd] + (t0 + tok) * a.stride[sd];
    uint8_t* out = a.pool[sd] + off;
    uint4 x[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k)
      if (w0 + 32 * k < words) x[k] = *reinterpret_cast<const uint4*>(src + (int64_t)(w0 + 32 * k) * 16);
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int w = w0 + 32 * k;
      if (w >= words) continue;
      const int h = w / row_words, c = w - h * row_words;
      *reinterpret_cast<uint4*>(out + h * head_bytes + c * 16) = x[k];
    }
  }
}

// The copy's page list travels in the launch's arguments: nothing is copied
// to the device first, and a captured launch keeps its list.
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
                               int max_pages, unsigned int* status, cudaStream_t s) {
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
  a.status = status;
  // one token per CTA until that fills the SMs four times
  a.tokens = 1;
  while (a.tokens < kWriteTokens && T >= (int64_t)sm_count() * 4 * a.tokens * 2) a.tokens <<= 1;
  return launch_pdl(paged_write_kernel, dim3((unsigned)((T + a.tokens - 1) / a.tokens)), dim3(kThreads), 0, s, a);
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
