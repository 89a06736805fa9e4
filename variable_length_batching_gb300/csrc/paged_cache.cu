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
constexpr int kWriteTokens = 8;       // tokens a CTA of the write takes

struct WriteArgs {
  const uint8_t* src[2];              // k, v
  uint8_t* pool[2];
  int64_t stride[2];                  // bytes between tokens
  int64_t T;
  int n_pages, page_size, H, row_bytes, B, max_pages;
  const int32_t* cu;
  const int32_t* pos0;
  const int32_t* table;
  unsigned int* status;
};

__global__ void __launch_bounds__(kThreads) paged_write_kernel(const WriteArgs a) {
  __shared__ int64_t dst[kWriteTokens];        // byte offset of the token's row of head 0, or -1
  const int64_t t0 = (int64_t)blockIdx.x * kWriteTokens;
  const int n = (int)min64(kWriteTokens, a.T - t0);
  if (threadIdx.x < n) {
    const int64_t t = t0 + threadIdx.x;
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.cu[mid] <= t) lo = mid; else hi = mid - 1;
    }
    const int start = a.cu[lo];
    int64_t off = -1;
    if (start >= 0 && start <= t && a.cu[lo + 1] > t) {
      const int64_t pos = t - start + (a.pos0 ? a.pos0[lo] : 0);
      const int64_t pg = pos / a.page_size;
      if (pos >= 0 && pg < a.max_pages) {
        const int id = a.table[(int64_t)lo * a.max_pages + pg];
        if (id >= 0 && id < a.n_pages)
          off = ((int64_t)id * a.H * a.page_size + (pos - pg * a.page_size)) * a.row_bytes;
      }
    }
    if (off < 0) flag_device(a.status, kDevCheck);
    dst[threadIdx.x] = off;
  }
  __syncthreads();
  const int row_words = a.row_bytes / 16, side_words = a.H * row_words, tok_words = 2 * side_words;
  const int64_t head_bytes = (int64_t)a.page_size * a.row_bytes;
  for (int e = threadIdx.x; e < n * tok_words; e += kThreads) {
    const int tok = e / tok_words;
    int w = e - tok * tok_words;
    const int sd = w >= side_words;
    w -= sd * side_words;
    const int h = w / row_words, c = w - h * row_words;
    if (dst[tok] < 0) continue;
    const uint4 x = *reinterpret_cast<const uint4*>(a.src[sd] + (t0 + tok) * a.stride[sd] + (int64_t)w * 16);
    *reinterpret_cast<uint4*>(a.pool[sd] + dst[tok] + h * head_bytes + c * 16) = x;
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
  paged_copy_kernel<N><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
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
  paged_write_kernel<<<(unsigned)((T + kWriteTokens - 1) / kWriteTokens), kThreads, 0, s>>>(a);
  return cudaGetLastError();
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
