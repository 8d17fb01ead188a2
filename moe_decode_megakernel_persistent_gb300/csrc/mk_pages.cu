// Page moves inside a paged pool: page src[i] of every layer is copied to page
// dst[i].  The pool is [n_layers][n_pages][page_bytes], whatever a page holds
// (the bf16 cache's pages, the 4-bit cache's).  Bound by the bytes: a block copies 16 KB
// with 16-byte words, so that one page of 49 layers (12.8 MB) is 784 blocks and takes 4.0
// us, and 150 pages of the 4-bit cache in 49 layers (512 MB, read and written) 151 us, 6.8 TB/s.
#include <algorithm>
#include <string>
#include <vector>

#include "mk_kv4_host.h"

namespace mk {
namespace {

constexpr int kMoves = 448;         // moves carried by one launch
constexpr int kChunk = 16 * 1024;   // bytes a block copies

struct PageMoves {
  uint8_t* pool;
  size_t page_bytes;
  int32_t n_layers, n_pages, n, chunks;  // chunks of a page
  int32_t src[kMoves], dst[kMoves];
};

__global__ void __launch_bounds__(256) k_page_copy(const __grid_constant__ PageMoves a) {
  const long long total = (long long)a.n_layers * a.n * a.chunks;
  for (long long b = blockIdx.x; b < total; b += gridDim.x) {
    const int c = (int)(b % a.chunks), i = (int)(b / a.chunks % a.n), l = (int)(b / a.chunks / a.n);
    const size_t off = (size_t)c * kChunk, end = min(off + kChunk, a.page_bytes);
    const uint8_t* s = a.pool + ((size_t)l * a.n_pages + a.src[i]) * a.page_bytes;
    uint8_t* d = a.pool + ((size_t)l * a.n_pages + a.dst[i]) * a.page_bytes;
    for (size_t o = off + 16 * threadIdx.x; o < end; o += 16 * blockDim.x)
      *reinterpret_cast<uint4*>(d + o) = *reinterpret_cast<const uint4*>(s + o);
  }
}

}  // namespace

int launch_page_copy(void* pool, int n_layers, int n_pages, size_t page_bytes, const int32_t* src, const int32_t* dst,
                     int n, cudaStream_t st) {
  for (int i0 = 0; i0 < n; i0 += kMoves) {
    PageMoves a;
    a.pool = static_cast<uint8_t*>(pool);
    a.page_bytes = page_bytes;
    a.n_layers = n_layers;
    a.n_pages = n_pages;
    a.n = std::min(kMoves, n - i0);
    a.chunks = (int)((page_bytes + kChunk - 1) / kChunk);
    std::copy(src + i0, src + i0 + a.n, a.src);
    std::copy(dst + i0, dst + i0 + a.n, a.dst);
    const long long blocks = (long long)n_layers * a.n * a.chunks;
    k_page_copy<<<(int)std::min(blocks, 1ll << 20), 256, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return host_fail(MK_ERR_CUDA, (std::string("page copy: ") + cudaGetErrorString(e)).c_str());
  }
  return MK_OK;
}

}  // namespace mk

using namespace mk;

extern "C" MK_API int mk_page_copy(void* pool, int32_t n_layers, int32_t n_pages, size_t page_bytes,
                                   const int32_t* src_host, const int32_t* dst_host, int32_t n, void* stream) {
  host_clear_error();
  if (n < 0 || n_layers < 1 || n_pages < 1) return host_fail(MK_ERR_INVALID_ARG, "n must be >= 0, n_layers and n_pages >= 1");
  if (page_bytes < 16 || page_bytes % 16 || page_bytes > (1ull << 40))
    return host_fail(MK_ERR_INVALID_ARG, "page_bytes must be a multiple of 16, at most 2^40");
  if (n == 0) return MK_OK;
  if (!pool || (reinterpret_cast<uintptr_t>(pool) & 15u)) return host_fail(MK_ERR_INVALID_ARG, "pool is NULL or not 16-byte aligned");
  if (!src_host || !dst_host) return host_fail(MK_ERR_INVALID_ARG, "NULL argument");
  try {
    // the moves of a call run at once: a page may be written once, and a page
    // that is written is not read
    std::vector<int32_t> d(dst_host, dst_host + n);
    std::sort(d.begin(), d.end());
    for (int i = 0; i < n; ++i) {
      if (src_host[i] < 0 || src_host[i] >= n_pages || dst_host[i] < 0 || dst_host[i] >= n_pages)
        return host_fail(MK_ERR_INVALID_ARG, "page index out of range");
      if (i && d[i] == d[i - 1]) return host_fail(MK_ERR_INVALID_ARG, "a page is the destination of two moves");
      if (std::binary_search(d.begin(), d.end(), src_host[i]))
        return host_fail(MK_ERR_INVALID_ARG, "a page is both source and destination");
    }
    return launch_page_copy(pool, n_layers, n_pages, page_bytes, src_host, dst_host, n, (cudaStream_t)stream);
  } catch (...) {
    return host_fail(MK_ERR_INVALID_ARG, "page copy: no host memory for the moves");
  }
}
