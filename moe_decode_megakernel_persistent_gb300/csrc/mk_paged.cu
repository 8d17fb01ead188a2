// The 16-bit paged K/V cache of the C ABI: storing rows, and the checks of
// arguments that its calls share (include/mk.h describes them).
#include <algorithm>
#include <climits>
#include <cmath>
#include <string>

#include "mk_paged.cuh"

namespace mk {
namespace {

__device__ __forceinline__ uint32_t two(float lo, float hi) {  // bf16x2, rounded to nearest even
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Eight values (one 16-byte word of the cache) a thread; the length, the page and the
// row itself are read without waiting for one another.  Bound by bytes where there are many (4096 fp32 rows of 4 heads
// of 128, 25 MB: 4.6 us a call, 5.5 TB/s), by the launch where there are few (16 rows 3.1 us).
template <int HD, class T>
__global__ void __launch_bounds__(256) k_paged_store(const __grid_constant__ Kv4Args a, Kv4Rows k, Kv4Rows v) {
  constexpr int W = HD / 8;  // words of a row
  const int parts = 2 * W * a.n_kv_heads;
  const long long at = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long sr = at / parts;
  if (sr >= (long long)a.n_seqs * a.rows) return;
  behind();
  const int part = (int)(at - sr * parts), seq = (int)(sr / a.rows), row = (int)(sr - (long long)seq * a.rows);
  const int w = part % W, kh = part / W, kv = kh >= a.n_kv_heads, head = kh - (kv ? a.n_kv_heads : 0);
  const Kv4Rows& r = kv ? v : k;
  const T* src = reinterpret_cast<const T*>(r.p) + seq * r.seq + row * r.row + head * r.head + 8 * w;
  uint4 x;
  if constexpr (sizeof(T) == 4) {
    const float4 lo = reinterpret_cast<const float4*>(src)[0], hi = reinterpret_cast<const float4*>(src)[1];
    x = make_uint4(two(lo.x, lo.y), two(lo.z, lo.w), two(hi.x, hi.y), two(hi.z, hi.w));
  } else {
    x = *reinterpret_cast<const uint4*>(src);
  }
  int len, nn;
  seq_extent(a, seq, len, nn);
  const int p = row < nn ? len - nn + row : -1;
  if (p < 0) return;
  const int page = page_of(a, seq, p);
  if (page < 0) return;
  reinterpret_cast<uint4*>(paged_at<HD>(a, paged_row(a, page, kv, head, p)))[w] = x;
}

}  // namespace

int paged_check_cache(const mk_paged_cache* c, bool* empty) {
  if (int r = kv4_check_cache(c, empty)) return r;
  if (!*empty && (long long)c->n_pages * 2 * c->n_kv_heads * kPageTokens > INT_MAX)
    return host_fail(MK_ERR_INVALID_ARG, "n_pages x 2 x n_kv_heads x 128 passes 31 bits");
  return MK_OK;
}

int paged_check_mass(const mk_paged_mass* m, const mk_paged_cache* c, const char* what) {
  const auto bad = [&](const char* why) { return host_fail(MK_ERR_INVALID_ARG, (std::string(what) + why).c_str()); };
  if (!m || !m->data || (reinterpret_cast<uintptr_t>(m->data) & 15u)) return bad(" is NULL or not 16-byte aligned");
  if (m->seq_stride < 0 || m->head_stride < 0 || m->seq_stride % 4 || m->head_stride % 4)
    return bad(": a stride is negative or not a multiple of 16 bytes");
  const long long row = (long long)c->max_pages * kPageTokens, all = m->head_stride * (c->n_kv_heads - 1) + row;
  if ((c->n_kv_heads > 1 && m->head_stride < row) || (c->n_seqs > 1 && m->seq_stride < all)) {
    // (heads outside sequences, or sequences outside heads)
    if ((c->n_seqs > 1 && m->seq_stride < row) ||
        (c->n_kv_heads > 1 && m->head_stride < m->seq_stride * (c->n_seqs - 1) + row))
      return bad(": rows of positions overlap");
  }
  if (!std::isfinite(m->decay)) return bad(": decay is not finite");
  return MK_OK;
}

}  // namespace mk

using namespace mk;

extern "C" MK_API int mk_paged_store(const mk_paged_cache* c, const mk_paged_rows* k, const mk_paged_rows* v,
                                     int32_t dtype, void* stream) {
  host_clear_error();
  bool empty = false;
  if (int r = paged_check_cache(c, &empty)) return r;
  if (empty) return MK_OK;
  if (int r = kv4_check_rows(k, dtype, "k")) return r;
  if (int r = kv4_check_rows(v, dtype, "v")) return r;
  Kv4Args a = kv4_args(*c);
  Kv4Rows kr = kv4_rows(*k), vr = kv4_rows(*v);
  const long long n = (long long)c->n_seqs * c->rows * 2 * c->n_kv_heads * (c->head_dim / 8);  // at most 2^19 x 2^15
  void* args[] = {&a, &kr, &vr};
  const void* f = c->head_dim == 64 ? dtype == MK_F32 ? reinterpret_cast<const void*>(&k_paged_store<64, float>)
                                                      : reinterpret_cast<const void*>(&k_paged_store<64, __nv_bfloat16>)
                  : dtype == MK_F32 ? reinterpret_cast<const void*>(&k_paged_store<128, float>)
                                    : reinterpret_cast<const void*>(&k_paged_store<128, __nv_bfloat16>);
  const cudaError_t e = launch(f, (unsigned)((n + 255) / 256), 256, 0, (cudaStream_t)stream, args);
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaSuccess ? MK_OK : host_fail(MK_ERR_CUDA, (std::string("paged store: ") + cudaGetErrorString(e)).c_str());
}
