// The 4-bit paged K/V cache of the C ABI: storing rows and loading them back, on
// pools the caller owns (include/mk.h describes the format and the calls;
// mk_kv4_attention.cu reads the cache).
//
// Format.  A row of one (position, kv head) is cut into groups of 64 values
// along head_dim; a group shares s = bf16(max|x| / 7), and a value is a sign
// bit and a magnitude min(7, rint(|x| / s)).  It is the symmetric int4 rule of
// the weights with the code kept as sign and magnitude instead of two's
// complement (-8 cannot occur: |x| / s <= 7 * (1 + 2^-8)).
#include <algorithm>
#include <climits>
#include <string>

#include "mk_kv4.cuh"

namespace mk {
namespace {

__device__ __forceinline__ float4 read4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 read4(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xFFFF0000u));
}
__device__ __forceinline__ void write4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void write4(__nv_bfloat16* p, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  uint2 w;
  w.x = *reinterpret_cast<const uint32_t*>(&a);
  w.y = *reinterpret_cast<const uint32_t*>(&b);
  *reinterpret_cast<uint2*>(p) = w;
}

// Sixteen lanes take one group of one row: four values each.
template <int HD>
struct Unit {
  int seq, row, head, kv, group, lane;
  bool valid;
  __device__ __forceinline__ Unit(const Kv4Args& a) {
    const long long u = ((long long)blockIdx.x * blockDim.x + threadIdx.x) / 16;
    lane = threadIdx.x % 16;
    const long long total = (long long)a.n_seqs * a.rows * a.n_kv_heads * 2 * Tile<HD>::NG;
    valid = u < total;
    long long r = valid ? u : 0;
    group = (int)(r % Tile<HD>::NG);
    r /= Tile<HD>::NG;
    kv = (int)(r % 2);
    r /= 2;
    head = (int)(r % a.n_kv_heads);
    r /= a.n_kv_heads;
    row = (int)(r % a.rows);
    seq = (int)(r / a.rows);
  }
};

// Largest |x| of a group as bits (a NaN's are above an infinity's).
__device__ __forceinline__ uint32_t group_max(float4 x) {
  uint32_t u = max(max(__float_as_uint(fabsf(x.x)), __float_as_uint(fabsf(x.y))),
                   max(__float_as_uint(fabsf(x.z)), __float_as_uint(fabsf(x.w))));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) u = max(u, __shfl_xor_sync(0xffffffffu, u, o));
  return u;
}

__device__ __forceinline__ uint32_t code_of(float x, float s) {
  const float m = s > 0.f ? fminf(rintf(fabsf(x) / s), 7.f) : 0.f;
  return (uint32_t)m | (m > 0.f && x < 0.f ? 8u : 0u);
}

template <int HD, class T>
__global__ void __launch_bounds__(256) k_kv4_store(const __grid_constant__ Kv4Args a, Rows k, Rows v) {
  const Unit<HD> u(a);
  int len, nn;
  seq_extent(a, u.seq, len, nn);
  const int p = len - nn + u.row;
  const bool there = u.valid && u.row < nn && p >= 0;
  const int page = there ? page_of(a, u.seq, p) : -1;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  if (page >= 0) {
    const Rows& r = u.kv ? v : k;
    x = read4(reinterpret_cast<const T*>(r.p) + u.seq * r.seq + u.row * r.row + u.head * r.head + u.group * kGroup + 4 * u.lane);
  }
  const uint32_t top = group_max(x);  // every lane of the warp takes part
  if (page < 0) return;
  uint8_t* t = tile_of<HD>(a, page, u.head, p) + u.kv * Tile<HD>::V;
  const int r = p % kTile;
  // a group with a NaN or an infinity reads back as NaN
  const bool finite = top < 0x7F800000u;
  const __nv_bfloat16 sb = __float2bfloat16_rn(__uint_as_float(top) / 7.f);
  const float s = finite ? __bfloat162float(sb) : 0.f;
  const uint32_t c = code_of(x.x, s) | (code_of(x.y, s) << 4) | (code_of(x.z, s) << 8) | (code_of(x.w, s) << 12);
  *reinterpret_cast<uint16_t*>(t + r * Tile<HD>::ROW + u.group * (kGroup / 2) + 2 * u.lane) = (uint16_t)c;
  if (u.lane == 0)
    *reinterpret_cast<uint16_t*>(t + Tile<HD>::CODES + (r * Tile<HD>::NG + u.group) * 2) =
        finite ? __bfloat16_as_ushort(sb) : (uint16_t)0x7FC0;
}

__device__ __forceinline__ float value_of(uint32_t code, float s) {
  const float m = (float)(code & 7u) * s;
  return code & 8u ? -m : m;
}

template <int HD, class T>
__global__ void __launch_bounds__(256) k_kv4_load(const __grid_constant__ Kv4Args a, Rows k, Rows v) {
  const Unit<HD> u(a);
  if (!u.valid) return;
  int len, nn;
  seq_extent(a, u.seq, len, nn);
  const int p = len - nn + u.row;
  const int page = u.row < nn && p >= 0 ? page_of(a, u.seq, p) : -1;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  if (page >= 0) {
    const uint8_t* t = tile_of<HD>(a, page, u.head, p) + u.kv * Tile<HD>::V;
    const int r = p % kTile;
    const uint32_t c = *reinterpret_cast<const uint16_t*>(t + r * Tile<HD>::ROW + u.group * (kGroup / 2) + 2 * u.lane);
    const float s = __uint_as_float(
        (uint32_t)*reinterpret_cast<const uint16_t*>(t + Tile<HD>::CODES + (r * Tile<HD>::NG + u.group) * 2) << 16);
    x = make_float4(value_of(c, s), value_of(c >> 4, s), value_of(c >> 8, s), value_of(c >> 12, s));
  }
  const Rows& r = u.kv ? v : k;
  write4(reinterpret_cast<T*>(const_cast<void*>(r.p)) + u.seq * r.seq + u.row * r.row + u.head * r.head +
             u.group * kGroup + 4 * u.lane,
         x);
}

int cuda_status(const char* what) {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? MK_OK : host_fail(MK_ERR_CUDA, (std::string(what) + ": " + cudaGetErrorString(e)).c_str());
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

// Checks of a cache description; *empty says that the call has no row.
int kv4_check_cache(const mk_kv4_cache* c, bool* empty) {
  if (!c) return host_fail(MK_ERR_INVALID_ARG, "cache is NULL");
  if (c->head_dim != 64 && c->head_dim != 128) return host_fail(MK_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (c->n_kv_heads < 1 || c->n_kv_heads > 1024) return host_fail(MK_ERR_INVALID_ARG, "n_kv_heads must be in [1, 1024]");
  if (c->n_seqs < 0 || c->rows < 0) return host_fail(MK_ERR_INVALID_ARG, "n_seqs and rows must be >= 0");
  *empty = c->n_seqs == 0 || c->rows == 0;
  if (*empty) return MK_OK;
  if (c->n_pages < 1 || c->max_pages < 1) return host_fail(MK_ERR_INVALID_ARG, "n_pages and max_pages must be >= 1");
  if (c->max_pages > INT_MAX / kPageTokens) return host_fail(MK_ERR_INVALID_ARG, "max_pages x 128 passes 32 bits");
  if ((long long)c->n_seqs * c->rows > INT_MAX / 4096)
    return host_fail(MK_ERR_INVALID_ARG, "n_seqs x rows must be at most 524287");
  if (!c->pool || !aligned16(c->pool)) return host_fail(MK_ERR_INVALID_ARG, "pool is NULL or not 16-byte aligned");
  if (!c->table || !c->lengths) return host_fail(MK_ERR_INVALID_ARG, "table or lengths is NULL");
  return MK_OK;
}

int kv4_check_rows(const mk_kv4_rows* r, int dtype, const char* what) {
  if (dtype != MK_F32 && dtype != MK_BF16) return host_fail(MK_ERR_INVALID_ARG, "dtype must be MK_F32 or MK_BF16");
  const int per = dtype == MK_F32 ? 4 : 8;  // elements of 16 bytes
  if (!r || !r->data || !aligned16(r->data) || r->seq_stride % per || r->row_stride % per || r->head_stride % per)
    return host_fail(MK_ERR_INVALID_ARG, (std::string(what) + ": NULL, or its address or a stride is not a multiple of 16 bytes").c_str());
  return MK_OK;
}

}  // namespace mk

using namespace mk;

extern "C" MK_API size_t mk_kv4_page_bytes(int32_t n_kv_heads, int32_t head_dim) {
  if (n_kv_heads < 1 || (head_dim != 64 && head_dim != 128)) return 0;
  return (size_t)n_kv_heads * (head_dim == 64 ? Tile<64>::RECORD : Tile<128>::RECORD);
}

// Launch KERNEL<head_dim, element type> with GRID blocks of BLOCK threads.
#define MK_KV4_LAUNCH(KERNEL, HD, DT, GRID, BLOCK, ST, ...)                                      \
  do {                                                                                           \
    if (HD == 64 && DT == MK_F32) KERNEL<64, float><<<GRID, BLOCK, 0, ST>>>(__VA_ARGS__);        \
    else if (HD == 64) KERNEL<64, __nv_bfloat16><<<GRID, BLOCK, 0, ST>>>(__VA_ARGS__);           \
    else if (DT == MK_F32) KERNEL<128, float><<<GRID, BLOCK, 0, ST>>>(__VA_ARGS__);              \
    else KERNEL<128, __nv_bfloat16><<<GRID, BLOCK, 0, ST>>>(__VA_ARGS__);                        \
  } while (0)

static int kv4_blocks(const mk_kv4_cache& c) {
  const long long units = (long long)c.n_seqs * c.rows * c.n_kv_heads * 2 * (c.head_dim / kGroup);
  return (int)((units * 16 + 255) / 256);
}

extern "C" MK_API int mk_kv4_store(const mk_kv4_cache* c, const mk_kv4_rows* k, const mk_kv4_rows* v, int32_t dtype,
                                   void* stream) {
  host_clear_error();
  bool empty = false;
  if (int r = kv4_check_cache(c, &empty)) return r;
  if (empty) return MK_OK;
  if (int r = kv4_check_rows(k, dtype, "k")) return r;
  if (int r = kv4_check_rows(v, dtype, "v")) return r;
  MK_KV4_LAUNCH(k_kv4_store, c->head_dim, dtype, kv4_blocks(*c), 256, (cudaStream_t)stream, kv4_args(*c), kv4_rows(*k), kv4_rows(*v));
  return cuda_status("kv4 store");
}

extern "C" MK_API int mk_kv4_load(const mk_kv4_cache* c, const mk_kv4_rows* k, const mk_kv4_rows* v, int32_t dtype,
                                  void* stream) {
  host_clear_error();
  bool empty = false;
  if (int r = kv4_check_cache(c, &empty)) return r;
  if (empty) return MK_OK;
  if (int r = kv4_check_rows(k, dtype, "k")) return r;
  if (int r = kv4_check_rows(v, dtype, "v")) return r;
  MK_KV4_LAUNCH(k_kv4_load, c->head_dim, dtype, kv4_blocks(*c), 256, (cudaStream_t)stream, kv4_args(*c), kv4_rows(*k), kv4_rows(*v));
  return cuda_status("kv4 load");
}
