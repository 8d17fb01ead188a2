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

// Eight values of a row.
struct V8 {
  float x[8];
};
__device__ __forceinline__ V8 read8(const float* p) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ V8 read8(const __nv_bfloat16* p) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  V8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v.x[2 * i] = __uint_as_float(u[i] << 16);
    v.x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
  return v;
}
__device__ __forceinline__ void write8(float* p, const V8& v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v.x[0], v.x[1], v.x[2], v.x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v.x[4], v.x[5], v.x[6], v.x[7]);
}
__device__ __forceinline__ void write8(__nv_bfloat16* p, const V8& v) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v.x[2 * i], v.x[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

// A thread's part of a token's rows: sixteen values of one group, so that four
// lanes take a group (two 16-byte loads of bf16, one 8-byte store of codes each)
// and a token is 8 * NG * n_kv_heads parts.
constexpr int kLanes = 4;
template <int HD>
struct Part {
  int kv, head, group, lane;
  __device__ __forceinline__ explicit Part(int i, int n_kv_heads) {
    lane = i % kLanes;
    group = i / kLanes % Tile<HD>::NG;
    head = i / (kLanes * Tile<HD>::NG);
    kv = head >= n_kv_heads;
    head -= kv ? n_kv_heads : 0;
  }
};

constexpr int kThreadsKv = 256;  // the most threads of a block

// Rows of one pass over a block's threads (a block stays within a sequence).
inline int pass_rows(int parts, int rows) { return std::max(1, std::min(kThreadsKv / parts, rows)); }

// The tile half that a row's values of this part lie in (null: padding, or a page
// outside the pool), and its row there.
template <int HD>
__device__ __forceinline__ uint8_t* place_of(const Kv4Args& a, const Part<HD>& pt, int seq, int row, int* at) {
  int len, nn;
  seq_extent(a, seq, len, nn);
  const int p = row < nn ? len - nn + row : -1, page = p >= 0 ? page_of(a, seq, p) : -1;
  *at = p % kTile;
  return page >= 0 ? tile_of<HD>(a, page, pt.head, p) + pt.kv * Tile<HD>::V : nullptr;
}

__device__ __forceinline__ float value_of(uint32_t code, float s) {
  const float m = (float)(code & 7u) * s;
  return code & 8u ? -m : m;
}

// One pass over the rows each way, a part of a row each thread.  Short calls are
// bound by two dependent reads (length, page), which the rows' own reads do not wait
// for (one row each of 16 sequences, 4 heads of 128: 2.0 us); long ones by issue, the
// quotient and the packing (4096 rows: 5.3 us for 10.6 MB; with eight values a thread, half
// the work beside a fixed part, 6.3; with two rows a thread 5.9).
// The division |x| / s is the IEEE quotient: r = RN(1 / s), q = RN(x r), then
// q + r (x - q s) in two fused steps (Markstein), which rounds correctly where
// nothing under- or overflows; scales outside [2^-60, 2^60] take the division itself.
template <int HD, class T>
__global__ void __launch_bounds__(kThreadsKv) k_kv4_store(const __grid_constant__ Kv4Args a, Kv4Rows k, Kv4Rows v, int tp, int chunks) {
  const int parts = 2 * kLanes * Tile<HD>::NG * a.n_kv_heads;
  const int seq = blockIdx.x / chunks, row_base = (blockIdx.x - seq * chunks) * tp;
  const int tk = parts < (int)blockDim.x ? threadIdx.x / parts : 0, row = row_base + tk;
  for (int i0 = 0; i0 < parts; i0 += blockDim.x) {
    const int i = i0 + threadIdx.x - tk * parts;
    const bool mine = tk < tp && i < parts;
    const Part<HD> pt(mine ? i : 0, a.n_kv_heads);
    const Kv4Rows& r = pt.kv ? v : k;
    const int there = min(row, a.rows - 1);
    long long off = seq * r.seq + there * r.row + pt.head * r.head;
    if (r.slot) {  // rows that lie in their slots of a page
      int len, nn;
      seq_extent(a, seq, len, nn);
      off += max(len - nn + there, 0) % kPageTokens * r.slot;
    }
    const T* src = reinterpret_cast<const T*>(r.p) + off + pt.group * kGroup + 16 * pt.lane;
    const V8 x[2] = {read8(src), read8(src + 8)};
    int at;
    uint8_t* t = place_of<HD>(a, pt, seq, row, &at);
    // largest |x| of the group as bits (a NaN's are above an infinity's); every lane takes part
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) top = max(top, __float_as_uint(fabsf(x[e / 8].x[e % 8])));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (!t || !mine) continue;
    // a group with a NaN or an infinity reads back as NaN
    const bool finite = top < 0x7F800000u;
    const __nv_bfloat16 sb = __float2bfloat16_rn(__uint_as_float(top) / 7.f);
    const float s = finite ? __bfloat162float(sb) : 0.f;
    uint32_t c[2] = {0, 0};
    if (s >= 8.6736174e-19f && s <= 1.1529215e18f) {
      const float rs = __frcp_rn(s);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float z = x[e / 8].x[e % 8], y = fabsf(z), q0 = y * rs, q = fmaf(fmaf(-q0, s, y), rs, q0);
        const uint32_t m = __float_as_uint(q + 12582912.f) & 7u;  // rounds to even; at most 7 (q <= 7 (1 + 2^-8))
        c[e / 8] |= (m | (m ? __float_as_uint(z) >> 28 & 8u : 0u)) << (4 * (e % 8));
      }
    } else if (s > 0.f) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float z = x[e / 8].x[e % 8];
        const uint32_t m = (uint32_t)fminf(rintf(fabsf(z) / s), 7.f);
        c[e / 8] |= (m | (m && z < 0.f ? 8u : 0u)) << (4 * (e % 8));
      }
    }
    *reinterpret_cast<uint2*>(t + at * Tile<HD>::ROW + pt.group * (kGroup / 2) + 8 * pt.lane) = make_uint2(c[0], c[1]);
    if (pt.lane == 0)
      *reinterpret_cast<uint16_t*>(t + Tile<HD>::CODES + (at * Tile<HD>::NG + pt.group) * 2) =
          finite ? __bfloat16_as_ushort(sb) : (uint16_t)0x7FC0;
  }
}

// The reverse, bound alike: 4096 rows 4.6 us.
template <int HD, class T>
__global__ void __launch_bounds__(kThreadsKv) k_kv4_load(const __grid_constant__ Kv4Args a, Kv4Rows k, Kv4Rows v, int tp, int chunks) {
  const int parts = 2 * kLanes * Tile<HD>::NG * a.n_kv_heads;
  const int seq = blockIdx.x / chunks, row_base = (blockIdx.x - seq * chunks) * tp;
  const int tk = parts < (int)blockDim.x ? threadIdx.x / parts : 0, row = row_base + tk;
  if (tk >= tp || row >= a.rows) return;
  for (int i = threadIdx.x - tk * parts; i < parts; i += blockDim.x) {
    const Part<HD> pt(i, a.n_kv_heads);
    const Kv4Rows& r = pt.kv ? v : k;
    T* dst = reinterpret_cast<T*>(const_cast<void*>(r.p)) + seq * r.seq + row * r.row + pt.head * r.head +
             pt.group * kGroup + 16 * pt.lane;
    int at;
    const uint8_t* t = place_of<HD>(a, pt, seq, row, &at);
    uint2 c = make_uint2(0, 0);
    uint32_t sc = 0;
    if (t) {
      c = *reinterpret_cast<const uint2*>(t + at * Tile<HD>::ROW + pt.group * (kGroup / 2) + 8 * pt.lane);
      sc = *reinterpret_cast<const uint16_t*>(t + Tile<HD>::CODES + (at * Tile<HD>::NG + pt.group) * 2);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      V8 x;
#pragma unroll
      for (int e = 0; e < 8; ++e) x.x[e] = value_of((h ? c.y : c.x) >> (4 * e), __uint_as_float(sc << 16));
      write8(dst + 8 * h, x);
    }
  }
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


// Launch KERNEL<head_dim, element type>.
#define MK_KV4_LAUNCH(KERNEL, C, HDIM, DT, ST, K, V)                                                     \
  do {                                                                                                   \
    const int parts_ = 2 * kLanes * (HDIM / kGroup) * (C).n_kv_heads, tp_ = pass_rows(parts_, (C).rows); \
    const int threads_ = std::min(kThreadsKv, (tp_ * parts_ + 31) / 32 * 32);                            \
    const int chunks_ = ((C).rows + tp_ - 1) / tp_, grid_ = (C).n_seqs * chunks_;                        \
    if (HDIM == 64 && DT == MK_F32) KERNEL<64, float><<<grid_, threads_, 0, ST>>>(C, K, V, tp_, chunks_); \
    else if (HDIM == 64) KERNEL<64, __nv_bfloat16><<<grid_, threads_, 0, ST>>>(C, K, V, tp_, chunks_);   \
    else if (DT == MK_F32) KERNEL<128, float><<<grid_, threads_, 0, ST>>>(C, K, V, tp_, chunks_);        \
    else KERNEL<128, __nv_bfloat16><<<grid_, threads_, 0, ST>>>(C, K, V, tp_, chunks_);                  \
  } while (0)

int kv4_store(const Kv4Args& a, int head_dim, const Kv4Rows& k, const Kv4Rows& v, int dtype, cudaStream_t st) {
  MK_KV4_LAUNCH(k_kv4_store, a, head_dim, dtype, st, k, v);
  return cuda_status("kv4 store");
}

int kv4_load(const Kv4Args& a, int head_dim, const Kv4Rows& k, const Kv4Rows& v, int dtype, cudaStream_t st) {
  MK_KV4_LAUNCH(k_kv4_load, a, head_dim, dtype, st, k, v);
  return cuda_status("kv4 load");
}

Kv4Args kv4_args(const mk_kv4_cache& c) {
  return {static_cast<uint8_t*>(c.pool), c.table, c.lengths, c.n_new, c.status, c.n_pages, c.n_kv_heads, c.n_seqs,
          c.max_pages, c.rows, nullptr, c.max_pages};
}
Kv4Rows kv4_rows(const mk_kv4_rows& r) { return {r.data, r.seq_stride, r.row_stride, r.head_stride, 0}; }

}  // namespace mk

using namespace mk;

extern "C" MK_API size_t mk_kv4_page_bytes(int32_t n_kv_heads, int32_t head_dim) {
  if (n_kv_heads < 1 || (head_dim != 64 && head_dim != 128)) return 0;
  return (size_t)n_kv_heads * (head_dim == 64 ? Tile<64>::RECORD : Tile<128>::RECORD);
}

// The checks of a store or load, then the launch.
static int store_or_load(int (*f)(const Kv4Args&, int, const Kv4Rows&, const Kv4Rows&, int, cudaStream_t),
                         const mk_kv4_cache* c, const mk_kv4_rows* k, const mk_kv4_rows* v, int32_t dtype, void* stream) {
  host_clear_error();
  bool empty = false;
  if (int r = kv4_check_cache(c, &empty)) return r;
  if (empty) return MK_OK;
  if (int r = kv4_check_rows(k, dtype, "k")) return r;
  if (int r = kv4_check_rows(v, dtype, "v")) return r;
  return f(kv4_args(*c), c->head_dim, kv4_rows(*k), kv4_rows(*v), dtype, (cudaStream_t)stream);
}

extern "C" MK_API int mk_kv4_store(const mk_kv4_cache* c, const mk_kv4_rows* k, const mk_kv4_rows* v, int32_t dtype,
                                   void* stream) {
  return store_or_load(kv4_store, c, k, v, dtype, stream);
}

extern "C" MK_API int mk_kv4_load(const mk_kv4_cache* c, const mk_kv4_rows* k, const mk_kv4_rows* v, int32_t dtype,
                                  void* stream) {
  return store_or_load(kv4_load, c, k, v, dtype, stream);
}
