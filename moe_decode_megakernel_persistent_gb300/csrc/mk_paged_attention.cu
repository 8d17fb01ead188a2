// Causal attention over the 16-bit paged K/V cache, first form: a warp for each
// (row, head), its dimensions over the lanes; the masses by a warp for each
// position, its lanes over the (row, head) pairs, added in a fixed order.
#include <algorithm>
#include <climits>
#include <string>

#include "mk_paged.cuh"

namespace mk {
namespace {

struct PagedAtt {
  Kv4Args a;
  Kv4Rows q, out;
  float* lse;  // what the masses read; may be the workspace
  PagedMass mass;
  float scale;
  int32_t n_heads, gqa;
};

template <int HD, class T>
__global__ void __launch_bounds__(128) k_att(const __grid_constant__ PagedAtt p) {
  constexpr int V = HD / 32;
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int hd = (int)(item % p.n_heads);
  const long long sr = item / p.n_heads;
  const int row = (int)(sr % p.a.rows), seq = (int)(sr / p.a.rows);
  if (seq >= p.a.n_seqs) return;
  int len, nn;
  seq_extent(p.a, seq, len, nn);
  const int lim = row < nn ? max(0, len - nn + row + 1) : 0, head = hd / p.gqa;
  const T* q = reinterpret_cast<const T*>(p.q.p) + seq * p.q.seq + row * p.q.row + hd * p.q.head + lane * V;
  float x[V], o[V], m = -INFINITY, l = 0.f;
  for (int i = 0; i < V; ++i) x[i] = (float)q[i] * p.scale, o[i] = 0.f;
  for (int t = 0; t < lim; ++t) {
    const int page = page_of(p.a, seq, t);
    if (page < 0) continue;
    const __nv_bfloat16* k = paged_at<HD>(p.a, paged_row(p.a, page, 0, head, t)) + lane * V;
    const __nv_bfloat16* v = paged_at<HD>(p.a, paged_row(p.a, page, 1, head, t)) + lane * V;
    float s = 0.f;
    for (int i = 0; i < V; ++i) s = fmaf(x[i], (float)k[i], s);
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    const float nm = fmaxf(m, s), f = m == -INFINITY ? 0.f : expf(m - nm), w = nm == -INFINITY ? 0.f : expf(s - nm);
    m = nm;
    l = l * f + w;
    for (int i = 0; i < V; ++i) o[i] = fmaf(w, (float)v[i], o[i] * f);
  }
  T* out = reinterpret_cast<T*>(const_cast<void*>(p.out.p)) + seq * p.out.seq + row * p.out.row + hd * p.out.head + lane * V;
  for (int i = 0; i < V; ++i) out[i] = (T)(l == 0.f ? 0.f : o[i] / l);
  if (p.lse && lane == 0) p.lse[(sr * p.n_heads) + hd] = l == 0.f ? -INFINITY : m + logf(l);
}

template <int HD, class T>
__global__ void __launch_bounds__(128) k_mass(const __grid_constant__ PagedAtt p) {
  const int lane = threadIdx.x & 31;
  const long long per = (long long)p.a.max_pages * (kPageTokens / 4), all = per * p.a.n_seqs * p.a.n_kv_heads;
  for (long long b = blockIdx.x; b < all; b += gridDim.x) {
  const int t = (int)(b % per) * 4 + (threadIdx.x >> 5), head = (int)(b / per % p.a.n_kv_heads), seq = (int)(b / per / p.a.n_kv_heads);
  int len, nn;
  seq_extent(p.a, seq, len, nn);
  if (t >= len || nn == 0) continue;
  const int page = page_of(p.a, seq, t);
  float sum = 0.f;
  if (page >= 0) {
    const __nv_bfloat16* k = paged_at<HD>(p.a, paged_row(p.a, page, 0, head, t));
    for (int c = lane; c < nn * p.gqa; c += 32) {
      const int row = c / p.gqa, hd = head * p.gqa + c % p.gqa;
      if (t >= len - nn + row + 1) continue;
      const T* q = reinterpret_cast<const T*>(p.q.p) + seq * p.q.seq + row * p.q.row + hd * p.q.head;
      float s = 0.f;
      for (int i = 0; i < HD; ++i) s = fmaf((float)q[i] * p.scale, (float)k[i], s);
      sum += expf(s - p.lse[((size_t)seq * p.a.rows + row) * p.n_heads + hd]);
    }
  }
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  float* to = p.mass.p + seq * p.mass.seq + head * p.mass.head + t;
  if (lane == 0) *to = (t < len - nn ? p.mass.decay * *to : 0.f) + sum;
  }
}

size_t bytes_of(const mk_paged_cache& c, int n_heads) { return (size_t)c.n_seqs * c.rows * n_heads * sizeof(float); }

}  // namespace
}  // namespace mk

using namespace mk;

static int check_attention(const mk_paged_cache* c, int n_heads, int dtype, bool* empty) {
  if (int r = paged_check_cache(c, empty)) return r;
  if (n_heads < 1 || n_heads % c->n_kv_heads || n_heads > 4096)
    return host_fail(MK_ERR_INVALID_ARG, "n_heads must be a multiple of n_kv_heads, at most 4096");
  if (dtype != MK_F32 && dtype != MK_BF16) return host_fail(MK_ERR_INVALID_ARG, "dtype must be MK_F32 or MK_BF16");
  return MK_OK;
}

extern "C" MK_API size_t mk_paged_attention_bytes(const mk_paged_cache* c, int32_t n_heads, int32_t dtype, int32_t with_mass) {
  bool empty = false;
  if (check_attention(c, n_heads, dtype, &empty) || empty) return 0;
  return with_mass ? bytes_of(*c, n_heads) : 0;
}

extern "C" MK_API int mk_paged_attention(const mk_paged_cache* c, int32_t n_heads, const mk_paged_rows* q, int32_t dtype,
                                         float scale, const mk_paged_rows* out, float* lse, const mk_paged_mass* mass,
                                         void* workspace, size_t workspace_bytes, void* stream) {
  host_clear_error();
  bool empty = false;
  if (int r = check_attention(c, n_heads, dtype, &empty)) return r;
  if (!(scale > -1e18f && scale < 1e18f)) return host_fail(MK_ERR_INVALID_ARG, "scale must lie within +-1e18");
  if (empty) return MK_OK;
  if (int r = kv4_check_rows(q, dtype, "q")) return r;
  if (int r = kv4_check_rows(out, dtype, "out")) return r;
  if (mass)
    if (int r = paged_check_mass(mass, c, "mass")) return r;
  const size_t need = mass ? bytes_of(*c, n_heads) : 0;
  if (need && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u) || workspace_bytes < need))
    return host_fail(MK_ERR_INVALID_ARG, "workspace is NULL, not 16-byte aligned or smaller than mk_paged_attention_bytes");
  PagedAtt p = {};
  p.a = kv4_args(*c);
  p.q = kv4_rows(*q);
  p.out = kv4_rows(*out);
  p.lse = lse ? lse : mass ? static_cast<float*>(workspace) : nullptr;
  if (mass) p.mass = {mass->data, mass->seq_stride, mass->head_stride, mass->decay};
  p.scale = scale;
  p.n_heads = n_heads;
  p.gqa = n_heads / c->n_kv_heads;
  cudaStream_t st = (cudaStream_t)stream;
  const dim3 g1((unsigned)(((long long)c->n_seqs * c->rows * n_heads + 3) / 4));
  const dim3 g2((unsigned)std::min<long long>((long long)c->max_pages * kPageTokens / 4 * c->n_kv_heads * c->n_seqs, 1 << 20));
#define RUN(HD, T)                                \
  do {                                            \
    k_att<HD, T><<<g1, 128, 0, st>>>(p);          \
    if (mass) k_mass<HD, T><<<g2, 128, 0, st>>>(p); \
  } while (0)
  if (c->head_dim == 64 && dtype == MK_F32) RUN(64, float);
  else if (c->head_dim == 64) RUN(64, __nv_bfloat16);
  else if (dtype == MK_F32) RUN(128, float);
  else RUN(128, __nv_bfloat16);
#undef RUN
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? MK_OK : host_fail(MK_ERR_CUDA, (std::string("paged attention: ") + cudaGetErrorString(e)).c_str());
}
