// The masses of cached positions: what a call's rows gave each of them.
//
// mass[p] = decay mass[p] (0 for the call's own new positions) + sum over the rows r that see
// p and the heads h of its kv head of 2^(s_rhp - lse_rh log2 e).  Calls of a few columns kept
// their scores (mk_paged_attention.cu): 4 bytes a column and position instead of
// K's 2 head_dim.
#include <algorithm>
#include <type_traits>

#include "mk_paged_att.cuh"

namespace mk {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// A thread for a position: its columns' scores in words of four.
__global__ void __launch_bounds__(256) k_mass_scores(const __grid_constant__ PagedAtt pa, const __grid_constant__ PagedMass ms, int chunks) {
  const AttArgs& p = pa.t;
  const int item = blockIdx.x / chunks, t = (blockIdx.x - item * chunks) * 256 + threadIdx.x;
  const int seq = item / p.a.n_kv_heads, head = item - seq * p.a.n_kv_heads;
  int len, nn;
  seq_extent(p.a, seq, len, nn);
  if (t >= len || nn == 0) return;
  float* to = ms.p + seq * ms.seq + head * ms.head + t;
  const float old = t < len - nn ? *to : 0.f;
  float sum = 0.f;  // (the weights by themselves: next to a large mass each would be rounded to its step)
  const bool there = page_of(p.a, seq, t) >= 0;
  const float* sc = pa.scores + ((size_t)item * p.a.max_pages * kPageTokens + t) * pa.score_cols;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (there)
    for (int c0 = 0; c0 < p.cols; c0 += 4) {
      const float4 s4 = *reinterpret_cast<const float4*>(sc + c0);
      const float s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int c = c0 + x;
        if (c >= p.cols) break;
        const int row = row_of(p, c);
        if (row >= nn || t >= len - nn + row + 1) continue;
        const float lse = p.lse[((size_t)seq * p.a.rows + row) * p.n_heads + head * p.gqa + c - row * p.gqa];
        if (lse != -INFINITY) sum += exp2_fast(fmaf(lse, -kLog2e, s[x]));
      }
    }
  *to = t < len - nn ? fmaf(ms.decay, old, sum) : sum;
}

template <int HD, class T>
__global__ void __launch_bounds__(128) k_mass(const __grid_constant__ PagedAtt pa, const __grid_constant__ PagedMass ms) {
  const AttArgs& p = pa.t;
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
        for (int i = 0; i < HD; ++i) s = fmaf((float)q[i], (float)k[i], s);
        const float lse = p.lse[((size_t)seq * p.a.rows + row) * p.n_heads + hd];
        if (lse != -INFINITY) sum += exp2f(fmaf(lse, -kLog2e, s * p.c));
      }
    }
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    float* to = ms.p + seq * ms.seq + head * ms.head + t;
    if (lane == 0) *to = t < len - nn ? fmaf(ms.decay, *to, sum) : sum;
  }
}

}  // namespace

cudaError_t paged_mass(const PagedAtt& p, const PagedMass& m, int head_dim, int dtype, const CUtensorMap& map, cudaStream_t st) {
  const Kv4Args& a = p.t.a;
  const long long items = (long long)a.n_seqs * a.n_kv_heads;
  if (p.scores) {
    const int chunks = (a.max_pages * kPageTokens + 255) / 256;
    if (items * chunks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 0;
    cfg.gridDim = dim3((unsigned)(items * chunks));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_mass_scores, p, m, chunks);
  }
  const int grid = (int)std::min<long long>(items * a.max_pages * (kPageTokens / 4), 1 << 20);
  if (head_dim == 64 && dtype == MK_F32) k_mass<64, float><<<grid, 128, 0, st>>>(p, m);
  else if (head_dim == 64) k_mass<64, __nv_bfloat16><<<grid, 128, 0, st>>>(p, m);
  else if (dtype == MK_F32) k_mass<128, float><<<grid, 128, 0, st>>>(p, m);
  else k_mass<128, __nv_bfloat16><<<grid, 128, 0, st>>>(p, m);
  return cudaGetLastError();
}

}  // namespace mk
