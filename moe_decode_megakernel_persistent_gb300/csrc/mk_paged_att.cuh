// What the attention kernels over the 16-bit paged cache share (mk_paged_attention.cu,
// mk_paged_wide.cu, mk_paged_mass.cu).  The split of the work, the bounded waits and the
// join of split items are those of the 4-bit cache's attention (mk_kv4_att.cuh).
//
// A page's K (or V) of one kv head is 128 rows of head_dim values in one range, which one
// tensor copy (TMA) brings into shared memory as [head_dim / 64][positions][128 bytes]
// with the 128-byte swizzle: what ldmatrix reads without bank conflicts and what
// tcgen05.mma takes as an operand, K by dimensions and V by positions.  A page outside the
// pool is copied from rows behind it, which the copy fills with zeros.
#pragma once
#include <cuda.h>

#include "mk_kv4_att.cuh"
#include "mk_paged.cuh"

namespace mk {

struct PagedAtt {
  AttArgs t;         // t.c = scale * log2(e)
  float* scores;     // workspace: [n_seqs][n_kv_heads][128 * max_pages][score_cols] in log2, or null
  int32_t score_cols;
  char* mass_ws;     // workspace of the masses without scores
};

__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int row, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(0), "r"(row), "r"(0), "r"(bar)
      : "memory");
}
// As bar_wait, without a call: a kernel whose warps split its registers unequally has none.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* give_up, int32_t* status) {
  if (bar_try(bar, parity)) return true;
  const uint64_t t0 = now_ns();
  for (uint32_t i = 0;; ++i) {
    if (bar_try(bar, parity)) return true;
    if (*give_up) return false;
    if ((i & 15u) == 15u && now_ns() - t0 > kWaitNs) {
      *give_up = 1;
      if (status) atomicCAS(status, 0, MK_ERR_BARRIER_TIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ void expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Of two bf16 values, bits 15 and 31: those that are no finite numbers.
__device__ __forceinline__ uint32_t odd_ones(uint32_t x) { return ((x & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }

// An fp32 value as three bf16 ones of its sign, by truncation: 3 x 8 bits are all of its 24.  A part
// that would be 0 is 2^-126 instead (2^-26 of the value at most, else left 0), because 0 times an
// infinite K is NaN where the value times it is infinite.
struct Parts {
  uint32_t h[3];  // bf16 in the high half
};
__device__ __forceinline__ Parts parts_of(float x) {
  Parts r;
  float rest = x;
  const uint32_t tiny = fabsf(x) >= 7.8886091e-31f ? (__float_as_uint(x) & 0x80000000u) | 0x00800000u : 0u;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    r.h[i] = __float_as_uint(rest) & 0xFFFF0000u;
    rest -= __uint_as_float(r.h[i]);
    if (i == 0 && fabsf(x) == INFINITY) rest = 0.f;  // (not inf - inf)
    if (i && !(r.h[i] << 1)) r.h[i] = tiny;
  }
  return r;
}
// Part i of two values as a word.
__device__ __forceinline__ uint32_t both(const Parts& lo, const Parts& hi, int i) { return __byte_perm(lo.h[i], hi.h[i], 0x7632); }

// What of V is no finite number, over a run's positions: the first +infinity, -infinity and NaN of the dimensions
// HD / 32 lane + i.  Where one is seen, the products may have made NaN of an infinity (times a weight, or a
// part of it, that is 0 or negative): the result is these values' sum instead.  Called by a warp, which reads the run's rows
// once (a thread for a column and two dimensions at a time took 280 times as long as the attention of 16384 positions,
// and other warps' waits ran out beyond 200000).
template <int HD>
struct Odd {
  int first[HD / 32][3];
  __device__ __forceinline__ void search(const Kv4Args& a, int seq, int head, int from, int to) {
    constexpr int V = HD / 32;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < V; ++i) first[i][0] = first[i][1] = first[i][2] = INT_MAX;
#pragma unroll 1
    for (int q = from, end; q < to; q = end) {
      end = min(to, (q / kPageTokens + 1) * kPageTokens);
      const int page = table_row(a, seq)[q / kPageTokens];
      if (page < 0 || page >= a.n_pages) continue;
      const uint32_t* v = reinterpret_cast<const uint32_t*>(paged_at<HD>(a, paged_row(a, page, 1, head, q)) + V * lane);
#pragma unroll 8
      for (int p = q; p < end; ++p, v += HD / 2) {
        uint32_t x[V / 2];
        if constexpr (V == 4) {
          const uint2 y = *reinterpret_cast<const uint2*>(v);
          x[0] = y.x, x[1] = y.y;
        } else {
          x[0] = *v;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const uint32_t w = i & 1 ? x[i / 2] >> 16 : x[i / 2] & 0xFFFFu;
          first[i][0] = min(first[i][0], w == 0x7F80u ? p : INT_MAX);
          first[i][1] = min(first[i][1], w == 0xFF80u ? p : INT_MAX);
          first[i][2] = min(first[i][2], (w & 0x7FFFu) > 0x7F80u ? p : INT_MAX);
        }
      }
    }
  }
  // The sum over the positions below lim in dimension d (0: there is none); called by the whole warp.
  __device__ __forceinline__ float sum(int d, int lim) const {
    constexpr int V = HD / 32;
    int at[3] = {INT_MAX, INT_MAX, INT_MAX};
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int x = 0; x < 3; ++x) {
        const int y = __shfl_sync(0xffffffffu, first[i][x], d / V);
        if (d % V == i) at[x] = y;
      }
    return at[2] < lim || (at[0] < lim && at[1] < lim) ? NAN : at[0] < lim ? INFINITY : at[1] < lim ? -INFINITY : 0.f;
  }
};
// Pairs of fp32 in one instruction, and the largest of three.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t z;
  asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(x), "f"(y));
  return z;
}
__device__ __forceinline__ float2 unpair(uint64_t z) {
  float2 x;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x.x), "=f"(x.y) : "l"(z));
  return x;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ bool is_finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// The wide kernel (mk_paged_wide.cu): tiles of CT columns and SP positions; null: none.
WideKernel paged_wide_kernel(int head_dim, int dtype, int cols, long long steps);
const void* paged_wide_join(int head_dim, int dtype);  // blocks of 256 threads for 16 columns of an item
// Rows of head_dim bf16 values as a tensor map whose copies bring `box` rows.
int rows_map(CUtensorMap* map, const void* base, long long rows, int head_dim, int box);
int device_sms();
// Masses from the scores that the narrow kernel kept, or formed again (mk_paged_mass.cu), and
// the workspace that these take.
bool paged_mass_fits(const Kv4Args& a, int n_heads, int dtype, bool wide);  // false: too large a call
size_t paged_mass_bytes(const Kv4Args& a, int head_dim, int n_heads, int dtype);
// What needs no log-sum-exp, before the attention.
cudaError_t paged_mass_begin(const PagedAtt& p, int head_dim, int dtype, cudaStream_t st);
cudaError_t paged_mass(const PagedAtt& p, const PagedMass& m, int head_dim, int dtype, const CUtensorMap& map, cudaStream_t st);

}  // namespace mk
