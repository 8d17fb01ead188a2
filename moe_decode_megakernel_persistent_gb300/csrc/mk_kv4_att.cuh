// What the two attention kernels over the 4-bit cache share (mk_kv4_attention.cu,
// mk_kv4_wide.cu): arguments, bounded waits, and how the work of a call is cut
// into runs.
#pragma once
#include <cuda_fp16.h>

#include <climits>
#include <type_traits>

#include "mk_kv4.cuh"

namespace mk {

constexpr uint64_t kWaitNs = 1000000000ull;        // bound of every wait
constexpr int kList = 256;                         // steps whose addresses a block looks up at a time
constexpr float kLow = -1e30f;                     // running maximum of a column that has seen nothing
constexpr float kLazy = 8.f;                       // a maximum moves when a score passes it by this (log2)
constexpr float kUp = 18446744073709551616.f;      // 2^64, carried by q
constexpr double kDown = 36893488147419103232.0;   // 2^65 = 2^129 / 2^64, taken out of the scores
constexpr float kCode = 1048576.f;                 // 2^20, taken out of the second product

struct AttArgs {
  Kv4Args a;
  Kv4Rows q, out;
  float* lse;
  float c;              // scale * log2(e) * 2^65
  int32_t n_heads, gqa;
  int32_t gqa_log;      // log2(gqa), or -1
  int32_t cols;         // rows * gqa: query columns of a (sequence, kv head)
  int32_t n_ctiles;     // column tiles of it
  int32_t n_entries;    // n_seqs * n_ctiles
  int32_t cluster;      // > 0: an item is one cluster of so many blocks (a power of two), and there is no workspace
  int32_t cluster_log;
  long long* total;     // workspace: places of the call (Runs)
  longlong2* item;      // workspace: [n_entries * n_kv_heads] first place and first block, or -1 (done)
  float* part;          // workspace: [2 * grid][columns][HD + 4] partial results
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Wait for a phase; gives up after kWaitNs (and at once when another warp of the
// block has): then *give_up is set and the block runs to its end without data.
static __device__ __noinline__ bool bar_wait_long(uint32_t bar, uint32_t parity, volatile int* give_up, int32_t* status) {
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
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* give_up, int32_t* status) {
  return bar_try(bar, parity) || bar_wait_long(bar, parity, give_up, status);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {  // bf16x2
  uint32_t y;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
  return y;
}
__device__ __forceinline__ uint32_t pack2h(float lo, float hi) {  // f16x2
  uint32_t y;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
  return y;
}
__device__ __forceinline__ float low_h(uint32_t x) { return __half2float(__ushort_as_half((unsigned short)x)); }
__device__ __forceinline__ float high_h(uint32_t x) { return __half2float(__ushort_as_half((unsigned short)(x >> 16))); }
__device__ __forceinline__ float low_f(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float high_f(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A part's sum of values, taken to the joined maximum.  A factor of 0 leaves infinities and NaN, which reach their
// dimension whatever their weight.  (The joins multiply alone where no part has a factor of 0: selected for every value, one
// row at 2049 positions took 0.3 us more of 7.6.)
__device__ __forceinline__ float taken(float x, float f) { return f == 0.f && !(fabsf(x) <= 3.402823466e38f) ? x : x * f; }
constexpr uint32_t kNib = 0x80708070u;

// The row of a query column.
__device__ __forceinline__ int row_of(const AttArgs& p, int col) {
  return p.gqa_log >= 0 ? col >> p.gqa_log : col / p.gqa;
}

// Column tile j of sequence s: how many steps of SP positions its columns see.
__device__ __forceinline__ int tiles_of(const AttArgs& p, int e, int CT, int SP) {
  const int s = p.n_ctiles == 1 ? e : e / p.n_ctiles, j = e - s * p.n_ctiles;
  int len, nn;
  seq_extent(p.a, s, len, nn);
  if (row_of(p, j * CT) >= nn) return 0;                                  // its rows are padding
  const int r = min(row_of(p, min((j + 1) * CT, p.cols) - 1), nn - 1);    // its last row
  const int end = len - nn + r + 1;
  return end <= 0 ? 0 : (end + SP - 1) / SP;
}

// The runs of a block.  All items are laid end to end, each as kOver places (an
// item's set-up and end cost a block about as much as so many steps) and then
// its steps; the block takes the steps of the places [pos, hi).
constexpr int kOver = 4;
constexpr int kMaxBlocks = 1024;
struct Runs {
  long long pos, hi, base;  // base: the first place of entry e
  int e, nt, head, t0, t1;
  __device__ __forceinline__ void take() {  // the steps of entry e from place pos on
    const int len = nt + kOver, at = (int)(pos - base);  // held to 31 bits by the entry point
    head = at / len;
    const int in = at - head * len;
    const int out = (int)min((long long)len, in + (hi - pos));
    pos += out - in;
    t0 = max(0, in - kOver);
    t1 = max(0, out - kOver);
  }
  __device__ __forceinline__ uint32_t steps(const AttArgs& p, int CT, int SP) const {  // of this run and all after it
    uint32_t n = t1 - t0;
    if (n)
      for (Runs r = *this; r.next(p, CT, SP);) n += r.t1 - r.t0;
    return n;
  }
  __device__ __forceinline__ bool next(const AttArgs& p, int CT, int SP) {  // the next run; false: none is left
    for (;;) {
      if (pos >= hi) return false;
      for (;; ++e) {
        if (e >= p.n_entries) return false;  // lengths that change under the call
        nt = tiles_of(p, e, CT, SP);
        const long long n = nt ? (long long)(nt + kOver) * p.a.n_kv_heads : 0;
        if (pos < base + n) break;
        base += n;
      }
      take();
      if (t1 > t0) return true;
    }
  }
};
// The first place of block b of G: the places cut into equal runs.
__device__ __forceinline__ long long first_place(long long total, long long b, int G) {
  if (total * G < 1ll << 32) return (uint32_t)total * (uint32_t)b / (uint32_t)G;
  return total * b / G;
}
// A partial run that starts inside an item, and one that ends inside it: a
// block has one of each at most, with a place of its own in the workspace.
__device__ __forceinline__ int part_slot(long long block, int t0) { return (int)(2 * block) + (t0 > 0 ? 0 : 1); }

// The first run of this block, found by one warp; lane 0 of block 0 leaves the
// number of places for the join.  Returned in all lanes.
__device__ __forceinline__ Runs first_run(const AttArgs& p, int CT, int SP, int lane) {
  int nt = lane < p.n_entries ? tiles_of(p, lane, CT, SP) : 0;
  auto places = [&] { return nt ? (long long)(nt + kOver) * p.a.n_kv_heads : 0ll; };
  Runs r;
  r.t0 = r.t1 = 0;
  if (p.n_entries <= 32 && __all_sync(0xffffffffu, places() < 1 << 26)) {  // one scan, in 32 bits
    const int n = (int)places();
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const int total = __shfl_sync(0xffffffffu, incl, 31);
    const int lo = (int)first_place(total, blockIdx.x, gridDim.x), hi = (int)first_place(total, blockIdx.x + 1, gridDim.x);
    if (blockIdx.x == 0 && lane == 0) *p.total = total;
    r.pos = lo;
    r.hi = hi;
    if (lo >= hi) return r;
    const int f = __ffs(__ballot_sync(0xffffffffu, lo < incl)) - 1;
    const int base = __shfl_sync(0xffffffffu, incl - n, f);
    r.base = base;
    r.e = f;
    r.nt = __shfl_sync(0xffffffffu, nt, f);
    r.take();
    if (r.t1 <= r.t0 && !r.next(p, CT, SP)) r.t0 = r.t1 = 0;
    return r;
  }
  long long total = places();
  for (int e = lane + 32; e < p.n_entries; e += 32) {
    nt = tiles_of(p, e, CT, SP);
    total += places();
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const long long lo = first_place(total, blockIdx.x, gridDim.x), hi = first_place(total, blockIdx.x + 1, gridDim.x);
  if (blockIdx.x == 0 && lane == 0) *p.total = total;
  long long base = 0;
  int entry = 0;
  if (lo < hi) {
    for (int e0 = 0; e0 < p.n_entries; e0 += 32) {
      nt = e0 + lane < p.n_entries ? tiles_of(p, e0 + lane, CT, SP) : 0;
      const long long n = places();
      long long incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      const uint32_t has = __ballot_sync(0xffffffffu, lo < base + incl);
      if (has) {
        const int f = __ffs(has) - 1;
        entry = e0 + f;
        base += __shfl_sync(0xffffffffu, incl - n, f);
        break;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  r.pos = lo;
  r.hi = hi;
  r.base = base;
  r.e = entry;
  if (!r.next(p, CT, SP)) r.t0 = r.t1 = 0;
  return r;
}

// The wide kernel (mk_kv4_wide.cu).
struct WideKernel {
  const void* fn;
  int CT, SP, smem, blocks, threads;
};
WideKernel kv4_wide_kernel(int head_dim, int dtype);
// The join of split items (mk_kv4_attention.cu), with 4 or 12 (many) parts in flight in a warp.
const void* kv4_join_kernel(int head_dim, int dtype, bool many);

}  // namespace mk
