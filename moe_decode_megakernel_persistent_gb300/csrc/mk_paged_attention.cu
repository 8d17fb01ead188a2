// Causal attention over the 16-bit paged K/V cache (mk_paged_attention): single rows of a
// decode step and a few rows of a sequence (up to 16 to 32 query columns); prompt chunks run in mk_paged_wide.cu.
//
// Mathematics.  For a row q and the positions p it sees, s_p = c q . K_p with c = scale log2 e,
// out = sum_p 2^(s_p - m) V_p / sum_p 2^(s_p - m).  Products are bf16 (mma.sync m16n8k16) with
// fp32 sums: K and V are exact, a bf16 q is exact, an fp32 q is three bf16 parts (24 bits).  The
// weights are two bf16 parts for bf16 rows (16 bits: of one part, 2^-8, the outputs' error against 64 bits was 0.0021 to
// 0.0026 of their size where their own rounding makes 0.0017) and three for fp32 rows; their sum, the maxima and the scores are fp32.
//
// Layout.  K is the first product's A operand (16 positions x 16 dimensions, ldmatrix) and q
// its B operand, so that the query columns of one kv head (rows x heads of the group) fill tiles of
// 8 columns and the 4 heads of a single row cost one.  The weights turn with movmatrix into the
// B operand of the second product, whose A operand is V transposed (ldmatrix.trans).
//
// Work.  The steps of all (sequence, kv head) items are laid end to end and cut into equal
// runs, one for each block, from the lengths on the device.  A block's steps of SP positions stream
// through a ring in shared memory (two tensor copies each), refilled by its warps in turn; each warp takes
// 16 U positions of a step, with running maxima of its own (moved only when a score passes them by 2^8)
// and one merge at the end of an item.  An item cut between blocks is joined by a second kernel,
// whose start overlaps the first one's end; short work makes each item a cluster of blocks that join
// through their shared memory.
//
// What a column does not see must not show in it, and 0 x NaN is NaN: V of positions that no
// column of a step sees is taken as 0, and where columns differ, a V that is no finite number is taken out
// of the product and added to the columns that see it.
//
// Bounds.  Large batches run at the memory's rate: 64 sequences of 4096 to 16384 positions, one row of 16 heads on 4 of 128
// dimensions, read 1.34 GB in 196 us and take 200 to 203 with the join (the copy's rate gives 197).  16 of 256 to 8448 take 31
// (21 by bytes: the join is 5, the start and the runs' ends as much).  One of 2049 takes 7.6, which is the chain
// launch, lengths and pages, first copies, a step or two, join in the cluster.  The few columns leave the tensor cores 13 %
// and the issue slots 13 % busy; 20 columns of one sequence of 8022 take 16.0 (2.4 by bytes: 16 blocks a head, 64 SMs).
#include <algorithm>
#include <atomic>
#include <climits>
#include <string>
#include <type_traits>

#include "mk_paged_att.cuh"

namespace mk {
namespace {

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint2 b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y));
}
__device__ __forceinline__ void ldsm(uint32_t at, uint32_t (&x)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t at, uint32_t (&x)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ uint32_t turn(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Store into another block's shared memory of the cluster.
__device__ __forceinline__ void put_peer(const float* local, int rank, float2 v) {
  uint32_t y;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(y) : "r"(smem_addr(local)), "r"(rank));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1,%2};" ::"r"(y), "f"(v.x), "f"(v.y) : "memory");
}

constexpr int kWindow = 128;  // steps whose places a block looks up at a time

// NT column tiles; W warps of U units of 16 positions in each step; R steps in the ring; B
// blocks of an SM.
template <int HD, class T, int NT, int W, int U, int R, int B>
struct Shape {
  static constexpr bool F32 = std::is_same<T, float>::value;
  static constexpr int CT = 8 * NT;          // columns of a tile
  static constexpr int P = F32 ? 3 : 1;      // bf16 parts of q
  static constexpr int WP = F32 ? 3 : 2;     // and of the weights
  static constexpr int RS = HD + 2;          // floats of a column in the reduction buffer
  static constexpr int SP = 16 * W * U;      // positions of a step, within a page
  static constexpr int HALF = SP * HD * 2;   // bytes of a step's K, or V
  static constexpr int RED = W * CT * RS * 4;
  static constexpr int SMEM = 1024 + R * 2 * HALF + RED;
  static_assert(kPageTokens % SP == 0, "steps within a page");
};

template <int HD, class T, int NT, int W, int U, int R, int B>
__global__ void __launch_bounds__(32 * W, B) k_paged_attention(const __grid_constant__ PagedAtt pa, const __grid_constant__ CUtensorMap map) {
  using S = Shape<HD, T, NT, W, U, R, B>;
  constexpr int CT = S::CT, SP = S::SP, NTHR = 32 * W, DT = HD / 16;
  const AttArgs& p = pa.t;
  extern __shared__ uint8_t sm_raw[];
  uint8_t* sm = sm_raw + ((1024 - (smem_addr(sm_raw) & 1023)) & 1023);
  __shared__ __align__(8) uint64_t full[R], empty[R];
  __shared__ int list[kWindow];     // rows of the pool where the block's next steps lie (-1: a page outside it)
  __shared__ uint32_t issued[R];    // 1 + the last step copied into each stage
  __shared__ float2 sm_ml[W][CT];   // a run's maximum and sum of each warp and column
  // The block's run and its number of steps, found by one thread: all warps pass the
  // same barriers even where someone writes the lengths while the call runs.
  __shared__ Runs s_run;
  __shared__ uint32_t s_steps;
  __shared__ volatile int give_up;
  float* red = reinterpret_cast<float*>(sm + R * 2 * S::HALF);
  // cluster: the partial results of the columns that this block joins, column c
  // (joined by block c mod cluster) of block r in [r][c / cluster][HD | M, sum]
  float* fin = red + W * CT * S::RS;
  // cluster: the first pages of the item's sequence, where the sums are joined at the end
  int* pages = reinterpret_cast<int*>(red);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  // a block's shared memory is there to be written once the block runs
  if (p.cluster > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  if (tid == 0) {
    for (int i = 0; i < R; ++i) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_addr(&full[i])) : "memory");
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(&empty[i])), "n"(W) : "memory");
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    for (int i = 0; i < R; ++i) issued[i] = 0;
    give_up = 0;
  }
  behind();
  // lane (g, t) of the mma fragments
  const int g = lane >> 2, t4 = lane & 3;
  // the B fragments of q: column nt * 8 + g, dimensions 16 j + 2 t + {0, 1} and 8 more
  uint2 qf[S::P][NT][DT];
  auto load_q = [&](int seq, int j, int head) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int col = j * CT + nt * 8 + g;
      const bool there = col < p.cols;
      const int row = there ? row_of(p, col) : 0, hd = there ? col - row * p.gqa : 0;
      const T* src = reinterpret_cast<const T*>(p.q.p) + seq * p.q.seq + row * p.q.row + (head * p.gqa + hd) * p.q.head + 2 * t4;
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        if constexpr (S::F32) {
          float2 x = make_float2(0.f, 0.f), y = x;
          if (there) {
            x = *reinterpret_cast<const float2*>(src + 16 * d);
            y = *reinterpret_cast<const float2*>(src + 16 * d + 8);
          }
          const Parts x0 = parts_of(x.x), x1 = parts_of(x.y), y0 = parts_of(y.x), y1 = parts_of(y.y);
#pragma unroll
          for (int i = 0; i < 3; ++i) qf[i][nt][d] = make_uint2(both(x0, x1, i), both(y0, y1, i));
        } else {
          uint2 b = make_uint2(0, 0);
          if (there) b = make_uint2(*reinterpret_cast<const uint32_t*>(src + 16 * d), *reinterpret_cast<const uint32_t*>(src + 16 * d + 8));
          qf[0][nt][d] = b;
        }
      }
    }
  };
  // Dimensions d, d + 1 of a column's result from its sums.
  auto put_out = [&](int seq, int col, int head, int d, float M, float l_sum, float2 v) {
    const int row = row_of(p, col), hd = head * p.gqa + col - row * p.gqa;
    const float f = 1.f / l_sum;
    v = l_sum == 0.f ? make_float2(0.f, 0.f) : make_float2(v.x * f, v.y * f);
    T* dst = reinterpret_cast<T*>(const_cast<void*>(p.out.p)) + seq * p.out.seq + row * p.out.row + hd * p.out.head + d;
    if constexpr (S::F32) *reinterpret_cast<float2*>(dst) = v;
    else *reinterpret_cast<uint32_t*>(dst) = pack2(v.x, v.y);
    if (p.lse && d == 0)
      p.lse[((size_t)seq * p.a.rows + row) * p.n_heads + hd] =
          l_sum == 0.f ? -INFINITY : (M + log2f(l_sum)) * 0.69314718055994530942f;
  };
  Runs run;
  if (p.cluster) {  // this block's share of its cluster's item, at once with the first reads of pages and q
    const int item = blockIdx.x >> p.cluster_log, rank = blockIdx.x & (p.cluster - 1);
    const int e = item / p.a.n_kv_heads, head = item - e * p.a.n_kv_heads;
    const int seq = p.n_ctiles == 1 ? e : e / p.n_ctiles;
    const int page = tid < p.a.max_pages ? table_row(p.a, seq)[tid] : -1;
    const uint32_t nt = tiles_of(p, e, CT, SP);  // at most 2^24
    load_q(seq, e - seq * p.n_ctiles, head);
    run.base = 0;
    run.e = e;
    run.head = head;
    run.nt = nt;
    run.t0 = nt * rank >> p.cluster_log;
    run.t1 = nt * (rank + 1) >> p.cluster_log;
    pages[tid] = page;
    if (tid == 0) {
      s_run = run;
      s_steps = run.t1 - run.t0;
    }
  } else if (w == 0) {  // this block's share of all steps
    const Runs r = first_run(p, CT, SP, lane);
    if (lane == 0) {
      s_run = r;
      s_steps = r.steps(p, CT, SP);
    }
  }
  __syncthreads();
  run = s_run;
  const Runs mine = run;
  const uint32_t n_steps = s_steps;
  uint32_t k = 0;  // steps done
  // Where the block's step i lies, looked up by one thread (all of a window at once).
  auto look_up = [&](uint32_t i) {
    Runs r = mine;
    int pg;
    if (p.cluster) {
      r.t0 += i;
      const int at = r.t0 * SP / kPageTokens;
      if (at < NTHR) {
        pg = pages[at];
        if (pg < 0 || pg >= p.a.n_pages) {
          refuse(p.a.status);
          pg = -1;
        }
      } else {
        pg = page_of(p.a, p.n_ctiles == 1 ? r.e : r.e / p.n_ctiles, r.t0 * SP);
      }
    } else {
      uint32_t before = 0;
      while (i >= before + (r.t1 - r.t0)) {
        before += r.t1 - r.t0;
        if (!r.next(p, CT, SP)) {
          list[i % kWindow] = -1;
          return;
        }
      }
      r.t0 += i - before;
      pg = page_of(p.a, p.n_ctiles == 1 ? r.e : r.e / p.n_ctiles, r.t0 * SP);
    }
    list[i % kWindow] = pg < 0 ? -1 : paged_row(p.a, pg, 0, r.head, r.t0 * SP);
  };
  // Copy step i into its stage, which is free; one thread.
  auto copy_step = [&](uint32_t i) {
    const int st = i % R, row = list[i % kWindow];
    const uint32_t bar = smem_addr(&full[st]), dst = smem_addr(sm + st * 2 * S::HALF);
    issued[st] = row < 0 ? 0 : i + 1;
    if (row < 0) {
      asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
      return;
    }
    expect(bar, 2 * S::HALF);
    tma_rows(dst, &map, row, bar);
    tma_rows(dst + S::HALF, &map, row + p.a.n_kv_heads * kPageTokens, bar);
  };
  for (uint32_t i = tid; i < kWindow && i < n_steps; i += NTHR) {
    look_up(i);
    if (i < R) copy_step(i);
  }
  __syncthreads();
  if (p.cluster > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");

  // a cluster's block has one run
  for (bool more = n_steps > 0; more;) {
    const int seq = p.n_ctiles == 1 ? run.e : run.e / p.n_ctiles, j = run.e - seq * p.n_ctiles;
    int len, nn;
    seq_extent(p.a, seq, len, nn);
    if (!p.cluster) load_q(seq, j, run.head);
    // positions that this lane's columns see (columns nt * 8 + 2 t, + 1), what all columns that see
    // something do and what any does
    int lim[NT][2], all = INT_MAX, any = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int col = j * CT + nt * 8 + 2 * t4 + x, row = row_of(p, col);
        lim[nt][x] = col < p.cols && row < nn ? max(0, len - nn + row + 1) : 0;
        if (lim[nt][x]) all = min(all, lim[nt][x]);
        any = max(any, lim[nt][x]);
      }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      all = min(all, __shfl_xor_sync(0xffffffffu, all, d));
      any = max(any, __shfl_xor_sync(0xffffffffu, any, d));
    }
    // running maximum (log2) and sum of each column, and the weighted sums
    float m[NT][2], l[NT][2], o[NT][DT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = kLow;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < DT; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
    }
    float* sc = pa.scores ? pa.scores + ((size_t)seq * p.a.n_kv_heads + run.head) * p.a.max_pages * kPageTokens * pa.score_cols : nullptr;

    // 16 positions from p0 on, row r0 of the step's tiles at `tile`; CUT: some column does not see all of them
    auto step = [&](uint32_t tile, int r0, int p0, auto cut_) {
      constexpr bool CUT = decltype(cut_)::value;
      float v[NT][4];
      {
        // (two chains of products a column tile: a chain's next waits for its last)
        float a[2][NT][4];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) a[c][nt][0] = a[c][nt][1] = a[c][nt][2] = a[c][nt][3] = 0.f;
        const int r = r0 + (lane & 15);
        const uint32_t at = tile + r * 128;
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          uint32_t x[4];
          ldsm(at + d / 4 * SP * 128 + (((d % 4 * 2 + (lane >> 4)) ^ (r & 7)) << 4), x);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = S::P - 1; i >= 0; --i) mma(a[d & 1][nt], x, qf[i][nt][d]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[nt][e] = a[0][nt][e] + a[1][nt][e];
      }
      if (sc) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            if (nt * 8 + 2 * t4 < pa.score_cols && p0 + g + 8 * r < any)
              *reinterpret_cast<float2*>(sc + (size_t)(p0 + g + 8 * r) * pa.score_cols + nt * 8 + 2 * t4) =
                  make_float2(v[nt][2 * r] * p.c, v[nt][2 * r + 1] * p.c);
      }
      // distance to the running maxima; a maximum that is passed moves.  Element x + 2 r is column 2 t + x, position g + 8 r
      float d[NT][4];
      bool over = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          d[nt][e] = fmaf(v[nt][e], p.c, -m[nt][e & 1]);
          if (CUT && p0 + g + 8 * (e >> 1) >= lim[nt][e & 1]) d[nt][e] = -INFINITY;
          over |= d[nt][e] > kLazy;
        }
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float t = m[nt][x];
#pragma unroll
            for (int r = 0; r < 2; ++r)
              if (d[nt][x + 2 * r] != -INFINITY) t = fmaxf(t, v[nt][x + 2 * r] * p.c);
#pragma unroll
            for (int y = 4; y < 32; y <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, y));
            const float f = exp2_fast(m[nt][x] - t);
            m[nt][x] = t;
            l[nt][x] *= f;
#pragma unroll
            for (int i = 0; i < DT; ++i) {
              o[nt][i][x] *= f;
              o[nt][i][x + 2] *= f;
            }
#pragma unroll
            for (int r = 0; r < 2; ++r)
              if (d[nt][x + 2 * r] != -INFINITY) d[nt][x + 2 * r] = fmaf(v[nt][x + 2 * r], p.c, -t);
          }
      }
      uint2 wf[S::WP][NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = exp2_fast(d[nt][e]);
          l[nt][e & 1] += x[e];
        }
#pragma unroll
        for (int i = 0; i < S::WP; ++i) {
          const uint32_t b0 = pack2(x[0], x[1]), b1 = pack2(x[2], x[3]);
          wf[i][nt] = make_uint2(turn(b0), turn(b1));
          if (i + 1 < S::WP) x[0] -= low_f(b0), x[1] -= high_f(b0), x[2] -= low_f(b1), x[3] -= high_f(b1);
        }
      }
      // V: positions 2 t, 2 t + 1 (words 0, 1) and 8 more (2, 3), dimensions 16 i + g (0, 2) and 8 more (1, 3)
      const int r = r0 + (lane & 7) + (lane >> 4) * 8;
      const uint32_t at = tile + S::HALF + r * 128;
      uint32_t gone[2] = {~0u, ~0u}, mixed[2] = {0u, 0u};  // halves that some column sees; that only some do
      if constexpr (CUT) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int q = p0 + 2 * t4 + 8 * h;
          gone[h] = (q < any ? 0xFFFFu : 0u) | (q + 1 < any ? 0xFFFF0000u : 0u);
          mixed[h] = gone[h] & ((q < all ? 0u : 0xFFFFu) | (q + 1 < all ? 0u : 0xFFFF0000u));
        }
      }
#pragma unroll
      for (int i = 0; i < DT; ++i) {
        uint32_t x[4];
        ldsm_t(at + i / 4 * SP * 128 + (((i % 4 * 2 + ((lane >> 3) & 1)) ^ (r & 7)) << 4), x);
        if constexpr (CUT) {
          uint32_t odd = 0;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            x[y] &= gone[y >> 1];
            odd |= odd_ones(x[y]) & mixed[y >> 1];
          }
          if (__any_sync(0xffffffffu, odd)) {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const uint32_t bad = odd_ones(x[y]) & mixed[y >> 1];
#pragma unroll 1
              for (int tt = 0; tt < 4; ++tt) {
                const uint32_t val = __shfl_sync(0xffffffffu, x[y], (lane & ~3) | tt), is = __shfl_sync(0xffffffffu, bad, (lane & ~3) | tt);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  if (!(is >> (16 * h + 15) & 1u)) continue;
                  const int q = p0 + 2 * tt + h + 8 * (y >> 1);
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                      if (q < lim[nt][c]) o[nt][i][c + 2 * (y & 1)] += h ? high_f(val) : low_f(val);
                }
              }
              x[y] &= ~((bad >> 15 & 1u) * 0xFFFFu | (bad >> 31) * 0xFFFF0000u);
            }
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if constexpr (S::F32) {  // 16 positions' terms by themselves: the products' own sums are cut off, not rounded
            float f[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int y = S::WP - 1; y >= 0; --y) mma(f, x, wf[y][nt]);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][i][e] += f[e];
          } else {
#pragma unroll
            for (int y = S::WP - 1; y >= 0; --y) mma(o[nt][i], x, wf[y][nt]);
          }
        }
      }
    };

#pragma unroll 1
    for (int t = run.t0; t < run.t1; ++t, ++k) {
      if (k % (kWindow / 2) == 0 && k) {  // half of the places are used up: the next ones
        asm volatile("bar.sync 1, %0;" ::"n"(NTHR) : "memory");
        for (uint32_t i = tid; i < kWindow / 2; i += NTHR)
          if (k + kWindow / 2 + i < n_steps) look_up(k + kWindow / 2 + i);
        asm volatile("bar.sync 1, %0;" ::"n"(NTHR) : "memory");
      }
      // the stage of the last step is refilled as soon as all warps have left it
      if (k && k - 1 + R < n_steps && w == (int)(k % W)) {
        const bool free = bar_wait(smem_addr(&empty[(k - 1) % R]), ((k - 1) / R) & 1, &give_up, p.a.status);
        if (free && lane == 0) copy_step(k - 1 + R);
        __syncwarp();
      }
      const int st = k % R;
      const bool fine = bar_wait(smem_addr(&full[st]), (k / R) & 1, &give_up, p.a.status);
      if (fine && issued[st]) {
        const uint32_t tile = smem_addr(sm + st * 2 * S::HALF);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r0 = 16 * (U * w + u), p0 = t * SP + r0;  // this warp's first position
          if (p0 + 16 <= all) step(tile, r0, p0, std::false_type());
          else if (p0 < any) step(tile, r0, p0, std::true_type());
        }
      }
      __syncwarp();
      if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(&empty[st])) : "memory");
    }

    // ---- the run's end: the warps' sums joined
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int col = nt * 8 + 2 * t4 + x;
        if (!lim[nt][x]) m[nt][x] = kLow, l[nt][x] = 0.f;  // padding went through the steps that all others see
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nt][x] += __shfl_xor_sync(0xffffffffu, l[nt][x], d);
        if (g == 0) sm_ml[w][col] = make_float2(m[nt][x], l[nt][x]);
        float* dst = red + (w * CT + col) * S::RS + g;
#pragma unroll
        for (int i = 0; i < DT; ++i) {
          dst[16 * i] = o[nt][i][x];
          dst[16 * i + 8] = o[nt][i][x + 2];
        }
      }
    asm volatile("bar.sync 1, %0;" ::"n"(NTHR) : "memory");
    const bool whole = p.cluster <= 1 && run.t0 == 0 && run.t1 == run.nt;
    const size_t slot = part_slot(blockIdx.x, run.t0);
    const int ncol = min(CT, p.cols - j * CT);
    Odd<HD> odd;
    bool searched = false;
    for (int x = tid; x < ncol * HD / 2; x += NTHR) {  // (a warp's elements are of one column)
      const int c = x / (HD / 2), d = x % (HD / 2) * 2;
      float M = kLow, l_sum = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) M = fmaxf(M, sm_ml[i][c].x);
      float2 v = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float f = exp2_fast(sm_ml[i][c].x - M);
        l_sum += sm_ml[i][c].y * f;
        const float2 y = *reinterpret_cast<const float2*>(red + (i * CT + c) * S::RS + d);
        v.x += y.x * f, v.y += y.y * f;
      }
      if (__any_sync(0xffffffffu, !(is_finite(v.x) && is_finite(v.y)) && is_finite(l_sum))) {
        if (!searched) odd.search(p.a, seq, run.head, run.t0 * SP, min(run.t1 * SP, any));
        searched = true;
        const int sees = len - nn + row_of(p, j * CT + c) + 1;
        const float2 s = make_float2(odd.sum(d, sees), odd.sum(d + 1, sees));
        if (s.x != 0.f) v.x = s.x;
        if (s.y != 0.f) v.y = s.y;
      }
      if (give_up) l_sum = v.x = v.y = NAN;
      if (whole) {
        put_out(seq, j * CT + c, run.head, d, M, l_sum, v);
      } else if (p.cluster) {
        const int rank = blockIdx.x & (p.cluster - 1), slots = (CT + p.cluster - 1) >> p.cluster_log;
        float* to = fin + (rank * slots + (c >> p.cluster_log)) * S::RS;
        put_peer(to + d, c & (p.cluster - 1), v);
        if (d == 0) put_peer(to + HD, c & (p.cluster - 1), make_float2(M, l_sum));
      } else {
        float* dst = p.part + (slot * CT + c) * (HD + 4);
        *reinterpret_cast<float2*>(dst + d) = v;
        if (d == 0) *reinterpret_cast<float2*>(dst + HD) = make_float2(M, l_sum);
      }
    }
    if (!p.cluster && tid == 0 && run.t0 == 0)
      p.item[(size_t)run.e * p.a.n_kv_heads + run.head] =
          make_longlong2(whole ? -1 : run.base + (long long)run.head * (run.nt + kOver), blockIdx.x);
    more = k < n_steps;
    if (more) {
      if (tid == 0) {
        Runs r = run;
        if (!r.next(p, CT, SP)) r.t0 = r.t1 = 0;
        s_run = r;
      }
      asm volatile("bar.sync 1, %0;" ::"n"(NTHR) : "memory");  // the buffers are used again
      run = s_run;
      run.t1 = min(run.t1, run.t0 + (int)(n_steps - k));
      more = run.t1 > run.t0;
    }
  }
  if ((give_up || k < n_steps) && tid == 0) {  // copies in flight land before the block ends
    int none = 0;
    for (int i = 0; i < R; ++i)
      if (issued[i]) bar_wait_long(smem_addr(&full[i]), ((issued[i] - 1) / R) & 1, &none, nullptr);
  }

  // ---- a cluster's item: the blocks have stored their sums with the block that
  // joins the column; it adds them in the blocks' order
  if (p.cluster) {
    const int item = blockIdx.x >> p.cluster_log, rank = blockIdx.x & (p.cluster - 1);
    const int e = item / p.a.n_kv_heads, head = item - e * p.a.n_kv_heads;
    const int seq = p.n_ctiles == 1 ? e : e / p.n_ctiles, j = e - seq * p.n_ctiles, ncol = min(CT, p.cols - j * CT);
    if (p.cluster == 1) {
      if (n_steps == 0)
        for (int x = tid; x < ncol * HD / 2; x += NTHR)
          put_out(seq, j * CT + x / (HD / 2), head, x % (HD / 2) * 2, kLow, 0.f, make_float2(0.f, 0.f));
      return;
    }
    const int slots = (CT + p.cluster - 1) >> p.cluster_log;
    if (n_steps == 0)  // nothing to add: a sum below 0 stands for it
      for (int c = tid; c < ncol; c += NTHR)
        put_peer(fin + (rank * slots + (c >> p.cluster_log)) * S::RS + HD, c & (p.cluster - 1), make_float2(kLow, -1.f));
    cluster_sync();
    for (int x = tid; x < slots * (HD / 2); x += NTHR) {
      const int sl = x / (HD / 2), d = x % (HD / 2) * 2, c = (sl << p.cluster_log) + rank;
      if (c >= ncol) break;  // (a warp's elements are of one column)
      // lane r takes block r's maximum and sum, every lane all blocks' values
      const float* from = fin + sl * S::RS;
      float2 ml = make_float2(kLow, -1.f);
      if ((lane & 15) < p.cluster) ml = *reinterpret_cast<const float2*>(from + (lane & 15) * slots * S::RS + HD);
      float M = ml.x;
#pragma unroll
      for (int o2 = 8; o2 > 0; o2 >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o2));
      const uint32_t some = __ballot_sync(0xffffffffu, !(ml.y < 0.f));  // others have stored no values
      if (ml.y < 0.f) ml.y = 0.f;
      const float f = exp2_fast(ml.x - M);
      float l_sum = ml.y * f;
#pragma unroll
      for (int o2 = 8; o2 > 0; o2 >>= 1) l_sum += __shfl_xor_sync(0xffffffffu, l_sum, o2);
      const uint32_t lost = __ballot_sync(0xffffffffu, f == 0.f) & some;
      float2 y[16], v = make_float2(0.f, 0.f);
#pragma unroll
      for (int r = 0; r < 16; ++r)
        y[r] = some >> r & 1u ? *reinterpret_cast<const float2*>(from + r * slots * S::RS + d) : make_float2(0.f, 0.f);
      if (lost) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float fr = __shfl_sync(0xffffffffu, f, r);
          v.x += taken(y[r].x, fr), v.y += taken(y[r].y, fr);
        }
      } else {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float fr = __shfl_sync(0xffffffffu, f, r);
          v.x += y[r].x * fr, v.y += y[r].y * fr;
        }
      }
      put_out(seq, j * CT + c, head, d, M, l_sum, v);
    }
  }
}

// ---------------------------------------------------------------- host

// A cluster for each item saves the second kernel but leaves SMs idle: it runs for blocks of up to kShort steps, and up to
// twice that where equal runs would save fewer than kJoin steps each (one row of 16 heads on 4 of 128; with the second part and
// without: 40 sequences of 1000 positions 20.0 and 25.4 us, 16 of 4100 26.7 and 30.1, 16 of 100 to 4100 20.7 and 20.1; one of
// 20000, 20 steps a block against 4, 19.6 and 16.9).  Steps are those of the table's width, which the host knows.
constexpr int kShort = 10, kJoin = 8;
// Columns up to which the narrow kernel runs, as far as registers hold the sums and q of a warp's columns (4 heads; one sequence
// of 8022 positions and 64 of 100 to 8022, narrow and wide, us): fp32 16 (128 dimensions 18.9 and 33.0, 127 and 236; 64 dimensions
// 12.8 and 26.3, 75 and 159), bf16 of 64 dimensions 32 (14.2 and 25.7, 81 and 103), of 128 dimensions 16 (13.8 and 27.5, 95 and 117) or 24.
// The third tile of 128 dimensions has one block an SM, so that large batches are faster in the wide kernel unless masses follow, for
// which that forms the scores again (24 columns: one sequence 16.7 and 28.7, 16 of 8022 68.2 and 63.6, 32 of 2049 45.5 and 48.8, 32 of
// 100 to 8022 83 and 67, 64 of these 163 and 118; with masses 32 116 and 121, 64 of 2049 111 and 136).
// steps: of tiles of 128 columns and pages, for an SM.
constexpr long long kBatch = 24;
int narrow_cols(int head_dim, int dtype, bool mass, long long steps) {
  if (dtype == MK_F32) return 16;
  if (head_dim == 64) return 32;
  return mass || steps <= kBatch ? 24 : 16;
}

struct Plan {
  bool wide = false;
  const void* main;
  int id;                                        // of the variant
  int CT, SP, smem, base_smem, blocks, threads;  // columns of a tile, positions of a step; blocks of an SM
  int n_ctiles, n_entries, items, grid, join_cols, join_threads, join_many;
  int cluster;                                   // blocks of an item's cluster; 0: the steps of all items in equal runs
  int score_cols;                                // columns of the scores kept for the masses; 0: none
  size_t item_off, part_off, lse_off, score_off, mass_off, bytes;
};

template <int HD, class T, int NT, int W, int U, int R, int B>
void take(Plan* pl) {
  using S = Shape<HD, T, NT, W, U, R, B>;
  pl->main = reinterpret_cast<const void*>(&k_paged_attention<HD, T, NT, W, U, R, B>);
  pl->id = (HD == 64 ? 0 : 10) + (S::F32 ? 5 : 0) + NT;
  pl->CT = S::CT;
  pl->SP = S::SP;
  pl->smem = pl->base_smem = S::SMEM;
  pl->blocks = B;
  pl->threads = 32 * W;
}

template <int HD>
void take_for(Plan* pl, int cols, int dtype, bool mass, long long steps) {
  if (cols > narrow_cols(HD, dtype, mass, steps)) {
    const WideKernel w = paged_wide_kernel(HD, dtype, cols, steps);
    pl->main = w.fn;
    pl->id = (HD == 64 ? 0 : 10) + (w.CT > 128 ? 8 : dtype == MK_F32 ? 5 : 0);
    pl->CT = w.CT;
    pl->SP = w.SP;
    pl->smem = pl->base_smem = w.smem;
    pl->blocks = w.blocks;
    pl->threads = w.threads;
    pl->wide = true;
    return;
  }
  // Two blocks an SM with two stages each (four of 64 dimensions): one fills the memory system while the other starts or
  // joins its warps (64 sequences of 4096 to 16384 202 us, 16 of 256 to 8448 with masses 38; one block with five stages 208 and 43).
  // Three tiles of 128 dimensions need the shared memory for the sums' join: one block with four stages.
  constexpr int R = HD == 128 ? 2 : 4;
  if (dtype == MK_F32) cols <= 8 ? take<HD, float, 1, 4, 1, R, 2>(pl) : take<HD, float, 2, 4, 1, R, 2>(pl);
  else if (cols <= 16) cols <= 8 ? take<HD, __nv_bfloat16, 1, 4, 1, R, 2>(pl) : take<HD, __nv_bfloat16, 2, 4, 1, R, 2>(pl);
  else if (HD == 128 || cols <= 24) take<HD, __nv_bfloat16, 3, 4, 1, 4, HD == 128 ? 1 : 2>(pl);
  else if constexpr (HD == 64) take<HD, __nv_bfloat16, 4, 4, 1, 4, 2>(pl);
}

// The kernels take more shared memory than the default: asked for once per device.
cudaError_t allow_smem(const Plan& pl) {
  static std::atomic<uint32_t> done[64];  // variants, by device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (done[dev].load() >> pl.id & 1u)) return cudaSuccess;
  // a cluster's blocks take 16 x (columns / 16, rounded up) partial columns more, at most
  e = cudaFuncSetAttribute(pl.main, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           pl.base_smem + (pl.wide ? 0 : (pl.CT + 16) * 130 * 4));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(pl.main, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && dev < 64) done[dev].fetch_or(1u << pl.id);
  return e;
}

// Bytes that a block of a cluster of n takes more, for the partial columns it joins.
int join_room(const Plan& pl, int head_dim, int n) {
  return n > 1 ? n * ((pl.CT + n - 1) / n) * (head_dim + 2) * (int)sizeof(float) : 0;
}

// How many clusters of n blocks run at once, asked for once per variant, size and device.
int clusters_at_once(const Plan& pl, int head_dim, int n) {
  static std::atomic<int> known[64][20][5];  // 1 + the number
  int dev = 0, log = 0, count = 0;
  while (1 << log < n) ++log;
  if (cudaGetDevice(&dev) == cudaSuccess && dev < 64) count = known[dev][pl.id][log].load();
  if (count) return count - 1;
  count = pl.blocks * device_sms() / n;
  cudaError_t e = allow_smem(pl);
  if (e == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = n;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(n);
    cfg.blockDim = dim3(pl.threads);
    cfg.dynamicSmemBytes = pl.base_smem + join_room(pl, head_dim, n);
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int c = 0;
    e = cudaOccupancyMaxActiveClusters(&c, pl.main, &cfg);
    if (e == cudaSuccess) {
      count = c;
      if (dev < 64) known[dev][pl.id][log].store(count + 1);
    }
  }
  if (e != cudaSuccess) cudaGetLastError();  // this query's own, no one else's
  return count;
}

size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

// Variant, grid and workspace of a call with rows; false: too many columns.
bool plan_of(const Kv4Args& c, int head_dim, int n_heads, int dtype, bool mass, Plan* pl) {
  const long long cols = (long long)c.rows * (n_heads / c.n_kv_heads);
  if (cols > INT_MAX / 64) return false;
  const int sms = device_sms();
  const long long steps = (cols + 127) / 128 * c.n_seqs * c.n_kv_heads * c.max_pages / sms;
  if (head_dim == 64) take_for<64>(pl, (int)cols, dtype, mass, steps);
  else take_for<128>(pl, (int)cols, dtype, mass, steps);
  const long long ct = (cols + pl->CT - 1) / pl->CT, entries = ct * c.n_seqs, items = entries * c.n_kv_heads;
  const long long most = (long long)c.max_pages * (kPageTokens / pl->SP);  // steps of an item
  if (items > INT_MAX / 32 || (most + kOver) * c.n_kv_heads > INT_MAX) return false;
  pl->n_ctiles = (int)ct;
  pl->n_entries = (int)entries;
  pl->items = (int)items;
  const long long room = std::min(pl->blocks * sms, kMaxBlocks);  // blocks that run at once
  pl->cluster = 0;
  pl->item_off = pl->part_off = pl->bytes = 0;
  int n = 1;
  while (n < 16 && 2 * n <= most && items <= clusters_at_once(*pl, head_dim, 2 * n)) n *= 2;
  const long long each = (most + n - 1) / n;  // steps of a cluster's block
  if (!pl->wide && (each <= kShort || (each <= 2 * kShort && each <= items * most / room + kJoin))) {
    pl->cluster = n;
    pl->smem += join_room(*pl, head_dim, n);
    pl->grid = (int)(items * n);
  } else {
    pl->grid = (int)std::min<long long>(room, items * most);
    const long long all_cols = items * std::min<long long>(cols, pl->CT);
    pl->join_cols = all_cols <= 10 * sms ? 1 : 8;
    int nw = 2;
    while (nw < 16 && nw * 2 * items <= pl->grid) nw *= 2;
    pl->join_many = pl->grid / 64 >= items && all_cols <= sms;  // 64 parts an item and more, a block an SM at most
    pl->join_threads = 32 * (pl->join_cols > 1 ? 8 : nw);
    pl->item_off = 16;
    pl->part_off = pl->item_off + (size_t)items * sizeof(longlong2);
    pl->bytes = pl->part_off + 2 * (size_t)pl->grid * pl->CT * (head_dim + 4) * sizeof(float);
  }
  pl->score_cols = 0;
  if (mass) {
    if (!paged_mass_fits(c, n_heads, dtype, pl->wide)) return false;
    pl->lse_off = up16(pl->bytes);
    pl->bytes = pl->lse_off + (size_t)c.n_seqs * c.rows * n_heads * sizeof(float);
    if (!pl->wide) {
      pl->score_cols = (int)(cols + 3) & ~3;
      pl->score_off = up16(pl->bytes);
      pl->bytes = pl->score_off + (size_t)c.n_seqs * c.n_kv_heads * c.max_pages * kPageTokens * pl->score_cols * sizeof(float);
    } else {
      pl->mass_off = (pl->bytes + 127) & ~(size_t)127;
      pl->bytes = pl->mass_off + paged_mass_bytes(c, head_dim, n_heads, dtype);
    }
  }
  return true;
}

}  // namespace

int device_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 152;
  }
  return n;
}

// The driver's encoder, looked up once.
int rows_map(CUtensorMap* map, const void* base, long long rows, int head_dim, int box_rows) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static std::atomic<void*> known{nullptr};
  void* f = known.load();
  if (!f) {
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !f) {
      cudaGetLastError();
      return host_fail(MK_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    }
    known.store(f);
  }
  const cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)head_dim / 64}, strides[2] = {(cuuint64_t)head_dim * 2, 128};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)head_dim / 64}, one[3] = {1, 1, 1};
  const CUresult r = reinterpret_cast<Encode>(f)(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, one,
                                                 CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MK_OK : host_fail(MK_ERR_CUDA, "no tensor map of these rows");
}

static int run_attention(const Kv4Args& a, int head_dim, int n_heads, const Kv4Rows& q, int dtype, float scale, const Kv4Rows& out,
                         float* lse, const PagedMass* mass, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  Plan pl;
  if (!plan_of(a, head_dim, n_heads, dtype, mass != nullptr, &pl))
    return host_fail(MK_ERR_INVALID_ARG, "n_seqs x rows x n_heads or max_pages x n_kv_heads is too large");
  if (pl.bytes && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u) || workspace_bytes < pl.bytes))
    return host_fail(MK_ERR_INVALID_ARG, "workspace is NULL, not 16-byte aligned or smaller than mk_paged_attention_bytes");
  CUtensorMap map;
  if (int r = rows_map(&map, a.pool, (long long)a.n_pages * 2 * a.n_kv_heads * kPageTokens, head_dim, pl.SP)) return r;
  char* ws = static_cast<char*>(workspace);
  PagedAtt pa;
  AttArgs& p = pa.t;
  p.a = a;
  p.q = q;
  p.out = out;
  p.lse = mass && !lse ? reinterpret_cast<float*>(ws + pl.lse_off) : lse;
  p.c = (float)((double)scale * 1.4426950408889634);
  p.n_heads = n_heads;
  p.gqa = n_heads / a.n_kv_heads;
  p.cols = a.rows * p.gqa;
  p.n_ctiles = pl.n_ctiles;
  p.n_entries = pl.n_entries;
  p.cluster = pl.cluster;
  p.cluster_log = p.gqa_log = -1;
  for (int i = 0; i < 13; ++i) {
    if (pl.cluster == 1 << i) p.cluster_log = i;
    if (p.gqa == 1 << i) p.gqa_log = i;
  }
  p.total = nullptr;
  p.item = nullptr;
  p.part = nullptr;
  if (!pl.cluster) {
    p.total = reinterpret_cast<long long*>(ws);
    p.item = reinterpret_cast<longlong2*>(ws + pl.item_off);
    p.part = reinterpret_cast<float*>(ws + pl.part_off);
  }
  pa.score_cols = pl.score_cols;
  pa.scores = pl.score_cols ? reinterpret_cast<float*>(ws + pl.score_off) : nullptr;
  pa.mass_ws = mass && !pl.score_cols ? ws + pl.mass_off : nullptr;
  cudaError_t e = allow_smem(pl);
  if (e == cudaSuccess && pa.mass_ws) e = paged_mass_begin(pa, head_dim, dtype, stream);
  void* args[] = {&pa, &map};
  if (e == cudaSuccess) e = launch(pl.main, pl.grid, pl.threads, pl.smem, stream, args, pl.cluster);
  if (e == cudaSuccess && !pl.cluster) {
    void* jargs[] = {&p, &pl.CT, &pl.SP, &pl.grid, &pl.join_cols};
    if (pl.wide) e = launch(paged_wide_join(head_dim, dtype), pl.items, 256, 0, stream, jargs, 0, pl.CT / 16);
    else e = launch(kv4_join_kernel(head_dim, dtype, pl.join_many), pl.items, pl.join_threads, 0, stream, jargs, 0,
               (pl.CT + pl.join_cols - 1) / pl.join_cols);
  }
  if (e == cudaSuccess && mass) e = paged_mass(pa, *mass, head_dim, dtype, map, stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return host_fail(MK_ERR_CUDA, (std::string("paged attention: ") + cudaGetErrorString(e)).c_str());
  }
  return MK_OK;
}

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
  Plan pl;
  return plan_of(kv4_args(*c), c->head_dim, n_heads, dtype, with_mass != 0, &pl) ? pl.bytes : 0;
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
  PagedMass m;
  if (mass) {
    if (int r = paged_check_mass(mass, c, "mass")) return r;
    m = {mass->data, mass->seq_stride, mass->head_stride, mass->decay};
  }
  return run_attention(kv4_args(*c), c->head_dim, n_heads, kv4_rows(*q), dtype, scale, kv4_rows(*out), lse, mass ? &m : nullptr,
                       workspace, workspace_bytes, (cudaStream_t)stream);
}
