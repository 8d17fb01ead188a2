// Causal attention over the 4-bit paged K/V cache (mk_kv4_attention): single
// rows of a decode step, drafted rows and prompt chunks.
//
// Mathematics.  For a row q and the positions p it sees, s_p = c q . K_p,
// out = sum_p e^(s_p - m) V_p / sum_p e^(s_p - m).  K_p = ks (codes), one scale
// per group of 64 dimensions, so q . K_p = sum_groups ks_g (q_g . code_g): the
// products run on the codes and the scale multiplies their fp32 sum.  V's scale
// multiplies the weight instead (one weight per group), so neither K nor V is
// ever formed: tensor cores (mma.sync m16n8k16) take the codes as they are.
//
// A code becomes an operand without arithmetic.  The nibble of a byte, moved to
// bits 15 (sign) and 6..4 (magnitude) of a half word, is the subnormal
// +-m 2^-129 of bf16 and +-m 2^-20 of fp16, exactly.  One byte permutation
// doubles two bytes into the halves of a word (two positions for V, two
// dimensions for K), one mask takes the high nibbles and one shift and mask the
// low ones: 1 instruction a value (the magic-number form takes 1.5).
//   q . code runs in bf16: q carries 2^64, so that the products (2^-65) stay far
// from fp32's ends whatever q's size.  A bf16 q is exact; an fp32 q is split into
// three bf16 parts (24 bits).
//   weight x V code runs in fp16: the weight (at most 2^8, see below) times V's
// scale is normalised by a power of two that follows the largest scale the warp
// has met, to at most 2^14; fp16 then keeps 11 bits over 28 binades below it and
// the weight is rounded by 2^-11 at most, where the output is rounded by 2^-8.  For
// fp32 rows it is split into two parts (22 bits).
// Everything else is fp32.
//
// Layout.  K is the mma's A operand (16 positions x 16 dimensions) and q its B
// operand, so that the query columns of one kv head (rows x heads of the group)
// fill tiles of 8 columns and the 4 heads of a single row cost one.  The weights
// come out transposed for the second product (V^T x weights^T) and turn with
// movmatrix.
//
// Work.  The tiles of all (sequence, column tile, kv head) items are laid end
// to end and cut into equal runs, one for each block, from the lengths on the
// device: a ragged batch costs what its sum costs, and a captured graph follows
// the lengths.  A block's steps of 64 or 128 positions stream (one bulk copy of 8.7 or
// 17.4 KB each at 128 dimensions) through a shared-memory ring, refilled by its warps
// in turn; each warp takes 16 or 32 positions of a step, with running maxima of its own
// (moved only when a score passes them by 2^8) and one merge at the end of an item.
// An item cut between blocks is joined by a second kernel, launched so that its
// start overlaps the first one's end.  Short work instead makes each item a cluster
// of blocks that join through their shared memory, in one kernel.  Calls of many
// columns run in mk_kv4_wide.cu.
//
// Measured (16 heads on 4 kv heads of 128, bf16 rows).  Short work is bound by its
// chain of set-up, first copies and join: one sequence of 2049 positions 7.0 us, with 6% of
// the issue slots busy; 16 of 256 to 8448 15.8 us (38 MB).  Long work is bound by issue
// and the unpacking: 64 of 4096 to 16384 76.9 us, 4.6 TB/s, the ALU 53% and the issue slots 55%
// busy, with 14 warps of 118 registers on an SM; one of 131071 23.6 us, 3.0 TB/s.  24 columns
// hold their sums in 243 registers, which leaves 8 warps an SM (issue slots 30% busy): 16 sequences of
// up to 8022 positions with up to 5 rows each 31.2 us.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <climits>
#include <string>
#include <type_traits>

#include "mk_kv4_att.cuh"

namespace mk {
namespace {

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint2 b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint2 b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
}
// The first product of a chain: d = a b.
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint2 b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y), "f"(0.f));
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
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
constexpr int kWindow = 128;  // steps whose addresses a block looks up at a time
// NT column tiles; W warps of U units of 16 positions in each step; R steps in
// the ring; B blocks of an SM.
template <int HD, class T, int NT, int W, int U, int R, int B>
struct Shape {
  static constexpr bool F32 = std::is_same<T, float>::value;
  static constexpr int CT = 8 * NT;              // columns of a tile
  static constexpr int NG = HD / kGroup;
  static constexpr int QP = F32 ? 3 : 1;         // parts of q
  static constexpr int WP = F32 ? 2 : 1;         // parts of the weights
  static constexpr bool QS = NT > 2;             // q's fragments in shared memory, to leave registers to the sums
  static constexpr int RS = HD + 2;              // floats of a column in the reduction buffer
  static constexpr int SP = 16 * W * U;          // positions of a step: 64 or 128, within a page
  static constexpr int BYTES = SP / kTile * Tile<HD>::BYTES;
  static constexpr int RED = W * CT * RS * 4;
  static constexpr int QB = QS ? NT * NG * 4 * 32 * 8 : 0;
  static constexpr int SMEM = R * BYTES + RED + QB;
};

template <int HD, class T, int NT, int W, int U, int R, int B>
__global__ void __launch_bounds__(32 * W, B) k_kv4_attention(const __grid_constant__ AttArgs p) {
  using S = Shape<HD, T, NT, W, U, R, B>;
  using L = Tile<HD>;
  constexpr int NG = S::NG, CT = S::CT, SP = S::SP, NTHR = 32 * W;
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ __align__(8) uint64_t full[R], empty[R];
  __shared__ unsigned long long list[kWindow];  // where the block's next steps lie (0: a page outside the pool)
  __shared__ uint32_t issued[R];              // 1 + the last step copied into each stage
  __shared__ float2 sm_ml[W][CT];  // a run's maximum and sum of each warp and column
  // The block's run and its number of steps, found by one thread: all warps pass the
  // same barriers even where someone writes the lengths while the call runs.
  __shared__ Runs s_run;
  __shared__ uint32_t s_steps;
  __shared__ volatile int give_up;
  // cluster: the partial results of the columns that this block joins, column c
  // (joined by block c mod cluster) of block r in [r][c / cluster][HD | M, sum]
  float* fin = reinterpret_cast<float*>(sm + S::SMEM);
  // cluster: the first pages of the item's sequence, where the sums are joined at the end
  int* pages = reinterpret_cast<int*>(sm + R * S::BYTES);
  static_assert(S::RED >= NTHR * (int)sizeof(int), "room for the pages");
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
  // lane (g, t) of the mma fragments
  const int g = lane >> 2, t4 = lane & 3;
  // the B fragments of q: column nt * 8 + g, dimensions 64 h + 16 t + 8 i + 4 jj + {0, 2 | 1, 3}
  uint2 qf[S::QS ? 1 : S::QP][S::QS ? 1 : NT][NG][2][2];
  uint2* qsm = reinterpret_cast<uint2*>(sm + R * S::BYTES + S::RED);  // [nt][h][i][lane][jj]
  auto load_q = [&](int seq, int j, int head) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (S::QS && nt % W != w) continue;
      const int col = j * CT + nt * 8 + g;
      const bool there = col < p.cols;
      const int row = there ? row_of(p, col) : 0, hd = there ? col - row * p.gqa : 0;
      const T* src = reinterpret_cast<const T*>(p.q.p) + seq * p.q.seq + row * p.q.row +
                     (head * p.gqa + hd) * p.q.head + 16 * t4;
#pragma unroll
      for (int h = 0; h < NG; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int jj = 0; jj < 2; ++jj) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (there) {
              if constexpr (S::F32) x = *reinterpret_cast<const float4*>(src + 64 * h + 8 * i + 4 * jj);
              else {
                const uint2 v = *reinterpret_cast<const uint2*>(src + 64 * h + 8 * i + 4 * jj);
                x = make_float4(low_f(v.x), high_f(v.x), low_f(v.y), high_f(v.y));
              }
            }
            x.x *= kUp, x.y *= kUp, x.z *= kUp, x.w *= kUp;
            if constexpr (S::QS) {
              qsm[(((nt * NG + h) * 2 + i) * 32 + lane) * 2 + jj] = make_uint2(pack2(x.x, x.z), pack2(x.y, x.w));
            } else {
#pragma unroll
              for (int q = 0; q < S::QP; ++q) {
                const uint2 b = make_uint2(pack2(x.x, x.z), pack2(x.y, x.w));
                qf[q][nt][h][i][jj] = b;
                if (q + 1 < S::QP) x.x -= low_f(b.x), x.z -= high_f(b.x), x.y -= low_f(b.y), x.w -= high_f(b.y);
              }
            }
          }
    }
    if constexpr (S::QS) asm volatile("bar.sync 1, %0;" ::"n"(NTHR) : "memory");
  };
  // Dimensions d, d + 1 of a column's result from its sums.
  auto put_out = [&](int seq, int col, int head, int d, float M, float l_sum, float2 v) {
    const int row = row_of(p, col), hd = head * p.gqa + col - row * p.gqa;
    const float f = l_sum == 0.f ? 0.f : 1.f / l_sum;
    T* dst = reinterpret_cast<T*>(const_cast<void*>(p.out.p)) + seq * p.out.seq + row * p.out.row + hd * p.out.head + d;
    if constexpr (S::F32) *reinterpret_cast<float2*>(dst) = make_float2(v.x * f, v.y * f);
    else *reinterpret_cast<uint32_t*>(dst) = pack2(v.x * f, v.y * f);
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
  } else if (w == 0) {  // this block's share of all tiles
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
  // Address of the block's step i, looked up by one thread (all of a window at once).
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
          list[i % kWindow] = 0;
          return;
        }
      }
      r.t0 += i - before;
      pg = page_of(p.a, p.n_ctiles == 1 ? r.e : r.e / p.n_ctiles, r.t0 * SP);
    }
    list[i % kWindow] = pg < 0 ? 0 : (unsigned long long)tile_of<HD>(p.a, pg, r.head, r.t0 * SP);
  };
  // Copy step i into its stage, which is free; one thread.
  auto copy_step = [&](uint32_t i) {
    const int st = i % R;
    const uint32_t bar = smem_addr(&full[st]);
    const unsigned long long src = list[i % kWindow];
    issued[st] = src ? i + 1 : 0;
    if (src) {
      asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "n"(S::BYTES) : "memory");
      asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                       smem_addr(sm + st * S::BYTES)),
                   "l"(src), "n"(S::BYTES), "r"(bar)
                   : "memory");
    }
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
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
    // positions that this lane's columns see (columns nt * 8 + 2 t, + 1), what
    // all columns see and what any does
    int lim[NT][2], all = INT_MAX, any = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int col = j * CT + nt * 8 + 2 * t4 + x, row = row_of(p, col);
        lim[nt][x] = col < p.cols && row < nn ? max(0, len - nn + row + 1) : 0;
        if (col < p.cols) all = min(all, lim[nt][x]);
        any = max(any, lim[nt][x]);
      }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      all = min(all, __shfl_xor_sync(0xffffffffu, all, d));
      any = max(any, __shfl_xor_sync(0xffffffffu, any, d));
    }
    // running maximum (log2) and sum of each column, the weighted sums, and the
    // normalisation of V's scales: they are below cap, and enter times vmul = 2^6 / cap
    float m[NT][2], l[NT][2], o[NT][NG][4][4], cap = 0.f, vmul = 1.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = kLow;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int h = 0; h < NG; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nt][h][i][0] = o[nt][h][i][1] = o[nt][h][i][2] = o[nt][h][i][3] = 0.f;
    }

    // U x 16 positions from p0 on, rows r0.. of a tile (`tile`: the K codes of
    // row r0); CUT: some column does not see all of them
    auto step = [&](uint32_t tile, int r0, int p0, auto cut_) {
      constexpr bool CUT = decltype(cut_)::value;
      constexpr int HG = NT > 2 ? 1 : NG;  // groups of dimensions in flight
      const uint32_t kr = tile + g * L::ROW + 8 * t4;
      // scales of positions g and g + 8
      float ks[U][2][NG], vs[U][2][NG];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t at = tile + L::CODES + (16 * u + g + 8 * r) * NG * 2 - r0 * (L::ROW - NG * 2);
          const uint32_t x = NG == 2 ? lds32(at) : lds16(at);
          uint32_t y = NG == 2 ? lds32(at + L::V) : lds16(at + L::V);
          if (CUT && p0 + 16 * u + g + 8 * r >= any) y = 0;  // a slot behind the end may hold anything
          ks[u][r][0] = low_f(x);
          vs[u][r][0] = low_f(y);
          if constexpr (NG == 2) {
            ks[u][r][1] = high_f(x);
            vs[u][r][1] = high_f(y);
          }
        }
      // scores without the factor c: element x + 2 r is column 2 t + x, position g + 8 r
      float v[U][NT][4];
#pragma unroll
      for (int hb = 0; hb < NG; hb += HG) {
        float a[U][HG][NT][4];
        uint2 kw[U][HG][2];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int h = 0; h < HG; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r) kw[u][h][r] = lds64(kr + (16 * u + 8 * r) * L::ROW + 32 * (hb + h));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint2 qs[HG][NT][2];
          if constexpr (S::QS) {
#pragma unroll
            for (int h = 0; h < HG; ++h)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const uint4 b = *reinterpret_cast<const uint4*>(qsm + (((nt * NG + hb + h) * 2 + i) * 32 + lane) * 2);
                qs[h][nt][0] = make_uint2(b.x, b.y);
                qs[h][nt][1] = make_uint2(b.z, b.w);
              }
          }
#pragma unroll
          for (int jj = 0; jj < 2; ++jj)
#pragma unroll
            for (int h = 0; h < HG; ++h)
#pragma unroll
              for (int u = 0; u < U; ++u) {
                const uint2 u0 = kw[u][h][0], u1 = kw[u][h][1];
                const uint32_t x0 = __byte_perm(i ? u0.y : u0.x, 0, jj ? 0x3322 : 0x1100);
                const uint32_t x1 = __byte_perm(i ? u1.y : u1.x, 0, jj ? 0x3322 : 0x1100);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  if constexpr (S::QS) {
                    if (i == 0 && jj == 0)
                      mma_bf16_first(a[u][h][nt], (x0 << 4) & kNib, (x1 << 4) & kNib, x0 & kNib, x1 & kNib, qs[h][nt][jj]);
                    else
                      mma_bf16(a[u][h][nt], (x0 << 4) & kNib, (x1 << 4) & kNib, x0 & kNib, x1 & kNib, qs[h][nt][jj]);
                  } else {
#pragma unroll
                    for (int q = S::QP - 1; q >= 0; --q)
                      if (i == 0 && jj == 0 && q == S::QP - 1)
                        mma_bf16_first(a[u][h][nt], (x0 << 4) & kNib, (x1 << 4) & kNib, x0 & kNib, x1 & kNib,
                                       qf[q][nt][hb + h][i][jj]);
                      else
                        mma_bf16(a[u][h][nt], (x0 << 4) & kNib, (x1 << 4) & kNib, x0 & kNib, x1 & kNib,
                                 qf[q][nt][hb + h][i][jj]);
                  }
                }
              }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int h = 0; h < HG; ++h)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                v[u][nt][e] = hb + h ? fmaf(a[u][h][nt][e], ks[u][e >> 1][hb + h], v[u][nt][e])
                                     : a[u][h][nt][e] * ks[u][e >> 1][0];
      }
      // distance to the running maxima; a maximum or the cap that is passed moves
      float d[U][NT][4];
      bool over = false;
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            d[u][nt][e] = fmaf(v[u][nt][e], p.c, -m[nt][e & 1]);
            if (CUT && p0 + 16 * u + g + 8 * (e >> 1) >= lim[nt][e & 1]) d[u][nt][e] = -INFINITY;
            over |= d[u][nt][e] > kLazy;
          }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int h = 0; h < NG; ++h) over |= vs[u][r][h] > cap;
      }
      if (__any_sync(0xffffffffu, over)) {
        float top = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int h = 0; h < NG; ++h) top = fmaxf(top, vs[u][r][h]);
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        float move = 1.f;
        const int old = (int)(__float_as_uint(cap) >> 23);  // the cap's exponent, 0: none yet
        if (top > cap) {  // the next power of two, and 2^3 of room
          const int e = min(max((int)(__float_as_uint(top) >> 23) + 4, 8), 254);
          const float mul = __uint_as_float((uint32_t)(260 - e) << 23);
          move = mul / vmul;
          cap = __uint_as_float((uint32_t)e << 23);
          vmul = mul;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float t = m[nt][x];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int r = 0; r < 2; ++r)
                if (d[u][nt][x + 2 * r] != -INFINITY) t = fmaxf(t, v[u][nt][x + 2 * r] * p.c);
#pragma unroll
            for (int y = 4; y < 32; y <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, y));
            const float f = exp2_fast(m[nt][x] - t);
            m[nt][x] = t;
            l[nt][x] *= f;
            const float fo = f * move;
#pragma unroll
            for (int h = 0; h < NG; ++h)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                o[nt][h][i][x] *= fo;
                o[nt][h][i][x + 2] *= fo;
              }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int r = 0; r < 2; ++r)
                if (d[u][nt][x + 2 * r] != -INFINITY) d[u][nt][x + 2 * r] = fmaf(v[u][nt][x + 2 * r], p.c, -t);
          }
        const int now = (int)(__float_as_uint(cap) >> 23);
        if constexpr (CUT) {
          // A column that sees the last of its positions here must not pay for a cap that
          // moved for one it does not see (its terms would fall below fp16's range): its
          // maximum goes down by what the cap went up beyond its own, its weights and sums up.
          if (now != old && any != all) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                float seen = 0.f;
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                  for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int h = 0; h < NG; ++h)
                      if (p0 + 16 * u + g + 8 * r < lim[nt][x]) seen = fmaxf(seen, vs[u][r][h]);
#pragma unroll
                for (int y = 4; y < 32; y <<= 1) seen = fmaxf(seen, __shfl_xor_sync(0xffffffffu, seen, y));
                const int own = max(old, seen > 0.f ? min(max((int)(__float_as_uint(seen) >> 23) + 4, 8), 254) : 0);
                const int up = own && lim[nt][x] < p0 + 16 * U ? min(now - own, 90) : 0;
                const float f = __uint_as_float((uint32_t)(127 + up) << 23);
                m[nt][x] -= (float)up;
                l[nt][x] *= f;
#pragma unroll
                for (int h = 0; h < NG; ++h)
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    o[nt][h][i][x] *= f;
                    o[nt][h][i][x + 2] *= f;
                  }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                  for (int r = 0; r < 2; ++r)
                    if (d[u][nt][x + 2 * r] != -INFINITY) d[u][nt][x + 2 * r] = fmaf(v[u][nt][x + 2 * r], p.c, -m[nt][x]);
              }
          }
        }
      }
      // weights times V's scales, as B fragments
      uint2 wf[U][S::WP][NT][NG];
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int h = 0; h < NG; ++h) vs[u][r][h] *= vmul;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            d[u][nt][e] = exp2_fast(d[u][nt][e]);
            l[nt][e & 1] += d[u][nt][e];
          }
#pragma unroll
          for (int h = 0; h < NG; ++h) {
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[e] = d[u][nt][e] * vs[u][e >> 1][h];
              if (CUT && p0 + 16 * u + g + 8 * (e >> 1) >= lim[nt][e & 1]) x[e] = 0.f;  // whatever the scale there
            }
#pragma unroll
            for (int q = 0; q < S::WP; ++q) {
              const uint32_t b0 = pack2h(x[0], x[1]), b1 = pack2h(x[2], x[3]);
              wf[u][q][nt][h] = make_uint2(turn(b0), turn(b1));
              if (q + 1 < S::WP) x[0] -= low_h(b0), x[1] -= high_h(b0), x[2] -= low_h(b1), x[3] -= high_h(b1);
            }
          }
        }
      }
      // V: positions 2 t, 2 t + 1 and 2 t + 8, 2 t + 9, dimensions 64 h + 8 g + {0..7}
      const uint32_t vr = tile + L::V + 2 * t4 * L::ROW + 4 * g;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int h = 0; h < NG; ++h) {
          const uint32_t at = vr + 16 * u * L::ROW + 32 * h;
          const uint32_t v0 = lds32(at), v1 = lds32(at + L::ROW), v8 = lds32(at + 8 * L::ROW), v9 = lds32(at + 9 * L::ROW);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t sel = 0x4400u + 0x1111u * i;
            const uint32_t x = __byte_perm(v0, v1, sel), y = __byte_perm(v8, v9, sel);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if constexpr (S::F32) {  // a unit's terms are summed on their own, then added
                float f[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int q = S::WP - 1; q >= 0; --q)
                  mma_f16(f, (x << 4) & kNib, x & kNib, (y << 4) & kNib, y & kNib, wf[u][q][nt][h]);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nt][h][i][e] += f[e];
              } else {
                mma_f16(o[nt][h][i], (x << 4) & kNib, x & kNib, (y << 4) & kNib, y & kNib, wf[u][0][nt][h]);
              }
            }
          }
        }
    };

#pragma unroll 1
    for (int t = run.t0; t < run.t1; ++t, ++k) {
      if (k % (kWindow / 2) == 0 && k) {  // half of the addresses are used up: the next ones
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
        // this warp's first position, its tile and row
        const int at = 16 * U * w, p0 = t * SP + at, r0 = at % kTile;
        const uint32_t tile = smem_addr(sm + st * S::BYTES) + at / kTile * L::BYTES + r0 * L::ROW;
        if (p0 + 16 * U <= all) step(tile, r0, p0, std::false_type());
        else if (p0 < any) step(tile, r0, p0, std::true_type());
      }
      __syncwarp();
      if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(&empty[st])) : "memory");
    }

    // ---- the run's end: the warps' sums joined
    float* red = reinterpret_cast<float*>(sm + R * S::BYTES);
    const float undo = kCode / vmul;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int col = nt * 8 + 2 * t4 + x;
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nt][x] += __shfl_xor_sync(0xffffffffu, l[nt][x], d);
        if (g == 0) sm_ml[w][col] = make_float2(m[nt][x], l[nt][x]);
        float* dst = red + (w * CT + col) * S::RS + 8 * g;
#pragma unroll
        for (int h = 0; h < NG; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float2*>(dst + 64 * h + 2 * i) = make_float2(o[nt][h][i][x] * undo, o[nt][h][i][x + 2] * undo);
      }
    asm volatile("bar.sync 1, %0;" ::"n"(NTHR) : "memory");
    const bool whole = p.cluster <= 1 && run.t0 == 0 && run.t1 == run.nt;
    const size_t slot = part_slot(blockIdx.x, run.t0);
    const int ncol = min(CT, p.cols - j * CT);
    for (int x = tid; x < ncol * HD / 2; x += NTHR) {
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
    if (n_steps == 0)  // nothing to add: a sum of 0 stands for it
      for (int c = tid; c < ncol; c += NTHR)
        put_peer(fin + (rank * slots + (c >> p.cluster_log)) * S::RS + HD, c & (p.cluster - 1), make_float2(kLow, 0.f));
    cluster_sync();
    for (int x = tid; x < slots * (HD / 2); x += NTHR) {
      const int sl = x / (HD / 2), d = x % (HD / 2) * 2, c = (sl << p.cluster_log) + rank;
      if (c >= ncol) break;  // (a warp's elements are of one column)
      // lane r takes block r's maximum and sum, every lane all blocks' values
      const float* from = fin + sl * S::RS;
      float2 ml = make_float2(kLow, 0.f);
      if ((lane & 15) < p.cluster) ml = *reinterpret_cast<const float2*>(from + (lane & 15) * slots * S::RS + HD);
      float M = ml.x;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      const uint32_t some = __ballot_sync(0xffffffffu, ml.x != kLow || ml.y != 0.f);  // others have stored no values
      const float f = exp2_fast(ml.x - M);
      float l_sum = ml.y * f;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) l_sum += __shfl_xor_sync(0xffffffffu, l_sum, o);
      float2 y[16], v = make_float2(0.f, 0.f);
#pragma unroll
      for (int r = 0; r < 16; ++r)
        y[r] = some >> r & 1u ? *reinterpret_cast<const float2*>(from + r * slots * S::RS + d) : make_float2(0.f, 0.f);
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float fr = __shfl_sync(0xffffffffu, f, r);
        if (some >> r & 1u) v.x += y[r].x * fr, v.y += y[r].y * fr;
      }
      put_out(seq, j * CT + c, head, d, M, l_sum, v);
    }
  }
}

// Items cut between blocks: a block joins the partial results of CC columns of
// an item, in the blocks' order.  First the places of the item's parts, once for
// all of its columns.  Of several columns each is a warp's work (1024 rows at 8022 positions,
// 16384 columns of about 3 parts: a block for every column with the places found by every
// warp took 33 us); a single column is all warps', every NW-th part each, the warps at the
// end.  Items without a tile (nothing seen) get zeros here.
// NB: parts in flight in each warp.
template <int HD, class T, int NB>
__global__ void __launch_bounds__(512) k_kv4_join(const __grid_constant__ AttArgs p, int CT, int SP, int G, int CC) {
  constexpr int V = HD / 32;  // dimensions of a lane
  __shared__ float red[16][HD], red_m[16], red_l[16];
  __shared__ int slot[kMaxBlocks], n_parts;  // -1: a block without steps of this item
  const int e = blockIdx.x / p.a.n_kv_heads, head = blockIdx.x - e * p.a.n_kv_heads;
  const int seq = e / p.n_ctiles, j = e - seq * p.n_ctiles;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, NW = blockDim.x >> 5;
  const int c0 = blockIdx.y * CC, c1 = min(min(c0 + CC, CT), p.cols - j * CT);
  if (c0 >= c1) return;
  const int nt = tiles_of(p, e, CT, SP);
  if (threadIdx.x == 0) n_parts = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();
  if (nt) {
    const longlong2 it = p.item[blockIdx.x];
    const long long total = *p.total;
    if (it.x < 0 || it.y < 0 || it.y >= G) return;  // done by its block
    for (int i = threadIdx.x; it.y + i < G; i += blockDim.x) {
      const long long lo = first_place(total, it.y + i, G) - it.x - kOver;
      if (lo >= nt) break;
      const long long hi = first_place(total, it.y + i + 1, G) - it.x - kOver;
      slot[i] = hi <= 0 || hi <= lo ? -1 : part_slot(it.y + i, lo > 0);
      atomicMax(&n_parts, i + 1);
    }
    __syncthreads();
  }
  const int n = n_parts;
  float m, l, o[V];
  // parts first, first + by .. of column c, NB at a time
  auto gather = [&](int c, int first, int by) {
    m = kLow, l = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = 0.f;
#pragma unroll 1
    for (int i0 = first; i0 < n; i0 += NB * by) {
      float2 ml[NB];
      float v[NB][V];
      uint32_t there = 0;
#pragma unroll
      for (int y = 0; y < NB; ++y) {
        const int i = i0 + y * by, at = i < n ? slot[i] : -1;
        ml[y] = make_float2(kLow, 0.f);
#pragma unroll
        for (int x = 0; x < V; ++x) v[y][x] = 0.f;
        if (at >= 0) {
          there |= 1u << y;
          const float* src = p.part + ((size_t)at * CT + c) * (HD + 4);
          ml[y] = *reinterpret_cast<const float2*>(src + HD);
#pragma unroll
          for (int x = 0; x < V; ++x) v[y][x] = src[lane * V + x];
        }
      }
      float M = m;
#pragma unroll
      for (int y = 0; y < NB; ++y) M = fmaxf(M, ml[y].x);
      const float f0 = exp2_fast(m - M);
      float f[NB];
      bool lost = i0 != first && f0 == 0.f;
#pragma unroll
      for (int y = 0; y < NB; ++y) {
        f[y] = exp2_fast(ml[y].x - M);
        lost = lost || (f[y] == 0.f && there >> y & 1u);
      }
      m = M;
      l *= f0;
#pragma unroll
      for (int y = 0; y < NB; ++y) l += ml[y].y * f[y];
      if (lost) {
#pragma unroll
        for (int x = 0; x < V; ++x) {
          o[x] = taken(o[x], f0);
#pragma unroll
          for (int y = 0; y < NB; ++y) o[x] += taken(v[y][x], f[y]);
        }
      } else {
#pragma unroll
        for (int x = 0; x < V; ++x) {
          o[x] *= f0;
#pragma unroll
          for (int y = 0; y < NB; ++y) o[x] += v[y][x] * f[y];
        }
      }
    }
  };
  auto place = [&](int c, int& row, int& hd) {
    const int col = j * CT + c;
    row = row_of(p, col);
    hd = head * p.gqa + col - row * p.gqa;
    return reinterpret_cast<T*>(const_cast<void*>(p.out.p)) + seq * p.out.seq + row * p.out.row + hd * p.out.head;
  };
  auto put_lse = [&](int row, int hd, float M, float ls) {
    p.lse[((size_t)seq * p.a.rows + row) * p.n_heads + hd] = ls == 0.f ? -INFINITY : (M + log2f(ls)) * 0.69314718055994530942f;
  };
  if (CC > 1) {
    for (int c = c0 + w; c < c1; c += NW) {
      gather(c, 0, 1);
      int row, hd;
      T* dst = place(c, row, hd);
#pragma unroll
      for (int x = 0; x < V; ++x) dst[lane * V + x] = (T)(l == 0.f ? 0.f : o[x] / l);
      if (p.lse && lane == 0) put_lse(row, hd, m, l);
    }
    return;
  }
  gather(c0, w, NW);
  if (lane == 0) {
    red_m[w] = m;
    red_l[w] = l;
  }
#pragma unroll
  for (int x = 0; x < V; ++x) red[w][lane * V + x] = o[x];
  __syncthreads();
  int row, hd;
  T* dst = place(c0, row, hd);
  for (int d = threadIdx.x; d < HD; d += blockDim.x) {
    float M = kLow, ls = 0.f, v = 0.f;
    for (int i = 0; i < NW; ++i) M = fmaxf(M, red_m[i]);
    for (int i = 0; i < NW; ++i) {
      const float f = exp2_fast(red_m[i] - M);
      ls += red_l[i] * f;
      v += taken(red[i][d], f);
    }
    dst[d] = (T)(ls == 0.f ? 0.f : v / ls);
    if (p.lse && d == 0) put_lse(row, hd, M, ls);
  }
}

// ---------------------------------------------------------------- host

// From so many columns on, tiles of 128 on tcgen05 (mk_kv4_wide.cu), us against the narrow
// kernel's, for 16 sequences of 8192 / one of 8022 / 16 of 700 positions and 4 heads a kv head.
// bf16: what no longer fits one tile of the narrow kernel, which unpacks a cache tile
// for each 32 columns: 36 columns 73 / 18.2 / 20.0 against 81 / 18.0 / 23.9, 32 columns
// 73 / 17.6 / 19.7 against 48 / 15.7 / 17.2.  fp32 (tiles of 16 columns, blocks of 256): 96
// columns 185 / 30.9 / 40.8 against 232 / 25.9 / 40.3, 80 columns 182 / 30.1 / 39.7 against
// 196 / 23.7 / 37.4.  The rule is one for batches: a single fp32 sequence is faster in the
// narrow kernel up to about 160 columns (128: 32.4 against 30.8, 192: 39.0 against 39.9).
constexpr int kWideCols = 33;
constexpr int kWideColsF32 = 81;
constexpr int kShort = 10;  // steps of a block, at most, for work that counts as short

struct Plan {
  bool wide = false;
  const void *main, *join[2];  // the join with 4 or 12 parts in flight in a warp
  int id;                    // of the variant
  int CT, SP, smem, base_smem, blocks, threads;  // columns of a tile, positions of a step; blocks of an SM
  int n_ctiles, n_entries, items, grid, join_cols, join_threads, join_many;
  int cluster;               // blocks of an item's cluster; 0: the tiles of all items in equal runs
  size_t item_off, part_off, bytes;
};

template <int HD, class T, int NT, int W, int U, int R, int B>
void take(Plan* pl) {
  using S = Shape<HD, T, NT, W, U, R, B>;
  pl->main = reinterpret_cast<const void*>(&k_kv4_attention<HD, T, NT, W, U, R, B>);
  pl->join[0] = reinterpret_cast<const void*>(&k_kv4_join<HD, T, 4>);
  pl->join[1] = reinterpret_cast<const void*>(&k_kv4_join<HD, T, 12>);
  pl->id = (HD == 64 ? 0 : 16) + (S::F32 ? 8 : 0) + NT;
  pl->CT = S::CT;
  pl->SP = S::SP;
  pl->smem = pl->base_smem = S::SMEM;
  pl->blocks = B;
  pl->threads = 32 * W;
}

// As many column tiles as the columns fill, so that the cache's tiles are
// unpacked once for all of them: up to four for bf16 rows, two for fp32 rows
// (registers hold the sums of 32 and 16 columns).
template <int HD>
void take_for(Plan* pl, int cols, int dtype) {
  if (cols >= (dtype == MK_F32 ? kWideColsF32 : kWideCols)) {
    const WideKernel w = kv4_wide_kernel(HD, dtype);
    pl->main = w.fn;
    pl->join[0] = dtype == MK_F32 ? reinterpret_cast<const void*>(&k_kv4_join<HD, float, 4>)
                                  : reinterpret_cast<const void*>(&k_kv4_join<HD, __nv_bfloat16, 4>);
    pl->join[1] = dtype == MK_F32 ? reinterpret_cast<const void*>(&k_kv4_join<HD, float, 12>)
                                  : reinterpret_cast<const void*>(&k_kv4_join<HD, __nv_bfloat16, 12>);
    pl->id = (HD == 64 ? 0 : 16) + (dtype == MK_F32 ? 8 : 0) + 7;
    pl->CT = w.CT;
    pl->SP = w.SP;
    pl->smem = pl->base_smem = w.smem;
    pl->blocks = w.blocks;
    pl->threads = w.threads;
    pl->wide = true;
    return;
  }
  if (dtype == MK_F32) cols <= 8 ? take<HD, float, 1, 4, 1, 4, 3>(pl) : take<HD, float, 2, 4, 1, 4, 2>(pl);
  else if (cols <= 8) take<HD, __nv_bfloat16, 1, 4, 2, 2, 4>(pl);
  else if (cols <= 16) take<HD, __nv_bfloat16, 2, 4, 1, 4, 3>(pl);
  else if (cols <= 24) take<HD, __nv_bfloat16, 3, 4, 1, 4, 2>(pl);
  else take<HD, __nv_bfloat16, 4, 4, 1, 4, 2>(pl);
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 152;
  }
  return n;
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
  static std::atomic<int> known[64][32][5];  // 1 + the number
  int dev = 0, log = 0, count = 0;
  while (1 << log < n) ++log;
  if (cudaGetDevice(&dev) == cudaSuccess && dev < 64) count = known[dev][pl.id][log].load();
  if (count) return count - 1;
  count = pl.blocks * sm_count() / n;
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

// Variant, grid and workspace of a call with rows; false: too many columns.
bool plan_of(const Kv4Args& c, int head_dim, int n_heads, int dtype, Plan* pl) {
  const long long cols = (long long)c.rows * (n_heads / c.n_kv_heads);
  if (cols > INT_MAX / 64) return false;
  if (head_dim == 64) take_for<64>(pl, (int)cols, dtype);
  else take_for<128>(pl, (int)cols, dtype);
  const long long ct = (cols + pl->CT - 1) / pl->CT, entries = ct * c.n_seqs, items = entries * c.n_kv_heads;
  const long long most = (long long)c.max_pages * (kPageTokens / pl->SP);  // steps of an item
  if (items > INT_MAX / 32 || (most + kOver) * c.n_kv_heads > INT_MAX) return false;
  pl->n_ctiles = (int)ct;
  pl->n_entries = (int)entries;
  pl->items = (int)items;
  const int sms = sm_count();
  const long long room = std::min(pl->blocks * sms, kMaxBlocks);  // blocks that run at once
  pl->cluster = 0;
  // Short work: an item is a cluster of up to 16 blocks, while all clusters run at
  // once (16 sequences of 256 to 8448 positions with clusters of 8: 15.8 us; as equal runs, with
  // the second kernel and the scan of all lengths, 18.0), joined through their shared memory.
  // But a ragged batch is not levelled and a long item has 16 blocks at most, which loses once
  // a block has more than about ten steps (131071 positions: 57.6 us against 23.6, 64 sequences of
  // 4096 to 16384: 112 against 77).
  int n = 1;
  while (n < 16 && 2 * n <= most && items <= clusters_at_once(*pl, head_dim, 2 * n)) n *= 2;
  if (!pl->wide && (most + n - 1) / n <= kShort) {
    pl->cluster = n;
    pl->smem += join_room(*pl, head_dim, n);
    pl->grid = (int)(items * n);
    pl->item_off = pl->part_off = pl->bytes = 0;
    return true;
  }
  pl->grid = (int)std::min<long long>(room, items * most);
  // The join.  Up to ten columns an SM are a block each, with as many warps as the item has
  // parts (about grid / items), and 12 parts in flight in each warp where blocks are few and parts many
  // (131071 positions, 152 parts: 23.8 us; 26.5 with 4, whose fewer registers serve more
  // blocks).  More columns are a warp each, 8 a block up to 54 an SM, then 16 (128 rows at 8022 positions, 2048
  // columns: 34.6 us, 49 by blocks; 16 sequences with up to 5 drafted rows, 1280: 30.9 by warps, 29.9).
  const long long all_cols = items * std::min<long long>(cols, pl->CT);
  pl->join_cols = all_cols <= 10 * sms ? 1 : all_cols <= 54 * sms ? 8 : 16;
  int nw = 2;
  while (nw < 16 && nw * 2 * items <= pl->grid) nw *= 2;
  pl->join_many = pl->grid / 64 >= items && all_cols <= sms;  // 64 parts an item and more, a block an SM at most
  pl->join_threads = 32 * (pl->join_cols > 1 ? 8 : nw);
  pl->item_off = 16;
  pl->part_off = pl->item_off + (size_t)items * sizeof(longlong2);
  pl->bytes = pl->part_off + 2 * (size_t)pl->grid * pl->CT * (head_dim + 4) * sizeof(float);
  return true;
}

template <int HD, class T>
const void* join_of(bool many) {
  return many ? reinterpret_cast<const void*>(&k_kv4_join<HD, T, 12>) : reinterpret_cast<const void*>(&k_kv4_join<HD, T, 4>);
}

}  // namespace

const void* kv4_join_kernel(int head_dim, int dtype, bool many) {
  if (dtype == MK_F32) return head_dim == 64 ? join_of<64, float>(many) : join_of<128, float>(many);
  return head_dim == 64 ? join_of<64, __nv_bfloat16>(many) : join_of<128, __nv_bfloat16>(many);
}

bool kv4_attention_bytes(const Kv4Args& a, int head_dim, int n_heads, int dtype, size_t* bytes) {
  Plan pl;
  if (!plan_of(a, head_dim, n_heads, dtype, &pl)) return false;
  *bytes = pl.bytes;
  return true;
}

int kv4_attention(const Kv4Args& a, int head_dim, int n_heads, const Kv4Rows& q, int dtype, float scale,
                  const Kv4Rows& out, float* lse, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  Plan pl;
  if (!plan_of(a, head_dim, n_heads, dtype, &pl))
    return host_fail(MK_ERR_INVALID_ARG, "n_seqs x rows x n_heads or max_pages x n_kv_heads is too large");
  if (pl.bytes && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u) || workspace_bytes < pl.bytes))
    return host_fail(MK_ERR_INVALID_ARG, "workspace is NULL, not 16-byte aligned or smaller than mk_kv4_attention_bytes");
  AttArgs p;
  p.a = a;
  p.q = q;
  p.out = out;
  p.lse = lse;
  p.c = (float)((double)scale * 1.4426950408889634 * kDown);
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
    char* ws = static_cast<char*>(workspace);
    p.total = reinterpret_cast<long long*>(ws);
    p.item = reinterpret_cast<longlong2*>(ws + pl.item_off);
    p.part = reinterpret_cast<float*>(ws + pl.part_off);
  }
  cudaError_t e = allow_smem(pl);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  cfg.gridDim = dim3(pl.grid);
  cfg.blockDim = dim3(pl.threads);
  cfg.dynamicSmemBytes = pl.smem;
  cfg.stream = stream;
  cfg.attrs = at;
  if (e == cudaSuccess) {
    if (pl.cluster > 1) {
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = pl.cluster;
      at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
      cfg.numAttrs = 1;
    }
    void* args[] = {&p};
    e = cudaLaunchKernelExC(&cfg, pl.main, args);
  }
  if (e == cudaSuccess && !pl.cluster) {
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(pl.items, (pl.CT + pl.join_cols - 1) / pl.join_cols);
    cfg.blockDim = dim3(pl.join_threads);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    void* args[] = {&p, &pl.CT, &pl.SP, &pl.grid, &pl.join_cols};
    e = cudaLaunchKernelExC(&cfg, pl.join[pl.join_many], args);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return host_fail(MK_ERR_CUDA, (std::string("kv4 attention: ") + cudaGetErrorString(e)).c_str());
  }
  return MK_OK;
}

}  // namespace mk

using namespace mk;

static int check_attention(const mk_kv4_cache* c, int n_heads, int dtype, bool* empty) {
  if (int r = kv4_check_cache(c, empty)) return r;
  if (n_heads < 1 || n_heads % c->n_kv_heads || n_heads > 4096)
    return host_fail(MK_ERR_INVALID_ARG, "n_heads must be a multiple of n_kv_heads, at most 4096");
  if (dtype != MK_F32 && dtype != MK_BF16) return host_fail(MK_ERR_INVALID_ARG, "dtype must be MK_F32 or MK_BF16");
  return MK_OK;
}

extern "C" MK_API size_t mk_kv4_attention_bytes(const mk_kv4_cache* c, int32_t n_heads, int32_t dtype) {
  bool empty = false;
  size_t bytes = 0;
  if (check_attention(c, n_heads, dtype, &empty) || empty) return 0;
  return kv4_attention_bytes(kv4_args(*c), c->head_dim, n_heads, dtype, &bytes) ? bytes : 0;
}

extern "C" MK_API int mk_kv4_attention(const mk_kv4_cache* c, int32_t n_heads, const mk_kv4_rows* q, int32_t dtype,
                                       float scale, const mk_kv4_rows* out, float* lse, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  host_clear_error();
  bool empty = false;
  if (int r = check_attention(c, n_heads, dtype, &empty)) return r;
  if (!(scale > -1e18f && scale < 1e18f)) return host_fail(MK_ERR_INVALID_ARG, "scale must lie within +-1e18");
  if (empty) return MK_OK;
  if (int r = kv4_check_rows(q, dtype, "q")) return r;
  if (int r = kv4_check_rows(out, dtype, "out")) return r;
  return kv4_attention(kv4_args(*c), c->head_dim, n_heads, kv4_rows(*q), dtype, scale, kv4_rows(*out), lse, workspace,
                       workspace_bytes, (cudaStream_t)stream);
}
