// The masses of cached positions: what a call's rows gave each of them.
//
// mass[p] = decay mass[p] (0 for the call's own new positions) + sum over the rows r that see
// p and the heads h of its kv head of 2^(s_rhp - lse_rh log2 e).  Calls of a few columns kept
// their scores (mk_paged_attention.cu): 4 bytes a column and position instead of
// K's 2 head_dim.  Calls of more form them again, next to the exponentials.
#include <algorithm>
#include <type_traits>

#include "mk_paged_att.cuh"
#include "mk_tcgen05.cuh"

namespace mk {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// A thread for a position: its columns' scores in words of four (16 sequences of 256 to 8448, one row: 7 us of 38).
__global__ void __launch_bounds__(256) k_mass_scores(const __grid_constant__ PagedAtt pa, const __grid_constant__ PagedMass ms, int chunks) {
  const AttArgs& p = pa.t;
  const int item = blockIdx.x / chunks, t = (blockIdx.x - item * chunks) * 256 + threadIdx.x;
  const int seq = item / p.a.n_kv_heads, head = item - seq * p.a.n_kv_heads;
  behind();
  int len, nn;
  seq_extent(p.a, seq, len, nn);
  if (t >= len || nn == 0) return;
  float* to = ms.p + seq * ms.seq + head * ms.head + t;
  const float old = t < len - nn ? *to : 0.f;
  float sum = 0.f;  // (the weights by themselves: next to a large mass each would be rounded to its step)
  const bool there = page_of(p.a, seq, t) >= 0;
  const float* sc = pa.scores + ((size_t)item * p.a.max_pages * kPageTokens + t) * pa.score_cols;
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

// ---------------------------------------------------------------- many columns: the scores formed again
//
// S^T = K Q^T on tcgen05: 128 positions of a page x N query columns, so that a thread has a
// position (a TMEM lane) and adds the columns' exponentials in its own registers, 32 scores at a time.  A
// block keeps the K of two pages in shared memory and streams tiles of query columns past them; two places of
// scores for each page let the products run beside the exponentials.  (With rows of the columns in TMEM's lanes, as in the
// attention, the sums over them would cross threads.)  1024 rows of 16 heads over 8022 positions: 38 us, of 16 for the
// products: the columns' warps take about 1,770 cycles for a tile of 128 columns and 256 positions, of which
// exponentials alone are 1,024 (32 a cycle and SM).
//
// The columns of a kv head lie in the workspace as rows of bf16 (k_columns: strides, fp32's three
// parts and padding are dealt with once).  All items (sequence, kv head, two pages) are laid end to end and cut into
// equal runs of tiles; items that are cut leave partial sums, which a second kernel adds in the runs' order.

template <int HD, class T>
struct MassShape {
  static constexpr bool F32 = std::is_same<T, float>::value;
  static constexpr int NG = HD / 64, P = F32 ? 3 : 1;
  static constexpr int N = F32 ? 64 : 128;           // columns of a tile
  static constexpr int KB = NG * 128 * 128;          // bytes of a page's K
  static constexpr int KS = F32 ? 1 : 2;             // places of two pages
  static constexpr int QT = NG * N * 128;            // bytes of a part of a tile of columns
  static constexpr int QS = 2;                       // places of tiles
  static constexpr int SMEM = 1024 + KS * 2 * KB + QS * P * QT;
  static constexpr int CW = 16, THREADS = 32 * (CW + 3);  // a page's four warps for each half of a tile's columns, copies, products, log-sum-exps
};
constexpr int kSpan = 2 * kPageTokens;  // positions of an item
constexpr int kSetUp = 2;               // tiles that an item's set-up counts as
constexpr int kLse = 8;                 // tiles whose log-sum-exps are held

struct MassArgs {
  PagedAtt pa;
  PagedMass ms;
  uint16_t* columns;  // [part][n_seqs][n_kv_heads][cols_up][HD]
  long long part_rows;  // rows of a part
  long long* total;   // places of the call
  longlong2* item;    // [n_seqs * n_kv_heads * spans]: first place and first block of an item, -1: done
  float* part;        // [2 * grid][kSpan]
  int cols_up, spans, N;
};

// A sequence's items: T tiles for spans that all its rows see, fewer for the others.
struct MassSeq {
  int len, nn, tiles, spans, same;  // same: spans that have all tiles
  long long per_head;               // places of a head
  // the first tile that sees span j
  __device__ __forceinline__ int first(const MassArgs& a, int j) const {
    const long long r0 = max(0ll, (long long)j * kSpan - (len - nn));
    return (int)(r0 * a.pa.t.gqa / a.N);
  }
  __device__ __forceinline__ MassSeq() {}
  __device__ __forceinline__ MassSeq(const MassArgs& a, int s) {
    per_head = 0;
    len = nn = tiles = spans = same = 0;
    if (s >= a.pa.t.a.n_seqs) return;
    seq_extent(a.pa.t.a, s, len, nn);
    if (!nn || !len) return;
    tiles = (int)(((long long)nn * a.pa.t.gqa + a.N - 1) / a.N);
    spans = (len + kSpan - 1) / kSpan;
    same = len >= nn ? min(spans, (len - nn) / kSpan + 1) : 0;
    per_head = (long long)same * (tiles + kSetUp);
    for (int j = same; j < spans; ++j) per_head += tiles - first(a, j) + kSetUp;
  }
};
// The part of an item that a block takes: tiles t0 .. t1 of the nt that see its span.
struct MassRun {
  int seq, head, span, c0, nt, t0, t1, len, nn;
  long long base;  // the item's first place
};
// The run at place pos, in sequence s whose first place is s_base; held to [pos, hi).
__device__ __forceinline__ MassRun mass_run(const MassArgs& a, const MassSeq& q, int s, long long s_base, long long pos, long long hi) {
  MassRun r;
  r.seq = s;
  r.len = q.len;
  r.nn = q.nn;
  const long long at = pos - s_base;
  r.head = (int)(at / q.per_head);
  long long in = at - r.head * q.per_head;
  const long long full = (long long)q.same * (q.tiles + kSetUp);
  if (in < full) {
    r.span = (int)(in / (q.tiles + kSetUp));
    in -= (long long)r.span * (q.tiles + kSetUp);
  } else {
    in -= full;
    for (r.span = q.same; r.span + 1 < q.spans; ++r.span) {
      const int n = q.tiles - q.first(a, r.span) + kSetUp;
      if (in < n) break;
      in -= n;
    }
  }
  r.c0 = q.first(a, r.span);
  r.nt = q.tiles - r.c0;
  r.base = pos - in;
  r.t0 = max(0, (int)in - kSetUp);
  r.t1 = max(0, (int)min((long long)(r.nt + kSetUp), in + hi - pos) - kSetUp);
  return r;
}

// Rows of query columns [part][seq][kv head][column][HD], 16 bytes a thread; zeros for padding.
template <int HD, class T>
__global__ void __launch_bounds__(256) k_columns(const __grid_constant__ MassArgs a) {
  constexpr int W = HD / 8;
  const AttArgs& p = a.pa.t;
  behind();
  const long long x = (long long)blockIdx.x * 256 + threadIdx.x, row = x / W;
  if (row >= a.part_rows) return;
  const int w = (int)(x % W), col = (int)(row % a.cols_up);
  const long long sh = row / a.cols_up;
  const int head = (int)(sh % p.a.n_kv_heads), seq = (int)(sh / p.a.n_kv_heads);
  int len, nn;
  seq_extent(p.a, seq, len, nn);
  const int r = row_of(p, col);
  const bool there = col < p.cols && r < nn && len - nn + r >= 0;
  const T* src = reinterpret_cast<const T*>(p.q.p) + seq * p.q.seq + r * p.q.row + (head * p.gqa + col - r * p.gqa) * p.q.head + 8 * w;
  uint4* dst = reinterpret_cast<uint4*>(a.columns) + x;
  if constexpr (std::is_same<T, float>::value) {
    float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
    if (there) u = reinterpret_cast<const float4*>(src)[0], v = reinterpret_cast<const float4*>(src)[1];
    const Parts y[8] = {parts_of(u.x), parts_of(u.y), parts_of(u.z), parts_of(u.w), parts_of(v.x), parts_of(v.y), parts_of(v.z), parts_of(v.w)};
#pragma unroll
    for (int i = 0; i < 3; ++i)
      dst[i * a.part_rows * W] = make_uint4(both(y[0], y[1], i), both(y[2], y[3], i), both(y[4], y[5], i), both(y[6], y[7], i));
  } else {
    *dst = there ? *reinterpret_cast<const uint4*>(src) : make_uint4(0, 0, 0, 0);
  }
}

constexpr int kMassRuns = 8;

template <int HD, class T>
__global__ void __launch_bounds__(MassShape<HD, T>::THREADS, 1)
    k_mass_wide(const __grid_constant__ MassArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap qmap) {
  using S = MassShape<HD, T>;
  constexpr int NG = S::NG, N = S::N, CW = S::CW, KS = S::KS, QS = S::QS;
  const AttArgs& p = a.pa.t;
  extern __shared__ uint8_t sm_raw[];
  uint8_t* sm = sm_raw + ((1024 - (smem_addr(sm_raw) & 1023)) & 1023);
  __shared__ __align__(8) uint64_t k_full[KS], k_empty[KS], q_full[QS], q_empty[QS], s_full[2][2], s_empty[2][2], l_full[kLse], l_empty[kLse], run_full[kMassRuns], h_full, h_empty, drain;
  __shared__ MassRun says[kMassRuns];
  __shared__ __align__(16) float less[kLse][N];  // minus the log-sum-exp (log2); -infinity: a column that gives nothing
  __shared__ int lims[kLse][N];                  // positions that a column sees
  __shared__ int cut[kLse];                      // a column of the tile does not see all of an item's positions
  __shared__ float halves[kSpan];                // a run's sums of the second half of the columns
  __shared__ uint32_t tm_base;
  __shared__ volatile int give_up;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  uint8_t *k_op = sm, *q_op = sm + KS * 2 * S::KB;  // [place][page][NG][128][128 bytes], [place][part][NG][N][128 bytes]
  if (tid == 0) {
    auto init = [](uint64_t* b, int n) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(b)), "r"(n) : "memory");
    };
    for (int i = 0; i < KS; ++i) init(&k_full[i], 1), init(&k_empty[i], 1);
    for (int i = 0; i < QS; ++i) init(&q_full[i], 1), init(&q_empty[i], 1);
    for (int i = 0; i < 4; ++i) init(&s_full[i >> 1][i & 1], 1), init(&s_empty[i >> 1][i & 1], CW / 2);
    for (int i = 0; i < kLse; ++i) init(&l_full[i], 1), init(&l_empty[i], CW);
    for (int i = 0; i < kMassRuns; ++i) init(&run_full[i], 1);
    init(&h_full, CW / 2);
    init(&h_empty, CW / 2);
    init(&drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    give_up = 0;
  }
  if (w == CW + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&tm_base)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  before_sync();
  __syncthreads();
  after_sync();
  const uint32_t tm = tm_base;  // scores of page x in place b at 256 b + 128 x
  auto take_run = [&](uint32_t i, MassRun& r) {
    if (!wait_for(smem_addr(&run_full[i % kMassRuns]), (i / kMassRuns) & 1, &give_up, p.a.status)) return false;
    r = says[i % kMassRuns];
    return r.t1 > r.t0;
  };
  behind();

  if (w == CW) {  // ---- runs, copies and log-sum-exps
    // the block's places, and the sequence of the first
    long long total = 0, lo, hi, s_base = 0;
    for (int s = lane; s < p.a.n_seqs; s += 32) total += MassSeq(a, s).per_head * p.a.n_kv_heads;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    lo = first_place(total, blockIdx.x, gridDim.x);
    hi = first_place(total, blockIdx.x + 1, gridDim.x);
    if (blockIdx.x == 0 && lane == 0) *a.total = total;
    int seq = 0;
    if (lo < hi)
      for (int s0 = 0; s0 < p.a.n_seqs; s0 += 32) {
        const long long n = MassSeq(a, s0 + lane).per_head * p.a.n_kv_heads;
        long long incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long up = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += up;
        }
        const uint32_t has = __ballot_sync(0xffffffffu, lo < s_base + incl);
        if (has) {
          const int f = __ffs(has) - 1;
          seq = s0 + f;
          s_base += __shfl_sync(0xffffffffu, incl - n, f);
          break;
        }
        s_base += __shfl_sync(0xffffffffu, incl, 31);
      }
    MassSeq q(a, seq);
    long long pos = lo;
    uint32_t n_runs = 0, n_items = 0, tile = 0;
    bool ok = true;
    while (pos < hi && ok) {
      while (seq < p.a.n_seqs && pos >= s_base + q.per_head * p.a.n_kv_heads) {
        s_base += q.per_head * p.a.n_kv_heads;
        q = MassSeq(a, ++seq);
      }
      if (seq >= p.a.n_seqs) break;  // lengths that change under the call
      const MassRun r = mass_run(a, q, seq, s_base, pos, hi);
      pos = min(hi, r.base + r.nt + kSetUp);
      if (r.t1 <= r.t0) continue;
      if (lane == 0) {
        says[n_runs % kMassRuns] = r;
        arrive(smem_addr(&run_full[n_runs % kMassRuns]));
      }
      ++n_runs;
      // the two pages' K; a page outside the pool, or none: zeros
      const int ks = n_items % KS;
      ok = n_items < KS || wait_for(smem_addr(&k_empty[ks]), (n_items / KS - 1) & 1, &give_up, p.a.status);
      ++n_items;
      if (ok && lane == 0) {
        const uint32_t bar = smem_addr(&k_full[ks]);
        expect(bar, 2 * S::KB);
        for (int x = 0; x < 2; ++x) {
          const int at = r.span * kSpan + x * kPageTokens, pg = at < r.len ? page_of(p.a, r.seq, at) : -1;
          tma_rows(smem_addr(k_op + (ks * 2 + x) * S::KB), &kmap,
                   pg < 0 ? p.a.n_pages * 2 * p.a.n_kv_heads * kPageTokens : paged_row(p.a, pg, 0, r.head, 0), bar);
        }
      }
      __syncwarp();
      for (int t = r.t0; t < r.t1 && ok; ++t, ++tile) {
        const int qs = tile % QS, col0 = (r.c0 + t) * N;
        ok = tile < QS || wait_for(smem_addr(&q_empty[qs]), (tile / QS - 1) & 1, &give_up, p.a.status);
        if (ok && lane == 0) {
          const uint32_t bar = smem_addr(&q_full[qs]);
          expect(bar, S::P * S::QT);
          for (int x = 0; x < S::P; ++x)
            tma_rows(smem_addr(q_op + (qs * S::P + x) * S::QT), &qmap,
                     (int)(x * a.part_rows + ((long long)r.seq * p.a.n_kv_heads + r.head) * a.cols_up + col0), bar);
        }
        __syncwarp();
        if (!ok) break;
      }
    }
    if (lane == 0) {
      says[n_runs % kMassRuns].t0 = says[n_runs % kMassRuns].t1 = 0;
      arrive(smem_addr(&run_full[n_runs % kMassRuns]));
    }
    if (give_up && lane == 0) {  // copies in flight land before the block ends
      int none = 0;
      for (uint32_t i = n_items > KS ? n_items - KS : 0; i < n_items; ++i) wait_for(smem_addr(&k_full[i % KS]), (i / KS) & 1, &none, nullptr);
      for (uint32_t i = tile > QS ? tile - QS : 0; i < tile; ++i) wait_for(smem_addr(&q_full[i % QS]), (i / QS) & 1, &none, nullptr);
    }
  } else if (w == CW + 2) {  // ---- log-sum-exps (next to the copies they took 1,200 cycles of a tile's 1,900)
    uint32_t tile = 0;
    bool ok = true;
    MassRun r;
    for (uint32_t n_runs = 0; ok && take_run(n_runs, r); ++n_runs) {
      float ahead[N / 32];  // a tile's, read while the last tile's are handed on
      auto read = [&](int t) {
#pragma unroll
        for (int i = 0; i < N / 32; ++i) {
          const int col = min((r.c0 + t) * N + 32 * i + lane, p.cols - 1), row = row_of(p, col);
          ahead[i] = __ldcg(&p.lse[((size_t)r.seq * p.a.rows + row) * p.n_heads + r.head * p.gqa + col - row * p.gqa]);
        }
      };
      read(r.t0);
      for (int t = r.t0; t < r.t1 && ok; ++t, ++tile) {
        const int ls = tile % kLse;
        float now[N / 32];
#pragma unroll
        for (int i = 0; i < N / 32; ++i) now[i] = ahead[i];
        if (t + 1 < r.t1) read(t + 1);
        ok = tile < kLse || wait_for(smem_addr(&l_empty[ls]), (tile / kLse - 1) & 1, &give_up, p.a.status);
        if (!ok) break;
        bool some = false;
#pragma unroll
        for (int i = 0; i < N / 32; ++i) {
          const int x = 32 * i + lane, col = (r.c0 + t) * N + x, row = row_of(p, col);
          const int lim = col < p.cols && row < r.nn ? max(0, r.len - r.nn + row + 1) : 0;
          float l = -INFINITY;
          if (lim) l = now[i] == -INFINITY ? now[i] : now[i] * -kLog2e;  // (its scores have no weight)
          // (a column that is none counts: its row of zeros times an infinite K is NaN)
          some = some || lim < min(r.len, (r.span + 1) * kSpan);
          less[ls][x] = l;
          lims[ls][x] = lim;
        }
        some = __any_sync(0xffffffffu, some);
        __syncwarp();  // (a vote does not order memory: lane 0 arrives for what all lanes have stored)
        if (lane == 0) {
          cut[ls] = some;
          arrive(smem_addr(&l_full[ls]));
        }
        __syncwarp();
      }
    }
  } else if (w == CW + 1) {  // ---- the products
    constexpr uint32_t id = (1u << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | ((128 >> 4) << 24);  // bf16, fp32 sums
    const uint32_t tmu = uniform(tm), ku = uniform(smem_addr(k_op)), qu = uniform(smem_addr(q_op));
    uint32_t tile = 0;
    MassRun r;
    bool ok = true;
    for (uint32_t n_runs = 0; take_run(n_runs, r); ++n_runs) {
      const uint32_t ks = uniform(n_runs % KS);
      ok = wait_for(smem_addr(&k_full[ks]), (n_runs / KS) & 1, &give_up, p.a.status) && ok;
      for (int t = r.t0; t < r.t1; ++t, ++tile) {
        const uint32_t qs = uniform(tile % QS), b = uniform(tile & 1), end = uniform(t + 1 == r.t1);
        ok = wait_for(smem_addr(&q_full[qs]), (tile / QS) & 1, &give_up, p.a.status) && ok;
#pragma unroll
        for (int pg = 0; pg < 2; ++pg) {
          if (tile >= 2) ok = wait_for(smem_addr(&s_empty[pg][b]), (tile / 2 - 1) & 1, &give_up, p.a.status) && ok;
          after_sync();
          if (ok && elect_one()) {
            const uint64_t kd = operand(ku + (ks * 2 + pg) * S::KB);
#pragma unroll
            for (int x = S::P - 1; x >= 0; --x) {  // q's low parts first
              const uint64_t qd = operand(qu + (qs * S::P + x) * S::QT);
#pragma unroll
              for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                  const uint64_t ka = kd + ((g * 128 * 128 + kk * 32) >> 4), qb = qd + ((g * N * 128 + kk * 32) >> 4);
                  if (g == 0 && kk == 0 && x == S::P - 1) mma_ss<false>(tmu + 256 * b + 128 * pg, ka, qb, id);
                  else mma_ss<true>(tmu + 256 * b + 128 * pg, ka, qb, id);
                }
            }
            commit(smem_addr(&s_full[pg][b]));
            if (pg) commit(smem_addr(&q_empty[qs]));
            if (pg && end) commit(smem_addr(&k_empty[ks]));
          }
          __syncwarp();
        }
      }
      if (!ok || give_up) break;
    }
    if (give_up) {  // products in flight end before the block does
      int none = 0;
      if (lane == 0) commit(smem_addr(&drain));
      wait_for(smem_addr(&drain), 0, &none, nullptr);
    }
  } else if (w < CW) {  // ---- a position each
    // (two threads: a half of the columns each)
    const int pg = w >> 2 & 1, half = w >> 3, me = tid & (kSpan - 1);
    const uint32_t tm_s = tm + 128 * pg + ((uint32_t)(32 * (w & 3)) << 16);
    uint32_t tile = 0;
    MassRun r;
    for (uint32_t n_runs = 0; take_run(n_runs, r); ++n_runs) {
      const int at = r.span * kSpan + me;  // the position (me: page pg, lane of TMEM)
      bool in = false;
      if (at < r.len) {
        const int page = table_row(p.a, r.seq)[at / kPageTokens];
        in = page >= 0 && page < p.a.n_pages;
      }
      uint64_t sum[2] = {0, 0};
      const uint64_t c2 = pair(p.c, p.c);
      bool ok = true;
      for (int t = r.t0; t < r.t1; ++t, ++tile) {
        const int ls = tile % kLse, b = tile & 1;
        ok = wait_for(smem_addr(&l_full[ls]), (tile / kLse) & 1, &give_up, p.a.status) && ok;
        ok = wait_for(smem_addr(&s_full[pg][b]), (tile / 2) & 1, &give_up, p.a.status) && ok;
        after_sync();
        if (ok && !give_up) {
          auto add = [&](auto cut_) {
            constexpr bool CUT = decltype(cut_)::value;
#pragma unroll 1
            for (int c = half * (N / 2); c < (half + 1) * (N / 2); c += 32) {
              float s[32];
              tm_read32(tm_s + 256 * b + c, s);
#pragma unroll
              for (int x = 0; x < 32; x += 4) {
                const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(&less[ls][c + x]);
                const uint64_t l2[2] = {l.x, l.y};
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  float2 e = unpair(fma2(pair(s[x + 2 * y], s[x + 2 * y + 1]), c2, l2[y]));
                  e.x = exp2_fast(e.x), e.y = exp2_fast(e.y);
                  if (CUT && at >= lims[ls][c + x + 2 * y]) e.x = 0.f;
                  if (CUT && at >= lims[ls][c + x + 2 * y + 1]) e.y = 0.f;
                  sum[y] = add2(sum[y], pair(e.x, e.y));
                }
              }
            }
          };
          if (cut[ls]) add(std::true_type());
          else add(std::false_type());
        }
        before_sync();
        __syncwarp();
        if (lane == 0) {
          arrive(smem_addr(&s_empty[pg][b]));
          arrive(smem_addr(&l_empty[ls]));
        }
      }
      const float2 both = unpair(add2(sum[0], sum[1]));
      float v = !ok ? NAN : in ? both.x + both.y : 0.f;
      if (half) {
        if (n_runs) ok = wait_for(smem_addr(&h_empty), (n_runs - 1) & 1, &give_up, p.a.status) && ok;  // the last run's are read
        halves[me] = v;
        __syncwarp();
        if (lane == 0) arrive(smem_addr(&h_full));
      } else {
        ok = wait_for(smem_addr(&h_full), n_runs & 1, &give_up, p.a.status) && ok;
        v = ok ? v + halves[me] : NAN;
        __syncwarp();
        if (lane == 0) arrive(smem_addr(&h_empty));
        const bool whole = r.t0 == 0 && r.t1 == r.nt;
        if (!whole) {
          a.part[(size_t)part_slot(blockIdx.x, r.t0) * kSpan + me] = v;
        } else if (at < r.len) {
          float* to = a.ms.p + r.seq * a.ms.seq + r.head * a.ms.head + at;
          *to = at < r.len - r.nn ? fmaf(a.ms.decay, *to, v) : v;
        }
        if (tid == 0 && r.t0 == 0)
          a.item[((size_t)r.seq * p.a.n_kv_heads + r.head) * a.spans + r.span] = make_longlong2(whole ? -1 : r.base, blockIdx.x);
      }
      if (!ok) break;
    }
  }
  before_sync();
  __syncthreads();
  if (w == CW + 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm));
}

// Items cut between blocks: their parts added in the blocks' order, a thread for a position.
__global__ void __launch_bounds__(kSpan) k_mass_join(const __grid_constant__ MassArgs a, int G, int items) {
  const Kv4Args& c = a.pa.t.a;
  behind();
  for (int i = blockIdx.x; i < items; i += gridDim.x) {
    const int span = i % a.spans, sh = i / a.spans, seq = sh / c.n_kv_heads, head = sh - seq * c.n_kv_heads;
    int len, nn;
    seq_extent(c, seq, len, nn);
    const int at = span * kSpan + threadIdx.x;
    if (!nn || at >= len) continue;
    const longlong2 it = a.item[i];
    if (it.x < 0 || it.y < 0 || it.y >= G) continue;  // done by its block
    const MassSeq q(a, seq);
    const long long total = *a.total, n = q.tiles - q.first(a, span);
    float v = 0.f;
    for (long long b = it.y; b < G; ++b) {
      const long long lo = first_place(total, b, G) - it.x - kSetUp, hi = first_place(total, b + 1, G) - it.x - kSetUp;
      if (lo >= n) break;
      if (hi > 0 && hi > lo) v += a.part[(size_t)part_slot(b, lo > 0) * kSpan + threadIdx.x];
    }
    float* to = a.ms.p + seq * a.ms.seq + head * a.ms.head + at;
    *to = at < len - nn ? fmaf(a.ms.decay, *to, v) : v;
  }
}

struct MassPlan {
  int N, P, cols_up, spans, grid;
  size_t item_off, part_off, col_off, bytes;
};
MassPlan plan_of(const Kv4Args& a, int head_dim, int n_heads, int dtype) {
  MassPlan m;
  m.N = dtype == MK_F32 ? 64 : 128;
  m.P = dtype == MK_F32 ? 3 : 1;
  const int cols = a.rows * (n_heads / a.n_kv_heads);
  m.cols_up = (cols + m.N - 1) / m.N * m.N;
  m.spans = (a.max_pages + 1) / 2;
  m.grid = device_sms();
  m.item_off = 16;
  m.part_off = m.item_off + (size_t)a.n_seqs * a.n_kv_heads * m.spans * sizeof(longlong2);
  m.col_off = (m.part_off + 2 * (size_t)m.grid * kSpan * sizeof(float) + 127) & ~(size_t)127;
  m.bytes = m.col_off + (size_t)m.P * a.n_seqs * a.n_kv_heads * m.cols_up * head_dim * 2;
  return m;
}
MassArgs args_of(const PagedAtt& p, const MassPlan& m, int head_dim) {
  MassArgs a;
  a.pa = p;
  a.ms = {nullptr, 0, 0, 0.f};
  a.total = reinterpret_cast<long long*>(p.mass_ws);
  a.item = reinterpret_cast<longlong2*>(p.mass_ws + m.item_off);
  a.part = reinterpret_cast<float*>(p.mass_ws + m.part_off);
  a.columns = reinterpret_cast<uint16_t*>(p.mass_ws + m.col_off);
  a.part_rows = (long long)p.t.a.n_seqs * p.t.a.n_kv_heads * m.cols_up;
  a.cols_up = m.cols_up;
  a.spans = m.spans;
  a.N = m.N;
  return a;
}
template <int HD, class T>
cudaError_t launch_wide(const MassArgs& a, const MassPlan& m, const CUtensorMap& kmap, const CUtensorMap& qmap, cudaStream_t st) {
  using S = MassShape<HD, T>;
  cudaError_t e = cudaFuncSetAttribute(k_mass_wide<HD, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
  if (e != cudaSuccess) return e;
  MassArgs g = a;
  CUtensorMap km = kmap, qm = qmap;
  int G = m.grid, items = a.pa.t.a.n_seqs * a.pa.t.a.n_kv_heads * a.spans;
  void* args[] = {&g, &km, &qm};
  e = launch(reinterpret_cast<const void*>(&k_mass_wide<HD, T>), m.grid, S::THREADS, S::SMEM, st, args);
  void* jargs[] = {&g, &G, &items};
  if (e == cudaSuccess) e = launch(reinterpret_cast<const void*>(&k_mass_join), std::min(items, 16 * m.grid), kSpan, 0, st, jargs);
  return e;
}

}  // namespace

// Grids (with room for the join's stride), rows of a tensor map and positions (of whole spans) in 31 bits.
bool paged_mass_fits(const Kv4Args& a, int n_heads, int dtype, bool wide) {
  const long long items = (long long)a.n_seqs * a.n_kv_heads, positions = (long long)a.max_pages * kPageTokens;
  if (positions + kSpan - 1 > INT_MAX || items * ((positions + kSpan - 1) / kSpan) > INT_MAX / 2) return false;
  if (!wide) return true;
  const long long N = dtype == MK_F32 ? 64 : 128, cols = (long long)a.rows * (n_heads / a.n_kv_heads);
  return items * ((cols + N - 1) / N * N) * (dtype == MK_F32 ? 3 : 1) <= INT_MAX;
}
size_t paged_mass_bytes(const Kv4Args& a, int head_dim, int n_heads, int dtype) { return plan_of(a, head_dim, n_heads, dtype).bytes; }

cudaError_t paged_mass_begin(const PagedAtt& p, int head_dim, int dtype, cudaStream_t st) {
  const MassArgs a = args_of(p, plan_of(p.t.a, head_dim, p.t.n_heads, dtype), head_dim);
  const long long threads = a.part_rows * (head_dim / 8);
  MassArgs g = a;
  void* args[] = {&g};
  const void* f = head_dim == 64 ? dtype == MK_F32 ? reinterpret_cast<const void*>(&k_columns<64, float>)
                                                   : reinterpret_cast<const void*>(&k_columns<64, __nv_bfloat16>)
                  : dtype == MK_F32 ? reinterpret_cast<const void*>(&k_columns<128, float>)
                                    : reinterpret_cast<const void*>(&k_columns<128, __nv_bfloat16>);
  return launch(f, (unsigned)((threads + 255) / 256), 256, 0, st, args);
}

cudaError_t paged_mass(const PagedAtt& p, const PagedMass& m, int head_dim, int dtype, const CUtensorMap& map, cudaStream_t st) {
  const Kv4Args& a = p.t.a;
  if (p.scores) {
    const int chunks = (a.max_pages * kPageTokens + 255) / 256, items = a.n_seqs * a.n_kv_heads;
    PagedAtt pa = p;
    PagedMass ms = m;
    int n = chunks;
    void* args[] = {&pa, &ms, &n};
    return launch(reinterpret_cast<const void*>(&k_mass_scores), (unsigned)(items * chunks), 256, 0, st, args);
  }
  const MassPlan pl = plan_of(a, head_dim, p.t.n_heads, dtype);
  MassArgs g = args_of(p, pl, head_dim);
  g.ms = m;
  CUtensorMap qmap;
  if (rows_map(&qmap, g.columns, g.part_rows * pl.P, head_dim, pl.N)) return cudaErrorInvalidValue;
  if (head_dim == 64 && dtype == MK_F32) return launch_wide<64, float>(g, pl, map, qmap, st);
  if (head_dim == 64) return launch_wide<64, __nv_bfloat16>(g, pl, map, qmap, st);
  if (dtype == MK_F32) return launch_wide<128, float>(g, pl, map, qmap, st);
  return launch_wide<128, __nv_bfloat16>(g, pl, map, qmap, st);
}

}  // namespace mk
