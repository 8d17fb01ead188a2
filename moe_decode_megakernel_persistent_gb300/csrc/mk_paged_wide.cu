// Attention over the 16-bit paged cache for many query columns (prompt chunks, batches of
// drafts) on the 5th-generation tensor cores (tcgen05).
//
//   S = Q K^T   128 columns x the 128 positions of a page, fp32 in TMEM
//   O += P V    P = 2^(c S - m) in bf16 over S's place in TMEM, V by positions
//
// K and V are operands as the tensor copies bring them.  A thread has a column (a TMEM lane):
// its maximum is its own and moves only when a score passes it by 2^8; then it rescales its
// sums, which the next product waits for.  An fp32 q is three bf16 parts, and so are its weights.
//
// Warps 4 TB: the columns.  One warp more looks up pages and issues the copies, another the
// products.  With two tiles a block (TB = 2) the tensor cores work on one tile while the
// columns of the other form weights; with one tile there are two places of scores, so that S of a step
// runs before the second product of the last.
//
// What a column does not see must not show in it, and 0 x NaN is NaN.  Rows of V behind the last
// position that the tile sees are set to 0 in shared memory.  Positions that only some
// columns see are searched for values that are no finite numbers; those are set to 0 too, and at the
// end given to the columns that see them.
//
// One warp decides the block's runs and hands them to the others with the lengths it saw, so that all
// agree should someone write the lengths while the call runs.
#include <algorithm>

#include "mk_paged_att.cuh"
#include "mk_tcgen05.cuh"

namespace mk {
namespace {

template <int HD, class T, int TB>
struct PWide {
  static constexpr bool F32 = std::is_same<T, float>::value;
  static constexpr int NG = HD / 64, CT = 128 * TB, SP = kPageTokens;
  static constexpr int P = F32 ? 3 : 1;             // bf16 parts of q, and of the weights
  static constexpr int NS = TB == 1 ? 2 : 1;        // places of scores of a tile
  static constexpr int QT = NG * 128 * 128;         // bytes of a tile's q of one part
  static constexpr int QB = TB * P * QT;
  static constexpr int KVB = NG * SP * 128;         // of a page's K, or V, of a head
  static constexpr int ROOM = (226 * 1024 - QB) / KVB;
  static constexpr int STAGES = ROOM < 6 ? ROOM : 6;
  static constexpr int SMEM = 1024 + QB + STAGES * KVB;
  // TMEM columns of a tile: scores [NS][128], sums [HD], and with three parts the third of the weights [NS][64]
  static constexpr int SUMS = NS * 128, THIRD = SUMS + 128;
  static constexpr int TM = TB == 2 ? 256 : 512;    // of a tile
  static constexpr int CW = 4 * TB;                 // warps of the columns
  static constexpr int THREADS = 32 * (CW + 2);
};

// What the copying warp says of a run (t1 = t0: there is none more).
struct RunSays {
  int e, head, nt, t0, t1, len, nn;
  long long base;
};
constexpr int kRuns = 8;  // the copying warp is at most five runs ahead of the columns

template <int HD, class T, int TB>
__global__ void __launch_bounds__(PWide<HD, T, TB>::THREADS, 1) k_paged_wide(const __grid_constant__ PagedAtt pa, const __grid_constant__ CUtensorMap map) {
  using W = PWide<HD, T, TB>;
  constexpr int NG = W::NG, CT = W::CT, SP = W::SP, NS = W::NS, CW = W::CW, ST = W::STAGES;
  const AttArgs& p = pa.t;
  extern __shared__ uint8_t sm_raw[];
  uint8_t* sm = sm_raw + ((1024 - (smem_addr(sm_raw) & 1023)) & 1023);
  __shared__ __align__(8) uint64_t kv_full[ST], kv_empty[ST], s_full[TB][NS], p_full[TB][NS], pv_done[TB], q_full, run_full[kRuns], o_full, drain;
  __shared__ RunSays says[kRuns];
  __shared__ int odd[2];  // a run's V had values that are no finite numbers where columns differ
  __shared__ uint32_t tm_base;
  __shared__ volatile int give_up;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  uint8_t* q_op = sm;            // [tile][part][NG][128][128 bytes]
  uint8_t* kv_op = sm + W::QB;   // [stage][NG][128][128 bytes]
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    auto init = [](uint64_t* b, int n) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(b)), "r"(n) : "memory");
    };
    for (int i = 0; i < ST; ++i) init(&kv_full[i], 1), init(&kv_empty[i], 1);
    for (int t = 0; t < TB; ++t) {
      for (int i = 0; i < NS; ++i) {
        init(&s_full[t][i], 1);
        init(&p_full[t][i], 4);  // by each of the tile's warps (of which one may be a place of scores ahead)
      }
      init(&pv_done[t], 1);
    }
    init(&q_full, CW);
    for (int i = 0; i < kRuns; ++i) init(&run_full[i], 1);
    init(&o_full, 1);
    init(&drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    give_up = 0;
    odd[0] = odd[1] = 0;
  }
  if (w == CW + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tm_base)), "n"(W::TM * TB)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  before_sync();
  __syncthreads();
  after_sync();
  const uint32_t tm = tm_base;
  // A run as the other warps take it; false: there is none more.
  auto take_run = [&](uint32_t i, RunSays& rs) {
    if (!bar_wait(smem_addr(&run_full[i % kRuns]), (i / kRuns) & 1, &give_up, p.a.status)) return false;
    rs = says[i % kRuns];
    return rs.t1 > rs.t0;
  };

  if (w == CW) {  // ---- runs, pages and copies
    Runs r = first_run(p, CT, SP, lane);
    uint32_t slot = 0, n_runs = 0;
    bool more = r.t1 > r.t0;
    // K (kv = 0) or V of the run's step; false: the wait for its stage ran out
    auto copy = [&](int row, int kv) {
      const int st = slot % ST;
      const bool ok = slot < ST || bar_wait(smem_addr(&kv_empty[st]), (slot / ST - 1) & 1, &give_up, p.a.status);
      if (ok && lane == 0) {
        const uint32_t bar = smem_addr(&kv_full[st]);
        expect(bar, W::KVB);
        // (behind the pool's rows: zeros)
        tma_rows(smem_addr(kv_op + st * W::KVB), &map,
                 row < 0 ? p.a.n_pages * 2 * p.a.n_kv_heads * kPageTokens : row + kv * p.a.n_kv_heads * kPageTokens, bar);
      }
      __syncwarp();
      if (ok) ++slot;
      return ok;
    };
    while (__shfl_sync(0xffffffffu, more, 0) && !give_up) {
      const int e = __shfl_sync(0xffffffffu, r.e, 0), head = __shfl_sync(0xffffffffu, r.head, 0);
      const int t0 = __shfl_sync(0xffffffffu, r.t0, 0), t1 = __shfl_sync(0xffffffffu, r.t1, 0);
      const int seq = p.n_ctiles == 1 ? e : e / p.n_ctiles;
      if (lane == 0) {
        RunSays& rs = says[n_runs % kRuns];
        seq_extent(p.a, seq, rs.len, rs.nn);
        rs.e = e;
        rs.head = head;
        rs.nt = r.nt;
        rs.t0 = t0;
        rs.t1 = t1;
        rs.base = r.base;
        arrive(smem_addr(&run_full[n_runs % kRuns]));
      }
      ++n_runs;
      // rows of the next 32 steps' K, one in each lane; K is NS steps ahead of V
      int rows = -1, rows_k = -1;
      auto look_up = [&](int t) {
        const int pg = t + lane < t1 ? page_of(p.a, seq, (t + lane) * SP) : -1;
        return pg < 0 ? -1 : paged_row(p.a, pg, 0, head, 0);
      };
      bool ok = true;
      rows = rows_k = look_up(t0);
      for (int i = 0; i < NS && t0 + i < t1 && ok; ++i) ok = copy(__shfl_sync(0xffffffffu, rows_k, i), 0);
      for (int t = t0; t < t1 && ok; ++t) {
        const int i = t - t0, ik = i + NS;
        if (i && i % 32 == 0) rows = look_up(t);
        ok = copy(__shfl_sync(0xffffffffu, rows, i & 31), 1);
        if (ok && t0 + ik < t1) {
          if (ik % 32 == 0) rows_k = look_up(t0 + ik);
          ok = copy(__shfl_sync(0xffffffffu, rows_k, ik & 31), 0);
        }
      }
      more = ok && r.next(p, CT, SP);
    }
    if (lane == 0) {
      RunSays& rs = says[n_runs % kRuns];
      rs.t0 = rs.t1 = 0;
      arrive(smem_addr(&run_full[n_runs % kRuns]));
    }
    if (give_up && lane == 0) {  // copies in flight land before the block ends
      int none = 0;
      for (uint32_t i = slot > ST ? slot - ST : 0; i < slot; ++i) bar_wait_long(smem_addr(&kv_full[i % ST]), (i / ST) & 1, &none, nullptr);
    }
  } else if (w == CW + 1) {  // ---- the products
    constexpr uint32_t id_qk = (1u << 4) | (1u << 7) | (1u << 10) | ((SP >> 3) << 17) | ((128 >> 4) << 24);               // bf16, fp32 sums
    constexpr uint32_t id_pv = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((HD >> 3) << 17) | ((128 >> 4) << 24);  // V by rows
    uint32_t slot = 0, k = 0;  // stages and steps taken
    RunSays rs;
    auto arrived = [&](uint32_t s) { return bar_wait(smem_addr(&kv_full[s % ST]), (s / ST) & 1, &give_up, p.a.status); };
    auto scores = [&](int tile, uint32_t step, uint32_t s) {  // lane 0: of the step into its place
      const uint32_t to = tm + W::TM * tile + 128 * (step % NS);
      const uint64_t kd = operand(smem_addr(kv_op + s % ST * W::KVB));
#pragma unroll
      for (int x = W::P - 1; x >= 0; --x) {  // q's low parts first
        const uint64_t q = operand(smem_addr(q_op + (tile * W::P + x) * W::QT));
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t qa = q + ((g * 128 * 128 + kk * 32) >> 4), kb = kd + ((g * SP * 128 + kk * 32) >> 4);
            if (g == 0 && kk == 0 && x == W::P - 1) mma_ss<false>(to, qa, kb, id_qk);
            else mma_ss<true>(to, qa, kb, id_qk);
          }
      }
      commit(smem_addr(&s_full[tile][step % NS]));
    };
    for (uint32_t n_runs = 0; take_run(n_runs, rs); ++n_runs) {
      const int n = rs.t1 - rs.t0, seq = p.n_ctiles == 1 ? rs.e : rs.e / p.n_ctiles, j = rs.e - seq * p.n_ctiles;
      const int last = min(row_of(p, min((j + 1) * CT, p.cols) - 1), rs.nn - 1);
      const int end = rs.len - rs.nn + last + 1;                                    // what some column sees
      const int common = max(0, rs.len - rs.nn + row_of(p, j * CT) + 1);            // what all columns (with a row) do
      if (lane == 0) odd[n_runs & 1] = 0;
      bool ok = bar_wait(smem_addr(&q_full), n_runs & 1, &give_up, p.a.status);
      for (int i = 0; i < NS && i < n; ++i, ++slot) {
        ok = arrived(slot) && ok;
        after_sync();
        if (lane == 0 && ok && !give_up) {
#pragma unroll
          for (int t = 0; t < TB; ++t) scores(t, k + i, slot);
          commit(smem_addr(&kv_empty[slot % ST]));
        }
        __syncwarp();
      }
      for (int i = 0; i < n; ++i, ++k) {
        const uint32_t v = slot++, kn = slot;
        const bool next = i + NS < n;
        if (next) ++slot;
        ok = arrived(v) && ok;
        const int have = end - (rs.t0 + i) * SP;
        const int from = max(common - (rs.t0 + i) * SP, 0);
        if (ok && (have < SP || from < SP)) {
          uint8_t* vb = kv_op + v % ST * W::KVB;
          // words of 16 bytes of the rows a .. b: f(word) where it is to be written
          auto each = [&](int a, int b, auto f) {
            for (int x = a * NG * 8 + lane; x < b * NG * 8; x += 32)
              f(*reinterpret_cast<uint4*>(vb + (x / 8 % NG) * SP * 128 + x / (8 * NG) * 128 + x % 8 * 16));
          };
          each(max(have, 0), SP, [](uint4& x) { x = make_uint4(0, 0, 0, 0); });
          uint32_t any = 0;
          each(from, min(have, SP), [&](uint4& x) { any |= odd_ones(x.x) | odd_ones(x.y) | odd_ones(x.z) | odd_ones(x.w); });
          if (__any_sync(0xffffffffu, any)) {
            auto clear = [](uint32_t& x) {
              const uint32_t bad = odd_ones(x);
              x &= ~((bad >> 15 & 1u) * 0xFFFFu | (bad >> 31) * 0xFFFF0000u);
            };
            each(from, min(have, SP), [&](uint4& x) { clear(x.x), clear(x.y), clear(x.z), clear(x.w); });
            if (lane == 0) odd[n_runs & 1] = 1;
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
        const uint64_t vd = operand(smem_addr(kv_op + v % ST * W::KVB), SP * 128);
#pragma unroll
        for (int t = 0; t < TB; ++t) {
          ok = bar_wait(smem_addr(&p_full[t][k % NS]), (k / NS) & 1, &give_up, p.a.status) && ok;
          after_sync();
          if (lane == 0 && ok && !give_up) {
            const uint32_t base = tm + W::TM * t, to = base + W::SUMS;
#pragma unroll
            for (int x = W::P - 1; x >= 0; --x) {  // the weights' low parts first
              const uint32_t pw = x < 2 ? base + 128 * (k % NS) + 64 * x : base + W::THIRD + 64 * (k % NS);
#pragma unroll
              for (int kk = 0; kk < SP / 16; ++kk)
                mma_ts(to, pw + 8 * kk, vd + ((kk * 16 * 128) >> 4), id_pv, kk || x < W::P - 1 || i ? 1 : 0);
            }
            commit(smem_addr(&pv_done[t]));
          }
          __syncwarp();
          if (next) {
            if (t == 0) ok = arrived(kn) && ok;
            if (lane == 0 && ok && !give_up) {
              scores(t, k + NS, kn);
              if (t == TB - 1) commit(smem_addr(&kv_empty[kn % ST]));
            }
          }
          if (t == TB - 1 && lane == 0 && ok && !give_up) commit(smem_addr(&kv_empty[v % ST]));
          __syncwarp();
        }
      }
      if (lane == 0) arrive(smem_addr(&o_full));
      if (!ok || give_up) break;
    }
    if (give_up) {  // products in flight end before the block does
      int none = 0;
      if (lane == 0) commit(smem_addr(&drain));
      bar_wait_long(smem_addr(&drain), 0, &none, nullptr);
    }
  } else if (w < CW) {  // ---- a query column each
    const int tile = w >> 2, tt = tid & 127;
    // this warp's lanes of its tile's scores and sums
    const uint32_t tm_s = tm + W::TM * tile + ((uint32_t)(32 * (w & 3)) << 16), tm_o = tm_s + W::SUMS;
    uint32_t k = 0;
    RunSays rs;
    const float cf = fabsf(p.c);
    for (uint32_t n_runs = 0; take_run(n_runs, rs); ++n_runs) {
      const int seq = p.n_ctiles == 1 ? rs.e : rs.e / p.n_ctiles, j = rs.e - seq * p.n_ctiles;
      const int col = j * CT + tid;
      const bool there = col < p.cols;
      const int row = there ? row_of(p, col) : 0, hd = rs.head * p.gqa + (there ? col - row * p.gqa : 0);
      const int lim = there && row < rs.nn ? max(0, rs.len - rs.nn + row + 1) : 0;  // positions that it sees
      {
        const T* src = reinterpret_cast<const T*>(p.q.p) + seq * p.q.seq + row * p.q.row + hd * p.q.head;
        const uint32_t flip = p.c < 0.f ? 0x80008000u : 0u;  // a negative scale goes into q
#pragma unroll
        for (int x = 0; x < HD / 8; ++x) {
          uint8_t* to = q_op + tile * W::P * W::QT + x / 8 * 128 * 128 + tt * 128 + (((x % 8) ^ (tt & 7)) << 4);
          if constexpr (W::F32) {
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
            if (lim) {
              a = __ldg(reinterpret_cast<const float4*>(src + 8 * x));
              b = __ldg(reinterpret_cast<const float4*>(src + 8 * x + 4));
            }
            const Parts y[8] = {parts_of(a.x), parts_of(a.y), parts_of(a.z), parts_of(a.w), parts_of(b.x), parts_of(b.y), parts_of(b.z), parts_of(b.w)};
#pragma unroll
            for (int i = 0; i < 3; ++i)
              *reinterpret_cast<uint4*>(to + i * W::QT) = make_uint4(both(y[0], y[1], i) ^ flip, both(y[2], y[3], i) ^ flip,
                                                                     both(y[4], y[5], i) ^ flip, both(y[6], y[7], i) ^ flip);
          } else {
            uint4 h = lim ? __ldg(reinterpret_cast<const uint4*>(src + 8 * x)) : make_uint4(0, 0, 0, 0);
            h.x ^= flip, h.y ^= flip, h.z ^= flip, h.w ^= flip;
            *reinterpret_cast<uint4*>(to) = h;
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive(smem_addr(&q_full));
      const int32_t* pages = table_row(p.a, seq);
      int page = pages[rs.t0];
      float m = kLow, l = 0.f;  // running maximum (log2) and the sum of the weights
      for (int t = rs.t0; t < rs.t1; ++t, ++k) {
        const bool in = page >= 0 && page < p.a.n_pages;
        if (t + 1 < rs.t1) page = pages[t + 1];
        const bool ok = bar_wait(smem_addr(&s_full[tile][k % NS]), (k / NS) & 1, &give_up, p.a.status);
        after_sync();
        if (ok && !give_up) {
          const int vis = in ? lim - t * SP : 0;  // of the step's positions
          const uint32_t at = tm_s + 128 * (k % NS);
          auto step = [&](auto cut_) {
            constexpr bool CUT = decltype(cut_)::value;
            float s[4][32], mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              tm_read32(at + 32 * c, s[c]);
#pragma unroll
              for (int x = 0; x < 32; ++x) {
                if (CUT && 32 * c + x >= vis) s[c][x] = -INFINITY;
                mx[x & 3] = fmaxf(mx[x & 3], s[c][x]);
              }
            }
            float most = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            most = most == -INFINITY ? most : most * cf;
            if (__any_sync(0xffffffffu, most > m + kLazy)) {
              const float nm = fmaxf(m, most), f = exp2_fast(m - nm);
              m = nm;
              l *= f;
              if (t > rs.t0) {
                bar_wait(smem_addr(&pv_done[tile]), (k - 1) & 1, &give_up, p.a.status);  // the sums hold the last step
                after_sync();
#pragma unroll 1
                for (int c = 0; c < HD; c += 16) {
                  float o[16];
                  uint32_t x16[16];
                  tm_read16(tm_o + c, o);
#pragma unroll
                  for (int x = 0; x < 16; ++x) x16[x] = __float_as_uint(o[x] * f);
                  tm_store16(tm_o + c, x16);
                }
              }
            }
            float la[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t b[W::P][16];
#pragma unroll
              for (int x = 0; x < 32; x += 2) {
                float w2[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const float z = s[c][x + y];
                  w2[y] = CUT && z == -INFINITY ? 0.f : exp2_fast(fmaf(z, cf, -m));
                  la[(x + y) & 3] += w2[y];
                }
#pragma unroll
                for (int i = 0; i < W::P; ++i) {
                  b[i][x / 2] = pack2(w2[0], w2[1]);
                  if (i + 1 < W::P) w2[0] -= low_f(b[i][x / 2]), w2[1] -= high_f(b[i][x / 2]);
                }
              }
              tm_store16(at + 16 * c, b[0]);  // over the scores, which are all in registers
              if constexpr (W::P == 3) {
                tm_store16(at + 64 + 16 * c, b[1]);
                tm_store16(tm_s + W::THIRD + 64 * (k % NS) + 16 * c, b[2]);
              }
            }
            l += (la[0] + la[1]) + (la[2] + la[3]);
          };
          if (__all_sync(0xffffffffu, vis >= SP)) step(std::false_type());
          else step(std::true_type());
          tm_stored();
        }
        before_sync();
        __syncwarp();
        if (lane == 0) arrive(smem_addr(&p_full[tile][k % NS]));
      }
      // ---- the run's end: this column's sums
      bool ok = bar_wait(smem_addr(&pv_done[tile]), (k - 1) & 1, &give_up, p.a.status);
      ok = bar_wait(smem_addr(&o_full), n_runs & 1, &give_up, p.a.status) && ok && !give_up;
      after_sync();
      const bool whole = rs.t0 == 0 && rs.t1 == rs.nt;
      const float f = whole ? 1.f / l : 1.f;
      const bool look = odd[n_runs & 1];
      float* part = p.part + ((size_t)part_slot(blockIdx.x, rs.t0) * CT + tid) * (HD + 4);
      T* dst = reinterpret_cast<T*>(const_cast<void*>(p.out.p)) + seq * p.out.seq + row * p.out.row + hd * p.out.head;
#pragma unroll 1
      for (int c = 0; c < HD; c += 16) {
        float o[16];
        tm_read16(tm_o + c, o);
        bool fine = !look;
#pragma unroll
        for (int x = 0; x < 16; ++x) fine = fine && is_finite(o[x]);
        if (!fine && lim && is_finite(l)) {  // (positions that all columns see went through the products as they are)
#pragma unroll
          for (int x = 0; x < 16; x += 2) {
            const float2 s = odd_sum<HD>(p.a, seq, rs.head, c + x, rs.t0 * SP, min(lim, rs.t1 * SP));
            if (s.x != 0.f) o[x] = s.x;
            if (s.y != 0.f) o[x + 1] = s.y;
          }
        }
        if (!there) continue;
#pragma unroll
        for (int x = 0; x < 16; ++x) o[x] = !ok ? NAN : l == 0.f ? 0.f : o[x] * f;
        if (whole && !W::F32) {
#pragma unroll
          for (int x = 0; x < 16; x += 8)
            *reinterpret_cast<uint4*>(dst + c + x) =
                make_uint4(pack2(o[x], o[x + 1]), pack2(o[x + 2], o[x + 3]), pack2(o[x + 4], o[x + 5]), pack2(o[x + 6], o[x + 7]));
        } else {
          float* to = whole ? reinterpret_cast<float*>(dst) : part;
#pragma unroll
          for (int x = 0; x < 16; x += 4) *reinterpret_cast<float4*>(to + c + x) = make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
        }
      }
      if (there) {
        if (!whole) *reinterpret_cast<float2*>(part + HD) = l == 0.f ? make_float2(kLow, 0.f) : make_float2(m, ok ? l : NAN);
        else if (p.lse)
          p.lse[((size_t)seq * p.a.rows + row) * p.n_heads + hd] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
      }
      if (tid == 0 && rs.t0 == 0)
        p.item[(size_t)rs.e * p.a.n_kv_heads + rs.head] =
            make_longlong2(whole ? -1 : rs.base + (long long)rs.head * (rs.nt + kOver), blockIdx.x);
      before_sync();  // the next run's products overwrite the sums
      if (!ok) break;
    }
  }
  before_sync();
  __syncthreads();
  if (w == CW + 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "n"(W::TM * TB));
}

template <int HD, class T, int TB>
WideKernel info() {
  using W = PWide<HD, T, TB>;
  return {reinterpret_cast<const void*>(&k_paged_wide<HD, T, TB>), W::CT, W::SP, W::SMEM, 1, W::THREADS};
}

}  // namespace

WideKernel paged_wide_kernel(int head_dim, int dtype, int cols) {
  if (dtype == MK_F32) return head_dim == 64 ? info<64, float, 1>() : info<128, float, 1>();
  if (cols <= 128) return head_dim == 64 ? info<64, __nv_bfloat16, 1>() : info<128, __nv_bfloat16, 1>();
  return head_dim == 64 ? info<64, __nv_bfloat16, 2>() : info<128, __nv_bfloat16, 2>();
}

}  // namespace mk
