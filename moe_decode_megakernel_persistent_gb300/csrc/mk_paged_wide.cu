// Attention over the 16-bit paged cache for many query columns (prompt chunks, batches of
// drafts) on the 5th-generation tensor cores (tcgen05).
//
//   S = Q K^T   128 columns x the 128 positions of a page, fp32 in TMEM
//   O += P V    P = 2^(c S - m) in bf16 parts over S's place in TMEM, V by positions
//
// K and V are operands as the tensor copies bring them.  A thread has a column (a TMEM lane):
// its maximum is its own and moves only when a score passes it by 2^8; then it rescales its
// sums, which the next product waits for.  An fp32 q is three bf16 parts, and so are its weights; a bf16 one's
// are two (one part, 2^-8, took 11 us less of the 85 below, and left an error of 0.0026 of the outputs' size for 0.0017).
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
// Bounds.  1024 rows of 16 heads over 8022 positions (4 kv heads of 128) are 49 us of products at the measured
// rate (33 with weights of one part); the call takes 85, of which the join is about 12.  Bytes (3 % of the memory's) do
// not bound it, nor do the tensor cores alone (50 % active): a step of two tiles and 128 positions takes about 4,900 cycles, of
// which the products are 3,072; the columns' reads from TMEM, maxima, exponentials (32 a cycle and SM: 1,024) and writes do
// not hide wholly behind the other tile's products.  fp32 rows (three sequences of up to 2049 positions, 641 rows) do the products of
// three parts, 26 us, in 94 with the join's 12, of which handing the sums over every second step is about 15.
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
  static constexpr int P = F32 ? 3 : 1;             // bf16 parts of q
  static constexpr int WP = F32 ? 3 : 2;            // and of the weights
  static constexpr int NS = TB == 1 ? 2 : 1;        // places of scores of a tile
  static constexpr int GR = NS;                     // groups of four warps of a tile, which take the steps in turn
  static constexpr int QT = NG * 128 * 128;         // bytes of a tile's q of one part
  static constexpr int QB = TB * P * QT;
  static constexpr int KVB = NG * SP * 128;         // of a page's K, or V, of a head
  static constexpr int EX = GR > 1 ? 3 * CT * 4 : 0;  // what the groups tell each other: maxima, two sums
  // What 227 KB hold beside the barriers and the like, of which fp32 rows of 128 dimensions leave 512 bytes.
  static constexpr int ROOM = (227 * 1024 - 1024 - (F32 && HD == 128 ? 512 : 1024) - QB - EX) / KVB;
  static constexpr int STAGES = ROOM < 6 ? ROOM : 6;
  static constexpr int SMEM = 1024 + QB + STAGES * KVB + EX;
  // TMEM columns of a tile: scores [NS][128], sums [HD], and with three parts the third of the weights [NS][64]
  static constexpr int SUMS = NS * 128, THIRD = SUMS + 128;
  static constexpr int TM = TB == 2 ? 256 : 512;    // of a tile
  // The products cut off what they add, about 2^-24 of the sum each time and always towards 0: after so many steps the
  // sums of fp32 rows are added, rounded, to others that the columns hold (even: the same group's step begins new
  // sums throughout a run).  Three sequences of 700 to 2049 positions, 641 rows: 2 steps are 8.2e-7 off (the same sums by fp32
  // products 7.9e-7) in 94 us; when that was 90, 4 steps were 1.3e-6 off in 79 and 8 steps 1.9e-6 in 74.
  // Of bf16 rows every 4096 positions: with V of one sign, 131072 in one sum left outputs 9.2e-4 too small, where their own
  // rounding is 2^-9 to 2^-8 (1024 rows at 8022 positions 83.3 us without, 85.0 with).
  static constexpr int FLUSH = F32 ? 2 : 32;
  static constexpr int DIMS = HD / GR;              // of a thread's sums
  static constexpr int CW = 4 * TB * GR;            // warps of the columns: eight
  static constexpr int THREADS = 32 * (CW + 2);
};

// What the copying warp says of a run (t1 = t0: there is none more).
struct RunSays {
  int e, head, nt, t0, t1, len, nn;
  long long base;
};
constexpr int kRuns = 5;  // the copying warp is at most four runs ahead of the columns

template <int HD, class T, int TB>
__global__ void __launch_bounds__(PWide<HD, T, TB>::THREADS, 1) k_paged_wide(const __grid_constant__ PagedAtt pa, const __grid_constant__ CUtensorMap map) {
  using W = PWide<HD, T, TB>;
  constexpr int NG = W::NG, CT = W::CT, SP = W::SP, NS = W::NS, GR = W::GR, CW = W::CW, ST = W::STAGES;
  const AttArgs& p = pa.t;
  extern __shared__ uint8_t sm_raw[];
  uint8_t* sm = sm_raw + ((1024 - (smem_addr(sm_raw) & 1023)) & 1023);
  __shared__ __align__(8) uint64_t kv_full[ST], kv_empty[ST], s_full[TB][NS], p_full[TB][NS][2], pv_done, run_done[TB], q_full, run_full[kRuns], o_full, m_full[GR][4], l_full, sums_done, flushed, out_done, drain;
  __shared__ RunSays says[kRuns];
  __shared__ int odd[2];  // a run's V had values that are no finite numbers where columns differ
  __shared__ uint32_t tm_base;
  __shared__ volatile int give_up;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  uint8_t* q_op = sm;            // [tile][part][NG][128][128 bytes]
  uint8_t* kv_op = sm + W::QB;   // [stage][NG][128][128 bytes]
  if (tid == 0) {
    auto init = [](uint64_t* b, int n) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(b)), "r"(n) : "memory");
    };
    for (int i = 0; i < ST; ++i) init(&kv_full[i], 1), init(&kv_empty[i], 1);
    for (int t = 0; t < TB; ++t) {
      for (int i = 0; i < NS; ++i) {
        init(&s_full[t][i], 1);
        for (int h = 0; h < 2; ++h) init(&p_full[t][i][h], 4);  // by each of the tile's warps (of which one may be a place of scores ahead)
      }
      init(&run_done[t], 1);
    }
    init(&pv_done, 1);
    for (int i = 0; i < 4 * GR; ++i) init(&m_full[i >> 2][i & 3], 1);
    init(&l_full, CW);
    init(&out_done, CW);
    init(&sums_done, 1);
    init(&flushed, CW);
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
  behind();
  // A run as the other warps take it; false: there is none more.
  auto take_run = [&](uint32_t i, RunSays& rs) {
    if (!wait_for(smem_addr(&run_full[i % kRuns]), (i / kRuns) & 1, &give_up, p.a.status)) return false;
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
      const bool ok = slot < ST || wait_for(smem_addr(&kv_empty[st]), (slot / ST - 1) & 1, &give_up, p.a.status);
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
      for (uint32_t i = slot > ST ? slot - ST : 0; i < slot; ++i) wait_for(smem_addr(&kv_full[i % ST]), (i / ST) & 1, &none, nullptr);
    }
  } else if (w == CW + 1) {  // ---- the products
    constexpr uint32_t id_qk = (1u << 4) | (1u << 7) | (1u << 10) | ((SP >> 3) << 17) | ((128 >> 4) << 24);               // bf16, fp32 sums
    constexpr uint32_t id_pv = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((HD >> 3) << 17) | ((128 >> 4) << 24);  // V by rows
    const uint32_t tmu = uniform(tm), qu = uniform(smem_addr(q_op)), kvu = uniform(smem_addr(kv_op));
    uint32_t st = 0, round = 0, k = 0;  // the next stage and its phase, steps taken
    uint32_t n_flush = 0;
    RunSays rs;
    bool ok = true;
    // the next stage, once it has arrived
    auto arrived = [&]() {
      ok = wait_for(smem_addr(&kv_full[st]), round, &give_up, p.a.status) && ok;
      const uint32_t got = uniform(st);
      if (++st == ST) st = 0, round ^= 1;
      return got;
    };
    auto scores = [&](int tile, uint32_t place, uint32_t stage) {  // one lane: of a tile into its place
      const uint32_t to = tmu + W::TM * tile + 128 * place;
      const uint64_t kd = operand(kvu + stage * W::KVB);
#pragma unroll
      for (int x = W::P - 1; x >= 0; --x) {  // q's low parts first
        const uint64_t q = operand(qu + (tile * W::P + x) * W::QT);
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t qa = q + ((g * 128 * 128 + kk * 32) >> 4), kb = kd + ((g * SP * 128 + kk * 32) >> 4);
            if (g == 0 && kk == 0 && x == W::P - 1) mma_ss<false>(to, qa, kb, id_qk);
            else mma_ss<true>(to, qa, kb, id_qk);
          }
      }
      commit(smem_addr(&s_full[tile][place]));
      if (tile == TB - 1) commit(smem_addr(&kv_empty[stage]));
    };
    for (uint32_t n_runs = 0; take_run(n_runs, rs); ++n_runs) {
      const int n = rs.t1 - rs.t0, seq = p.n_ctiles == 1 ? rs.e : rs.e / p.n_ctiles, j = rs.e - seq * p.n_ctiles;
      const int last = min(row_of(p, min((j + 1) * CT, p.cols) - 1), rs.nn - 1);
      const int end = rs.len - rs.nn + last + 1;                                    // what some column sees
      const int common = max(0, rs.len - rs.nn + row_of(p, j * CT) + 1);            // what all columns (with a row) do
      ok = wait_for(smem_addr(&q_full), n_runs & 1, &give_up, p.a.status) && ok;
      if (lane == 0) odd[(n_runs + 1) & 1] = 0;  // which the columns have read: the next run's
      for (int i = 0; i < NS && i < n; ++i) {
        const uint32_t su = arrived(), pu = uniform((k + i) % NS);
        after_sync();
        if (ok && elect_one()) {
#pragma unroll
          for (int t = 0; t < TB; ++t) scores(t, pu, su);
        }
        __syncwarp();
      }
      // V of a step in its stage, with zeros where no column sees it and for what is no finite number where columns differ
      auto clean = [&](int i, uint32_t v) {
        const int have = end - (rs.t0 + i) * SP;
        const int from = max(common - (rs.t0 + i) * SP, 0);
        if (!ok || (have >= SP && from >= SP)) return;
        uint8_t* vb = kv_op + v * W::KVB;
        // words of 16 bytes of the rows a .. b: f(word) where it is to be written
        auto each = [&](int a, int b, auto f) {
#pragma unroll 4
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
      };
      uint32_t v = arrived(), kn = NS < n ? arrived() : 0;
      clean(0, v);
      for (int i = 0; i < n; ++i, ++k) {
        const uint32_t pu = uniform(k % NS), add = uniform(i % W::FLUSH != 0), nu = uniform(i + NS < n), lu = uniform(i + 1 == n);
        const uint32_t last = uniform(i + 1 < n && (i + 1) % W::FLUSH == 0);  // of these sums
        const uint64_t vd = operand(kvu + v * W::KVB, SP * 128);
        uint32_t vn = 0, kn2 = 0;
        if (i && i % W::FLUSH == 0) ok = wait_for(smem_addr(&flushed), n_flush++ & 1, &give_up, p.a.status) && ok;  // the sums are read
#pragma unroll
        for (int t = 0; t < TB; ++t) {
          // the weights come in halves of 64 positions
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            ok = wait_for(smem_addr(&p_full[t][pu][h]), (k / NS) & 1, &give_up, p.a.status) && ok;
            after_sync();
            if (ok && elect_one()) {
              const uint32_t base = tmu + W::TM * t;
#pragma unroll
              for (int x = W::WP - 1; x >= 0; --x) {  // the weights' low parts first
#pragma unroll
                for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
                  mma_ts(base + W::SUMS, x < 2 ? base + 128 * pu + 32 * (kk / 2) + 16 * x + 8 * (kk % 2) : base + W::THIRD + 64 * pu + 8 * kk, vd + ((kk * 16 * 128) >> 4), id_pv, kk || x < W::WP - 1 ? 1 : add);
              }
              if (h) {
                if (t == TB - 1) commit(smem_addr(&kv_empty[v]));
                if (NS > 1) commit(smem_addr(&pv_done));
                if (t == TB - 1 && last) commit(smem_addr(&sums_done));
                if (lu) commit(smem_addr(&run_done[t]));
                if (nu) scores(t, pu, kn);
              }
            }
            __syncwarp();
            // The next step's operands are waited for behind products: the queue holds a few of them, and
            // what takes longer between two groups leaves the tensor cores idle.
            if (t == 0 && h == 0 && i + 1 < n) {
              vn = arrived();
              clean(i + 1, vn);
            }
            if (t == TB - 1 && h == (TB == 1) && i + 1 + NS < n) kn2 = arrived();
          }
        }
        v = vn;
        kn = kn2;
      }
      if (lane == 0) arrive(smem_addr(&o_full));
      if (!ok || give_up) break;
    }
    if (give_up) {  // products in flight end before the block does
      int none = 0;
      if (lane == 0) commit(smem_addr(&drain));
      wait_for(smem_addr(&drain), 0, &none, nullptr);
    }
  } else if (w < CW) {  // ---- a query column each
    // With one tile a column has two threads, which take the steps in turn: a step's maximum passes
    // from one to the other before its exponentials, and each has the sum of its own steps' weights.
    const int tile = GR > 1 ? 0 : w >> 2, group = GR > 1 ? w >> 2 : 0, quarter = w & 3, me = GR > 1 ? tid & 127 : tid;
    // this warp's lanes of its tile's scores and sums
    const uint32_t tm_s = tm + W::TM * tile + ((uint32_t)(32 * quarter) << 16), tm_o = tm_s + W::SUMS;
    [[maybe_unused]] float* ex = reinterpret_cast<float*>(kv_op + ST * W::KVB);  // maxima [CT], sums [2][CT]
    uint32_t k = 0;
    uint32_t n_flush = 0;
    RunSays rs;
    const float cf = fabsf(p.c);
    // word x of row y of these lanes' part of the q operand, which also holds the sums on their way out
    auto place = [&](int y, int x) { return q_op + tile * W::P * W::QT + x / 8 * 128 * 128 + (32 * quarter + y) * 128 + (((x % 8) ^ (y & 7)) << 4); };
    for (uint32_t n_runs = 0; take_run(n_runs, rs); ++n_runs) {
      const int seq = p.n_ctiles == 1 ? rs.e : rs.e / p.n_ctiles, j = rs.e - seq * p.n_ctiles;
      const int col = j * CT + me;
      const bool there = col < p.cols;
      const int row = there ? row_of(p, col) : 0, hd = rs.head * p.gqa + (there ? col - row * p.gqa : 0);
      const int lim = there && row < rs.nn ? max(0, rs.len - rs.nn + row + 1) : 0;  // positions that it sees
      if constexpr (GR > 1)  // the other group's sums have left the place of q
        if (n_runs && !wait_for(smem_addr(&out_done), (n_runs - 1) & 1, &give_up, p.a.status)) break;
      {  // these lanes' 32 rows of q, a row after another, so that a warp reads them in one piece
        const uint32_t flip = p.c < 0.f ? 0x80008000u : 0u;  // a negative scale goes into q
        constexpr int ALL = NG * 8 / GR, AT = W::F32 ? 4 : ALL;  // reads, and reads in flight
        const int x = lane % (NG * 8);                           // 16-byte word of the operand
#pragma unroll 1
        for (int i0 = group * ALL; i0 < (group + 1) * ALL; i0 += AT) {
          uint4 h[AT][W::F32 ? 2 : 1];
          bool some[AT];
#pragma unroll
          for (int i = 0; i < AT; ++i) {
            // (a row that is none, or padding, reads another's and counts as 0; not by the read-only path, for the
            // kernel may begin while its predecessor writes q)
            const int c = col - lane + (32 * (i0 + i) + lane) / (NG * 8), cc = min(c, p.cols - 1), rw = row_of(p, cc);
            const T* src = reinterpret_cast<const T*>(p.q.p) + seq * p.q.seq + rw * p.q.row + (rs.head * p.gqa + cc - rw * p.gqa) * p.q.head + 8 * x;
            some[i] = c < p.cols && rw < rs.nn && rs.len - rs.nn + rw >= 0;
#pragma unroll
            for (int z = 0; z < (W::F32 ? 2 : 1); ++z) h[i][z] = __ldcg(reinterpret_cast<const uint4*>(src) + z);
          }
#pragma unroll
          for (int i = 0; i < AT; ++i) {
            uint8_t* to = place((32 * (i0 + i) + lane) / (NG * 8), x);
            if constexpr (W::F32) {
              const uint32_t u[8] = {h[i][0].x, h[i][0].y, h[i][0].z, h[i][0].w, h[i][1].x, h[i][1].y, h[i][1].z, h[i][1].w};
              Parts z[8];
#pragma unroll
              for (int y = 0; y < 8; ++y) z[y] = parts_of(some[i] ? __uint_as_float(u[y] ^ (flip & 0x80000000u)) : 0.f);
#pragma unroll
              for (int q = 0; q < 3; ++q)
                *reinterpret_cast<uint4*>(to + q * W::QT) = make_uint4(both(z[0], z[1], q), both(z[2], z[3], q), both(z[4], z[5], q), both(z[6], z[7], q));
            } else {
              uint4 v = h[i][0];
              v.x ^= flip, v.y ^= flip, v.z ^= flip, v.w ^= flip;
              *reinterpret_cast<uint4*>(to) = some[i] ? v : make_uint4(0, 0, 0, 0);
            }
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive(smem_addr(&q_full));
      const int32_t* pages = table_row(p.a, seq);
      const int skip = GR > 1 ? (k ^ group) & 1 : 0;  // the group's first step of the run
      int page = rs.t0 + skip < rs.t1 ? pages[rs.t0 + skip] : -1;
      float m = kLow, l = 0.f;  // running maximum (log2) that l is relative to, and the sum of the weights
      // sums of earlier steps of this thread's dimensions (in local memory), and the maximum they are relative to
      float held[W::DIMS], m_held = -INFINITY;  // (none yet)
      // the sums so far, relative to the maximum `now`, to those held
      auto flush = [&](float now) {
        wait_for(smem_addr(&sums_done), n_flush++ & 1, &give_up, p.a.status);
        after_sync();
        const float f = exp2_fast(m_held - now);
        constexpr int AT = W::F32 ? W::DIMS : 32;  // (of fp32 rows often: the products go on before the sums are added)
#pragma unroll 1
        for (int c0 = 0; c0 < W::DIMS; c0 += AT) {
          float o[AT];
#pragma unroll
          for (int c = 0; c < AT; c += 32) tm_read32(tm_o + group * W::DIMS + c0 + c, *reinterpret_cast<float(*)[32]>(o + c));
          if (c0 + AT == W::DIMS) {
            before_sync();
            __syncwarp();
            if (lane == 0) arrive(smem_addr(&flushed));
          }
#pragma unroll
          for (int c = 0; c < AT; ++c) held[c0 + c] = m_held == -INFINITY ? o[c] : fmaf(held[c0 + c], f, o[c]);
        }
        m_held = now;
      };
      for (int t = rs.t0 + skip;; t += GR) {
        const uint32_t kk = k + (t - rs.t0);
        {  // all groups, before the first step of new sums or the one behind it
          const int i = t - rs.t0, in = (int)((uint32_t)i % W::FLUSH);
          if (i >= W::FLUSH && in < GR && i - in < rs.t1 - rs.t0) {
            float now = m;
            if (GR > 1 && in == 0) {  // (the other group had the last step)
              wait_for(smem_addr(&m_full[group ^ 1][quarter]), ((kk - 1) >> 1) & 1, &give_up, p.a.status);
              now = *reinterpret_cast<volatile float*>(ex + me);
            }
            flush(now);
          }
        }
        if (t >= rs.t1) break;
        const bool in = page >= 0 && page < p.a.n_pages;
        if (t + GR < rs.t1) page = pages[t + GR];
        bool ok = wait_for(smem_addr(&s_full[tile][kk % NS]), (kk / NS) & 1, &give_up, p.a.status);
        after_sync();
        if (ok && !give_up) {
          const int vis = in ? lim - t * SP : 0;  // of the step's positions
          auto given = [&](int h) {  // half of the weights are in TMEM
            tm_stored();
            before_sync();
            __syncwarp();
            if (lane == 0) arrive(smem_addr(&p_full[tile][kk % NS][h]));
          };
          const uint32_t at = tm_s + 128 * (kk % NS);
          auto step = [&](auto cut_) {
            constexpr bool CUT = decltype(cut_)::value;
            // 32 scores at a time, once for the maximum and once for the exponentials: rolled loops, whose code stays in
            // the instruction cache (all 128 held in registers: bf16 75.4 us against 71.8, fp32 with its three parts 109 against 69)
            float s[32], mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            auto read = [&](int c, float (&z)[32]) {
              tm_read32(at + 32 * c, z);
              const int v = vis - 32 * c;
#pragma unroll
              for (int x = 0; x < 32; ++x)
                if (CUT && x >= v) z[x] = -INFINITY;
            };
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              read(c, s);
#pragma unroll
              for (int x = 0; x < 32; x += 2) mx[x / 2 & 3] = max3(mx[x / 2 & 3], s[x], s[x + 1]);
            }
            float most = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            most = most == -INFINITY ? most : most * cf;
            float last = m;  // the column's maximum so far, which the sums are relative to
            if constexpr (GR > 1) {
              last = kLow;
              if (t > rs.t0) {
                wait_for(smem_addr(&m_full[group ^ 1][quarter]), ((kk - 1) >> 1) & 1, &give_up, p.a.status);
                last = *reinterpret_cast<volatile float*>(ex + me);
              }
            }
            float now = last;
            const bool moves = __any_sync(0xffffffffu, most > last + kLazy);
            if (moves) now = fmaxf(last, most);
            if constexpr (GR > 1) {
              ex[me] = now;
              __syncwarp();
              if (lane == 0) arrive(smem_addr(&m_full[group][quarter]));
            }
            l *= exp2_fast(m - now);
            m = now;
            const bool fresh = (uint32_t)(t - rs.t0) % W::FLUSH == 0;  // the sums begin with this step
            if (moves && !fresh) {
              if constexpr (NS > 1) {  // the sums hold the last step (with one place of scores these have waited for it)
                wait_for(smem_addr(&pv_done), (kk - 1) & 1, &give_up, p.a.status);
                after_sync();
              }
              const float f = exp2_fast(last - now);
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
            const uint64_t cf2 = pair(cf, cf), sub2 = pair(-m, -m);
            uint64_t la[2] = {0, 0};
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t b[W::WP][16];
              read(c, s);
              const int v = vis - 32 * c;
#pragma unroll
              for (int x = 0; x < 32; x += 2) {
                float2 z = unpair(fma2(pair(s[x], s[x + 1]), cf2, sub2));
                z.x = exp2_fast(z.x), z.y = exp2_fast(z.y);
                if (CUT && x >= v) z.x = 0.f;
                if (CUT && x + 1 >= v) z.y = 0.f;
                la[x / 2 & 1] = add2(la[x / 2 & 1], pair(z.x, z.y));
#pragma unroll
                for (int i = 0; i < W::WP; ++i) {
                  b[i][x / 2] = pack2(z.x, z.y);
                  if (i + 1 < W::WP) z.x -= low_f(b[i][x / 2]), z.y -= high_f(b[i][x / 2]);
                }
              }
              // over these scores, which are in registers; the third part has a place of its own
              tm_store16(at + 32 * c, b[0]);
              tm_store16(at + 32 * c + 16, b[1]);
              if constexpr (W::WP == 3) {
                tm_store16(tm_s + W::THIRD + 64 * (kk % NS) + 16 * c, b[2]);
              }
              if (c == 1) given(0);
            }
            const float2 a = unpair(add2(la[0], la[1]));
            l += a.x + a.y;
          };
          if (__all_sync(0xffffffffu, vis >= SP)) step(std::false_type());
          else step(std::true_type());
          given(1);
        }
      }
      k += rs.t1 - rs.t0;
      // ---- the run's end: this column's sums
      bool ok = wait_for(smem_addr(&run_done[tile]), n_runs & 1, &give_up, p.a.status);
      ok = wait_for(smem_addr(&o_full), n_runs & 1, &give_up, p.a.status) && ok && !give_up;
      after_sync();
      if constexpr (GR > 1) {  // both threads' sums, relative to the last maximum
        const float now = ex[me];
        ex[CT * (1 + group) + me] = l * exp2_fast(m - now);
        m = now;
        __syncwarp();
        if (lane == 0) arrive(smem_addr(&l_full));
        ok = wait_for(smem_addr(&l_full), n_runs & 1, &give_up, p.a.status) && ok;
        l = ex[CT + me] + ex[2 * CT + me];
      }
      const bool whole = rs.t0 == 0 && rs.t1 == rs.nt;
      const float f = whole ? 1.f / l : 1.f;
      const bool none = l == 0.f && (whole || !lim);  // (of a part without a weight, infinities and NaN are the join's; the rest is 0)
      const bool look = odd[n_runs & 1];
      float* part = p.part + ((size_t)part_slot(blockIdx.x, rs.t0) * CT + me) * (HD + 4);
      // Through the operand's place in shared memory, so that a warp writes its rows in one piece
      // each (the columns' own rows, 16 bytes a lane, took 11,000 cycles).  A group takes its half of the dimensions
      // in words of its own: of another part of q, or its half of a row's.
      auto leave = [&](auto wide_) {
        constexpr bool F = decltype(wide_)::value;                                    // fp32 words
        constexpr int WORDS = GR > 1 && W::P == 1 ? NG * 4 : NG * 8;                  // 16-byte words of a row
        constexpr int DP = WORDS * (F ? 4 : 8), CH = DP < 32 ? DP : 32;               // dimensions of a pass, of a read
        const int w0 = GR > 1 && W::P == 1 ? group * WORDS : 0, part0 = GR > 1 && W::P == 3 ? group * W::QT : 0;
        Odd<HD> search;
        bool searched = false;
#pragma unroll 1
        for (int c0 = group * (HD / GR); c0 < (group + 1) * (HD / GR); c0 += DP) {
#pragma unroll 1
          for (int c = c0; c < c0 + DP; c += CH) {
            float o[CH], top = 0.f;
            if constexpr (CH == 32) tm_read32(tm_o + c, o);
            else tm_read16(tm_o + c, o);
            if (m_held != -INFINITY) {
              const float g = exp2_fast(m_held - m);
#pragma unroll
              for (int x = 0; x < CH; ++x) o[x] = fmaf(held[c - group * W::DIMS + x], g, o[x]);
            }
            bool nan = look;
#pragma unroll
            for (int x = 0; x < CH; ++x) top = fmaxf(top, fabsf(o[x])), nan = nan || o[x] != o[x];
            const bool fine = !nan && is_finite(top);
            const bool mend = !fine && lim && is_finite(l);  // (positions that all columns see went through the products as they are)
            if (__any_sync(0xffffffffu, mend)) {
              if (!searched) search.search(p.a, seq, rs.head, rs.t0 * SP, min(__reduce_max_sync(0xffffffffu, lim), rs.t1 * SP));
              searched = true;
#pragma unroll 1
              for (int q = 0; q < CH; ++q) {
                const float s = search.sum(c + q, lim);
#pragma unroll
                for (int x = 0; x < CH; ++x)
                  if (x == q && mend && s != 0.f) o[x] = s;
              }
            }
#pragma unroll
            for (int x = 0; x < CH; ++x) o[x] = !ok ? NAN : none ? 0.f : o[x] * f;
            if constexpr (F) {
#pragma unroll
              for (int x = 0; x < CH; x += 4)
                *reinterpret_cast<float4*>(place(lane, w0 + (c - c0 + x) / 4) + part0) = make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
            } else {
#pragma unroll
              for (int x = 0; x < CH; x += 8)
                *reinterpret_cast<uint4*>(place(lane, w0 + (c - c0 + x) / 8) + part0) =
                    make_uint4(pack2(o[x], o[x + 1]), pack2(o[x + 2], o[x + 3]), pack2(o[x + 4], o[x + 5]), pack2(o[x + 6], o[x + 7]));
            }
          }
          __syncwarp();
#pragma unroll 8
          for (int i = 0; i < WORDS; ++i) {
            const int y = (32 * i + lane) / WORDS, x = lane % WORDS, c = col - lane + y;
            if (c >= p.cols) continue;
            const uint4 v = *reinterpret_cast<const uint4*>(place(y, w0 + x) + part0);
            if (!whole) {
              reinterpret_cast<uint4*>(part + (ptrdiff_t)(y - lane) * (HD + 4) + c0)[x] = v;
            } else {
              const int rw = row_of(p, c), at = rs.head * p.gqa + c - rw * p.gqa;
              T* dst = reinterpret_cast<T*>(const_cast<void*>(p.out.p)) + seq * p.out.seq + rw * p.out.row + at * p.out.head;
              reinterpret_cast<uint4*>(dst + c0)[x] = v;
            }
          }
          __syncwarp();
        }
      };
      if (whole && !W::F32) leave(std::false_type());
      else leave(std::true_type());
      if constexpr (GR > 1)
        if (lane == 0) arrive(smem_addr(&out_done));  // (behind the warp's last __syncwarp)
      if (there && group == 0) {
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

// Items cut between blocks: a warp joins two columns of an item, in the blocks' order, up to four parts of each on their
// way; each lane finds the part of a block.  (The join that the few-column kernel uses, a column after another and the parts found
// once a block: 11 us of 1024 rows' 69.)  Items without a step get zeros.
template <int HD, class T>
__global__ void __launch_bounds__(256) k_wide_join(const __grid_constant__ AttArgs p, int CT, int SP, int G) {
  constexpr int V = HD / 32;  // dimensions of a lane
  const int e = blockIdx.x / p.a.n_kv_heads, head = blockIdx.x - e * p.a.n_kv_heads;
  const int seq = e / p.n_ctiles, j = e - seq * p.n_ctiles;
  const int lane = threadIdx.x & 31, c0 = blockIdx.y * 16 + (threadIdx.x >> 5) * 2;
  behind();
  if (c0 >= min(CT, p.cols - j * CT)) return;
  const longlong2 it = p.item[blockIdx.x];
  const long long total = *p.total;
  const int nt = tiles_of(p, e, CT, SP);
  if (nt && (it.x < 0 || it.y < 0 || it.y >= G)) return;  // done by its block
  float m[2] = {kLow, kLow}, l[2] = {0.f, 0.f}, o[2][V];
  bool none = true;  // no part yet
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int x = 0; x < V; ++x) o[c][x] = 0.f;
  for (long long b0 = it.y; nt && b0 < G; b0 += 32) {
    const long long b = b0 + lane, lo = b < G ? first_place(total, b, G) - it.x - kOver : nt;
    const long long hi = b < G ? first_place(total, b + 1, G) - it.x - kOver : nt;
    const bool mine = b < G && lo < nt && hi > 0 && hi > lo;
    const int slot = mine ? part_slot(b, lo > 0) : 0;
    uint32_t has = __ballot_sync(0xffffffffu, mine);
    const bool end = __any_sync(0xffffffffu, lo >= nt);
    while (has) {
      // (all reads first: where there are fewer parts the first one is read again, and counts nothing)
      float2 ml[4][2];
      float v[4][2][V];
      bool part[4];
      const int one = __ffs(has) - 1;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        part[i] = has != 0;
        const int s = __shfl_sync(0xffffffffu, slot, has ? __ffs(has) - 1 : one);
#pragma unroll
        for (int c = 0; c < 2; ++c) {  // (a column behind the last has a place too)
          const float* src = p.part + ((size_t)s * CT + c0 + c) * (HD + 4);
          ml[i][c] = __ldcg(reinterpret_cast<const float2*>(src + HD));
          if constexpr (V == 4) {
            const float4 y = __ldcg(reinterpret_cast<const float4*>(src) + lane);
            v[i][c][0] = y.x, v[i][c][1] = y.y, v[i][c][2] = y.z, v[i][c][3] = y.w;
          } else {
            const float2 y = __ldcg(reinterpret_cast<const float2*>(src) + lane);
            v[i][c][0] = y.x, v[i][c][1] = y.y;
          }
        }
        has &= has - 1;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (!part[i]) ml[i][c] = make_float2(kLow, 0.f);
#pragma unroll
          for (int x = 0; x < V; ++x) v[i][c][x] = part[i] ? v[i][c][x] : 0.f;
        }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float M = m[c];
#pragma unroll
        for (int i = 0; i < 4; ++i) M = fmaxf(M, ml[i][c].x);
        const float f0 = exp2_fast(m[c] - M);
        float f[4];
        bool lost = !none && f0 == 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[i] = exp2_fast(ml[i][c].x - M);
          lost = lost || (f[i] == 0.f && part[i]);
        }
        m[c] = M;
        l[c] *= f0;
#pragma unroll
        for (int i = 0; i < 4; ++i) l[c] += ml[i][c].y * f[i];
        if (lost) {
#pragma unroll
          for (int x = 0; x < V; ++x) {
            o[c][x] = taken(o[c][x], f0);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[c][x] += taken(v[i][c][x], f[i]);
          }
        } else {
#pragma unroll
          for (int x = 0; x < V; ++x) {
            o[c][x] *= f0;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[c][x] += v[i][c][x] * f[i];
          }
        }
      }
      none = false;
    }
    if (end) break;
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int col = j * CT + c0 + c;
    if (c0 + c >= CT || col >= p.cols) break;
    const int row = row_of(p, col), hd = head * p.gqa + col - row * p.gqa;
    T* dst = reinterpret_cast<T*>(const_cast<void*>(p.out.p)) + seq * p.out.seq + row * p.out.row + hd * p.out.head + V * lane;
#pragma unroll
    for (int x = 0; x < V; ++x) o[c][x] = l[c] == 0.f ? 0.f : o[c][x] / l[c];
    if constexpr (std::is_same<T, float>::value) {
      if constexpr (V == 4) *reinterpret_cast<float4*>(dst) = make_float4(o[c][0], o[c][1], o[c][2], o[c][3]);
      else *reinterpret_cast<float2*>(dst) = make_float2(o[c][0], o[c][1]);
    } else {
      if constexpr (V == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(pack2(o[c][0], o[c][1]), pack2(o[c][2], o[c][3]));
      else *reinterpret_cast<uint32_t*>(dst) = pack2(o[c][0], o[c][1]);
    }
    if (p.lse && lane == 0)
      p.lse[((size_t)seq * p.a.rows + row) * p.n_heads + hd] =
          l[c] == 0.f ? -INFINITY : (m[c] + log2f(l[c])) * 0.69314718055994530942f;
  }
}

template <int HD, class T, int TB>
WideKernel info() {
  using W = PWide<HD, T, TB>;
  return {reinterpret_cast<const void*>(&k_paged_wide<HD, T, TB>), W::CT, W::SP, W::SMEM, 1, W::THREADS};
}

}  // namespace

const void* paged_wide_join(int head_dim, int dtype) {
  if (dtype == MK_F32)
    return head_dim == 64 ? reinterpret_cast<const void*>(&k_wide_join<64, float>) : reinterpret_cast<const void*>(&k_wide_join<128, float>);
  return head_dim == 64 ? reinterpret_cast<const void*>(&k_wide_join<64, __nv_bfloat16>)
                        : reinterpret_cast<const void*>(&k_wide_join<128, __nv_bfloat16>);
}

WideKernel paged_wide_kernel(int head_dim, int dtype, int cols, long long steps) {
  if (dtype == MK_F32) return head_dim == 64 ? info<64, float, 1>() : info<128, float, 1>();
  // Two tiles a block read K and V half as often and leave the products less idle, one tile runs in finer shares (rows of 4
  // columns, 4 heads of 128; one and two tiles: one sequence of 8022 positions, 64 rows 26.3 and 36.1 us, 512 52.3 and 54.3, 1024 89.6
  // and 83.8; two of 20000, 1024 rows 529 and 504; 32 of 8022, 40 rows 206 and 182, 64 rows 206 and 176).  An odd tile leaves a half
  // of its block idle: no more than one of nine.
  const int tiles = (cols - 1) / 128 + 1;
  if (steps <= 40 || (tiles < 8 && tiles % 2)) return head_dim == 64 ? info<64, __nv_bfloat16, 1>() : info<128, __nv_bfloat16, 1>();
  return head_dim == 64 ? info<64, __nv_bfloat16, 2>() : info<128, __nv_bfloat16, 2>();
}

}  // namespace mk
