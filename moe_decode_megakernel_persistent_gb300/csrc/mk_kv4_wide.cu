// Attention over the 4-bit paged cache for many query columns (prompt chunks, batches
// of drafts): tiles of 128 columns on the 5th-generation tensor cores (tcgen05).  The
// mathematics, the split of the work and the join are those of
// mk_kv4_attention.cu; what differs is where the scales go and who does what.
//
//   S = Q K^T   128 columns x 64 positions.  K = code x scale in fp16: 3 bits x 8
//               bits are exact in its 11.  The code is the subnormal +-m 2^-20 times 2^15,
//               the scale is times a power of two of the tile (its largest maps to
//               2^14..2^15), so that all is exact down to a scale of 2^-26 of the tile's
//               largest: positions that a row does not see, or gives no weight, may be so much
//               larger than those that it does.  (A smaller scale's values are rounded to
//               2^-25, at most 2^-36 of the tile's largest value.  With the codes left
//               subnormal that was 2^-21, and a hidden outlier of 2^12 showed.)  Q is fp16
//               times a power of two of the row (a bf16 value is exact down to 2^-31 of
//               its row's largest).  The powers multiply the fp32 scores.
//   O += P V    P = weights in fp16 (rounded by 2^-11, where the output is rounded
//               by 2^-8) over S's place in TMEM; V as K, its power following the largest
//               scale of the run with 2^3 of room (exact down to 2^-23 of the largest, else
//               rounded by at most 2^-33 of it), O rescaled when it moves.
// So the 128 x 64 scores of a step need no scale of their own, and one pass: 64
// scores a thread in registers, their maximum, one exponential each.  (With the
// scales applied to scores and weights, as the narrow kernel does, a step took
// 3,700 cycles of a column warp, and the call below 195 us.)
//
// Warps 0..3: a thread has a query column (a TMEM lane).  Its maximum moves only
// when a score passes it by 2^8; then the warp rescales its sums in TMEM.
// Warps 4..7 unpack: 16 bytes of codes become four 16-byte words of operands in
// the 128-byte swizzled layout, dimensions 0 2 1 3 4 6 5 7 of every eight (q is laid
// the same, and the sums are put back).  The next tile's codes are in registers
// meanwhile.  K's operand of a step is laid while the second product of the step before
// the last still reads its V, and one lane of the four warps in turn issues the
// products, S of a step while the columns work on the one before it.  (By one warp
// for all steps 122 us where this took 115, by a warp of its own next to three that unpack 127.)
// Two blocks of an SM (256 TMEM columns each) fill each other's waits.
//
// fp32 rows: q and the weights are two fp16 parts each (22 bits), the products run on
// both, and V has no room but rescales O each time its largest scale passes a power of two
// (exact down to 2^-26 of the largest, else rounded by at most 2^-36 of it).  Their q fills the shared memory that a second
// block would need, so a block has two tiles of 128 columns, which share the unpacked operands.  (For
// bf16 rows that is no faster: 115 us against 113.)
//
// Measured, 1024 rows of 16 heads on 4 kv heads of 128 dimensions at 8022 positions: bf16
// 116 us, 545 TFLOP/s of 4 x dimensions x seen pairs, tensor cores 24% active (113 us with the
// codes left subnormal); fp32 157 us (546 by the narrow kernel).  A bf16 step takes about 2,900 cycles of a block, in which a column
// warp works 2,200 and waits for the scores otherwise.
#include <algorithm>

#include "mk_kv4_att.cuh"
#include "mk_tcgen05.cuh"

namespace mk {
namespace {

// TB tiles of 128 columns of a block, for rows of type T.
template <int HD, class T, int TB>
struct Wide {
  static constexpr bool F32 = std::is_same<T, float>::value;
  static constexpr int NG = HD / kGroup, CT = 128 * TB, SP = kTile;
  static constexpr int QP = F32 ? 2 : 1;            // fp16 parts of q, and of the weights
  static constexpr int QT = NG * 128 * 128;         // bytes of a tile's q operand of one part
  static constexpr int QB = TB * QP * QT;
  static constexpr int KVB = NG * SP * 128;         // of K's (or V's) operand of a step
  static constexpr int SMEM = 1024 + QB + 4 * KVB;
  static constexpr int TM = 256;                    // TMEM columns of a tile: S of two steps [2][64], O [HD]
  static constexpr int UW = 4 * TB;                 // the first unpacking warp
  static constexpr int THREADS = 32 * (UW + 4), BLOCKS = TB == 1 ? 2 : 1;
  static constexpr int ROOM = F32 ? 0 : 3;          // V's scales may grow by 2^ROOM before O is rescaled
};

// Two codes as subnormals, times 2^15 (+-m 2^-5, exactly), times b.
__device__ __forceinline__ uint32_t scaled(uint32_t a, uint32_t b) {  // f16x2
  uint32_t y;
  asm("{ .reg .b32 t; mul.rn.f16x2 t, %1, %3; mul.rn.f16x2 %0, t, %2; }" : "=r"(y) : "r"(a), "r"(b), "r"(0x78007800));
  return y;
}
constexpr float kUnit = 32.f;  // an operand value is code x scale / kUnit
// Four bytes of codes times the scale pair h as eight operand values, dimensions
// 0 2 1 3 4 6 5 7.
__device__ __forceinline__ uint4 unpack(uint32_t w, uint32_t h) {
  const uint32_t x = __byte_perm(w, 0, 0x1100), y = __byte_perm(w, 0, 0x3322);
  return make_uint4(scaled((x << 4) & kNib, h), scaled(x & kNib, h), scaled((y << 4) & kNib, h), scaled(y & kNib, h));
}
// 2^n, n held to fp32's normal range.
__device__ __forceinline__ float power(int n) { return __uint_as_float((uint32_t)(min(max(n, -126), 127) + 127) << 23); }
__device__ __forceinline__ int exponent(float x) { return (int)(__float_as_uint(x) >> 23 & 255u) - 127; }
__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

constexpr int kFirst = 1 << 8;  // of a step's note: the first of a run (low bits: positions that exist)
constexpr float kRoom = 6.f;    // the weights are at most 2^(kLazy + kRoom) in fp16

// What the unpacking warps say of a step.
struct StepSays {
  float k_mul;       // what the scores are times, but for the row's power
  float v_exp;       // V's power of two: the operand is V 2^v_exp / kUnit
  uint32_t bad[4];   // V scales that are no numbers: [group][positions 0..31, 32..63]
};

template <int HD, class T, int TB>
__global__ void __launch_bounds__(Wide<HD, T, TB>::THREADS, Wide<HD, T, TB>::BLOCKS) k_kv4_wide(const __grid_constant__ AttArgs p) {
  using W = Wide<HD, T, TB>;
  using L = Tile<HD>;
  constexpr int NG = W::NG, CT = W::CT, SP = W::SP, UW = W::UW;
  extern __shared__ uint8_t sm_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~(uintptr_t)1023);
  __shared__ __align__(8) uint64_t k_full[4], v_full[2], s_full[2][TB], p_full[2][TB], pv_done[2], q_full;
  __shared__ unsigned long long list[kList];
  __shared__ int note[kList];
  __shared__ StepSays says[4];
  __shared__ uint32_t tm_base;
  __shared__ Runs s_run;       // the block's first run and number of steps, the same for all warps
  __shared__ uint32_t s_steps;  // (should someone write the lengths while the call runs)
  __shared__ volatile int give_up;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  uint8_t* q_op = sm;
  uint8_t* kv_op = sm + W::QB;  // [stage][K | V][g][64][128]
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // A wait's one bit tells neighbouring phases apart, so none may be two ahead of who
  // waits for it.  K's operand of step i is laid when S of i - 2 is done and V's when
  // pv_done of i - 2 is, so v_full, s_full, p_full and pv_done of a stage wait for
  // who reads the last one; k_full may be a stage's round ahead of the columns and has four.
  if (tid == 0) {
    auto init = [](uint64_t* b, int n) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(b)), "r"(n) : "memory");
    };
    for (int i = 0; i < 4; ++i) init(&k_full[i], 4);  // by each unpacking warp
    for (int i = 0; i < 2; ++i) {
      init(&v_full[i], 4);
      init(&pv_done[i], 1);
      for (int t = 0; t < TB; ++t) {
        init(&s_full[i][t], 1);
        init(&p_full[i][t], 4);  // by each of the tile's warps
      }
    }
    init(&q_full, 4 * TB);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    give_up = 0;
  }
  if (w == 0) {
    const Runs r = first_run(p, CT, SP, lane);
    if (lane == 0) {
      s_run = r;
      s_steps = r.steps(p, CT, SP);
    }
  }
  if (w == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tm_base)), "n"(W::TM * TB)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  before_sync();
  __syncthreads();
  after_sync();
  const uint32_t tm = tm_base;  // tile t: S at 256 t, O at 256 t + 128
  Runs run = s_run;
  const Runs mine = run;
  const uint32_t n_steps = s_steps;

  if (w >= UW) {  // ---- unpacking, and the products (the warps take turns)
    const int u = tid - 32 * UW;
    auto look_up = [&](uint32_t i) {
      Runs r = mine;
      uint32_t before = 0;
      while (i >= before + (r.t1 - r.t0)) {
        before += r.t1 - r.t0;
        if (!r.next(p, CT, SP)) {
          list[i % kList] = 0;
          note[i % kList] = 0;
          return;
        }
      }
      const int t = r.t0 + (int)(i - before), seq = p.n_ctiles == 1 ? r.e : r.e / p.n_ctiles;
      int len, nn;
      seq_extent(p.a, seq, len, nn);
      const int pg = page_of(p.a, seq, t * SP);
      list[i % kList] = pg < 0 ? 0 : (unsigned long long)tile_of<HD>(p.a, pg, r.head, t * SP);
      note[i % kList] = (pg < 0 ? 0 : min(SP, len - t * SP)) | (i == before ? kFirst : 0);
    };
    for (uint32_t i = u; i < kList && i < n_steps; i += 128) look_up(i);
    asm volatile("bar.sync 2, 128;" ::: "memory");
    // a thread's part of a tile: NG 16-byte words of K codes and of V codes, and
    // each warp all positions' scales
    uint4 kc[NG], vc[NG];
    uint32_t ks[2], vs[2];  // of positions lane and lane + 32, both groups
    // (eight neighbouring threads take eight rows: their stores meet all banks once)
    auto place = [&](int c, int& r, int& cc) {
      const int x = u + 128 * c;
      r = (x >> 3) / (2 * NG) * 8 + (x & 7);
      cc = (x >> 3) % (2 * NG);
    };
    auto word = [&](int c) {
      int r, cc;
      place(c, r, cc);
      return r * 2 * NG + cc;
    };
    auto fetch_k = [&](uint32_t i) {
      const uint8_t* src = reinterpret_cast<const uint8_t*>(list[i % kList]);
      const int have = note[i % kList] & (kFirst - 1);
#pragma unroll
      for (int c = 0; c < NG; ++c)
        kc[c] = src ? __ldg(reinterpret_cast<const uint4*>(src) + word(c)) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = lane + 32 * h;
        ks[h] = vs[h] = 0;
        if (at < have) {  // a slot behind the end may hold anything: its scales count as 0
          if constexpr (NG == 2) {
            ks[h] = __ldg(reinterpret_cast<const uint32_t*>(src + L::CODES) + at);
            vs[h] = __ldg(reinterpret_cast<const uint32_t*>(src + L::V + L::CODES) + at);
          } else {
            ks[h] = __ldg(reinterpret_cast<const uint16_t*>(src + L::CODES) + at);
            vs[h] = __ldg(reinterpret_cast<const uint16_t*>(src + L::V + L::CODES) + at);
          }
        }
      }
    };
    auto fetch_v = [&](uint32_t i) {
      const uint8_t* src = reinterpret_cast<const uint8_t*>(list[i % kList]);
#pragma unroll
      for (int c = 0; c < NG; ++c)
        vc[c] = src ? __ldg(reinterpret_cast<const uint4*>(src + L::V) + word(c)) : make_uint4(0, 0, 0, 0);
    };
    // a thread's words of codes as operands, times their scales and f
    auto lay = [&](uint8_t* to, const uint4* from, uint32_t of0, uint32_t of1, float f, bool v) {
#pragma unroll
      for (int c = 0; c < NG; ++c) {
        int r, cc;
        place(c, r, cc);
        const int g = cc / 2;
        const uint32_t both = __shfl_sync(0xffffffffu, (r & 32) ? of1 : of0, r & 31);  // (a warp's rows of one c are in one half)
        float x = g ? high_f(both) : low_f(both);
        if (v && !finite(x)) x = 0.f;  // what sees such a position is told of it instead
        x *= f;
        const uint32_t h = pack2h(x, x), word4[4] = {from[c].x, from[c].y, from[c].z, from[c].w};
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4)
          *reinterpret_cast<uint4*>(to + g * SP * 128 + r * 128 + ((((cc & 1) * 4 + i4) ^ (r & 7)) << 4)) = unpack(word4[i4], h);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
    };
    // the largest finite of a tile's scales
    auto largest = [&](uint32_t a, uint32_t b) {
      float top = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const float x = fabsf(g ? high_f(h ? b : a) : low_f(h ? b : a));
          if (finite(x)) top = fmaxf(top, x);
        }
      return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));  // (non-negative floats: in their bits' order)
    };
    if (n_steps) {
      fetch_k(0);
      fetch_v(0);
    }
    uint32_t n_runs = 0;
    constexpr uint32_t id_qk = (1u << 4) | ((SP >> 3) << 17) | ((128 >> 4) << 24);               // fp16, fp32 sums
    constexpr uint32_t id_pv = (1u << 4) | (1u << 16) | ((HD >> 3) << 17) | ((128 >> 4) << 24);  // V by rows
    // the second product of step i, once its weights are there
    auto second = [&](uint32_t i) {
      bool ok = bar_wait(smem_addr(&v_full[i & 1]), (i >> 1) & 1, &give_up, p.a.status);
      const uint32_t add = note[i % kList] & kFirst ? 0 : 1;
      const uint64_t v = operand(smem_addr(kv_op + ((i & 1) * 2 + 1) * W::KVB), SP * 128);
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        ok = bar_wait(smem_addr(&p_full[i & 1][t]), (i >> 1) & 1, &give_up, p.a.status) && ok;
        after_sync();
        if (lane == 0 && ok && !give_up) {
          const uint32_t pw = tm + W::TM * t + SP * (i & 1), to = tm + W::TM * t + 2 * SP;
#pragma unroll
          for (int x = W::QP - 1; x >= 0; --x)  // the weights' low part first
#pragma unroll
            for (int kk = 0; kk < SP / 16; ++kk)
              mma_ts(to, pw + 32 * x + 8 * kk, v + ((kk * 16 * 128) >> 4), id_pv, kk || x < W::QP - 1 ? 1 : add);
          if (t == TB - 1) commit(smem_addr(&pv_done[i & 1]));
        }
        __syncwarp();
      }
    };
    float cap = 0.f;  // V's scales of the run are below it
    for (uint32_t i = 0; i < n_steps; ++i) {
      if (i % (kList / 2) == 0 && i) {
        asm volatile("bar.sync 2, 128;" ::: "memory");
        // (the notes of the last steps are still read: 16 of them stay)
        if (i + kList / 2 - 16 + u < n_steps) look_up(i + kList / 2 - 16 + u);
        asm volatile("bar.sync 2, 128;" ::: "memory");
      }
      const int st = i & 1;
      const bool first = note[i % kList] & kFirst;
      if (first) ++n_runs;
      if (i >= 2)
        for (int t = 0; t < TB; ++t) bar_wait(smem_addr(&s_full[st][t]), ((i - 2) >> 1) & 1, &give_up, p.a.status);
      const int nk = min(max(14 - exponent(largest(ks[0], ks[1])), -100), 100);  // K's scales times 2^nk: below 2^15
      const float tv = largest(vs[0], vs[1]);
      if (first) cap = 0.f;
      if (tv > cap || cap == 0.f) cap = power(min(max(exponent(tv) + 1 + W::ROOM, -80), 100));  // the next power of two, and some room
      const int nv = 15 - exponent(cap);
      if (w == UW) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const uint32_t bad = __ballot_sync(0xffffffffu, !finite(g ? high_f(vs[h]) : low_f(vs[h])));
            if (lane == 0) says[i & 3].bad[2 * g + h] = bad;
          }
        if (lane == 0) {
          says[i & 3].k_mul = kUnit * power(-nk);
          says[i & 3].v_exp = (float)nv;
        }
      }
      uint8_t* kd = kv_op + st * 2 * W::KVB;
      lay(kd, kc, ks[0], ks[1], power(nk), false);
      const uint32_t v0 = vs[0], v1 = vs[1];
      if (lane == 0) arrive(smem_addr(&k_full[i & 3]));
      if (i + 1 < n_steps) fetch_k(i + 1);
      if (i >= 2) bar_wait(smem_addr(&pv_done[st]), ((i - 2) >> 1) & 1, &give_up, p.a.status);
      if (w - UW == (i & 3)) {
        bool ok = bar_wait(smem_addr(&k_full[i & 3]), (i >> 2) & 1, &give_up, p.a.status);
        if (first) {  // the columns lay q after they have read the last run's sums
          ok = bar_wait(smem_addr(&q_full), (n_runs - 1) & 1, &give_up, p.a.status) && ok;
        }
        after_sync();
        if (lane == 0 && ok && !give_up) {
          const uint64_t k = operand(smem_addr(kd));
#pragma unroll
          for (int t = 0; t < TB; ++t) {
            const uint32_t to = tm + W::TM * t + SP * st;  // the weights of step i - 2 were there
#pragma unroll
            for (int x = W::QP - 1; x >= 0; --x) {  // q's low part first
              const uint64_t q = operand(smem_addr(q_op + (t * W::QP + x) * W::QT));
#pragma unroll
              for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                  const uint64_t qa = q + ((g * 128 * 128 + kk * 32) >> 4), kb = k + ((g * SP * 128 + kk * 32) >> 4);
                  if (g == 0 && kk == 0 && x == W::QP - 1) mma_ss<false>(to, qa, kb, id_qk);
                  else mma_ss<true>(to, qa, kb, id_qk);
                }
            }
            commit(smem_addr(&s_full[st][t]));
          }
        }
        __syncwarp();
      }
      lay(kd + W::KVB, vc, v0, v1, power(nv), true);
      if (lane == 0) arrive(smem_addr(&v_full[st]));
      if (i + 1 < n_steps) fetch_v(i + 1);
      // (the sums take one step's products after another's: step i - 2's are done)
      if (w - UW == ((i + 2) & 3) && i) second(i - 1);
    }
    if (w == UW && n_steps) {
      if (n_steps >= 2) bar_wait(smem_addr(&pv_done[n_steps & 1]), ((n_steps - 2) >> 1) & 1, &give_up, p.a.status);
      second(n_steps - 1);
    }
  } else {  // ---- a query column each
    const int tile = w >> 2, tt = tid & 127;
    // this warp's lanes of its tile's scores and sums
    const uint32_t tm_s = tm + W::TM * tile + ((uint32_t)(32 * (w & 3)) << 16), tm_o = tm_s + 2 * SP;
    uint32_t k = 0;
    for (bool more = n_steps > 0; more; more = run.next(p, CT, SP)) {
      const int seq = p.n_ctiles == 1 ? run.e : run.e / p.n_ctiles, j = run.e - seq * p.n_ctiles;
      const int col = j * CT + tid;
      const bool there = col < p.cols;
      const int row = there ? row_of(p, col) : 0, hd = run.head * p.gqa + (there ? col - row * p.gqa : 0);
      int len, nn;
      seq_extent(p.a, seq, len, nn);
      const int lim = there && row < nn ? max(0, len - nn + row + 1) : 0;  // positions that it sees
      float c_row;  // times a step's k_mul, the scores' factor
      {
        const T* src = reinterpret_cast<const T*>(p.q.p) + seq * p.q.seq + row * p.q.row + hd * p.q.head;
        // (bf16 rows wait in registers for their largest value, fp32 rows are read twice)
        uint4 qr[W::F32 ? 1 : HD / 8];
        if constexpr (!W::F32) {
#pragma unroll
          for (int x = 0; x < HD / 8; ++x) qr[x] = there ? *reinterpret_cast<const uint4*>(src + 8 * x) : make_uint4(0, 0, 0, 0);
        }
        auto eight = [&](int x, float (&y)[8]) {
          if constexpr (W::F32) {
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
            if (there) {
              a = __ldg(reinterpret_cast<const float4*>(src + 8 * x));
              b = __ldg(reinterpret_cast<const float4*>(src + 8 * x + 4));
            }
            y[0] = a.x, y[1] = a.y, y[2] = a.z, y[3] = a.w, y[4] = b.x, y[5] = b.y, y[6] = b.z, y[7] = b.w;
          } else {
            const uint32_t u4[4] = {qr[x].x, qr[x].y, qr[x].z, qr[x].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) y[2 * i] = low_f(u4[i]), y[2 * i + 1] = high_f(u4[i]);
          }
        };
        float top = 0.f;
#pragma unroll
        for (int x = 0; x < HD / 8; ++x) {
          float y[8];
          eight(x, y);
#pragma unroll
          for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(y[i]));
        }
        const int nq = min(max(14 - exponent(top), -100), 100);
        const float f = p.c < 0.f ? -power(nq) : power(nq);
        c_row = fabsf(p.c) * power(-65) * power(-nq);
#pragma unroll
        for (int x = 0; x < HD / 8; ++x) {
          float y[8];
          eight(x, y);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] *= f;
          uint8_t* to = q_op + tile * W::QP * W::QT + x / 8 * 128 * 128 + tt * 128 + (((x % 8) ^ (tt & 7)) << 4);
#pragma unroll
          for (int q = 0; q < W::QP; ++q) {
            const uint4 h = make_uint4(pack2h(y[0], y[2]), pack2h(y[1], y[3]), pack2h(y[4], y[6]), pack2h(y[5], y[7]));
            *reinterpret_cast<uint4*>(to + q * W::QT) = h;
            if (q + 1 < W::QP) {
              y[0] -= low_h(h.x), y[2] -= high_h(h.x), y[1] -= low_h(h.y), y[3] -= high_h(h.y);
              y[4] -= low_h(h.z), y[6] -= high_h(h.z), y[5] -= low_h(h.w), y[7] -= high_h(h.w);
            }
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive(smem_addr(&q_full));
      // running maximum (log2), the sum of the weights times 2^kRoom, V's power,
      // and whether a V that is no number was seen in a group
      float m = kLow, l = 0.f, e = 0.f;
      bool bad[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) bad[g] = false;
      for (int t = run.t0; t < run.t1; ++t, ++k) {
        const int st = k & 1;
        bool ok = bar_wait(smem_addr(&k_full[k & 3]), (k >> 2) & 1, &give_up, p.a.status);
        ok = bar_wait(smem_addr(&s_full[st][tile]), (k >> 1) & 1, &give_up, p.a.status) && ok;
        after_sync();
        if (ok && !give_up) {
          const int vis = min(lim - t * SP, note[k % kList] & (kFirst - 1));  // of the step's positions
          const float cf = c_row * says[k & 3].k_mul, ne = says[k & 3].v_exp;
          const uint32_t at = tm_s + SP * st;
          auto step = [&](auto cut_) {
            constexpr bool CUT = decltype(cut_)::value;
            float s[4][16], mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 4; c += 2) tm_read32(at + 16 * c, *reinterpret_cast<float(*)[32]>(s[c]));
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int x = 0; x < 16; ++x) {
                if (CUT && 16 * c + x >= vis) s[c][x] = -INFINITY;
                mx[x & 3] = fmaxf(mx[x & 3], s[c][x]);
              }
            float most = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            most = most == -INFINITY ? most : most * cf;
            if (__any_sync(0xffffffffu, most > m + kLazy || ne != e)) {
              const float nm = fmaxf(m, most), f = exp2_fast(m - nm), fo = f * exp2_fast(ne - e);
              m = nm;
              e = ne;
              l *= f;
              if (t > run.t0) {
                bar_wait(smem_addr(&pv_done[(k - 1) & 1]), ((k - 1) >> 1) & 1, &give_up, p.a.status);  // the sums hold the last step
                after_sync();
#pragma unroll 1
                for (int c = 0; c < HD; c += 16) {
                  float o[16];
                  uint32_t x16[16];
                  tm_read16(tm_o + c, o);
#pragma unroll
                  for (int x = 0; x < 16; ++x) x16[x] = __float_as_uint(o[x] * fo);
                  tm_store16(tm_o + c, x16);
                }
              }
            }
            const float sub = kRoom - m;
            float la[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 4; c += 2) {
              uint32_t b[16];
              [[maybe_unused]] uint32_t low[W::F32 ? 16 : 1];
#pragma unroll
              for (int x = 0; x < 32; x += 2) {
                float w2[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  float& z = s[c + x / 16][x % 16 + y];
                  w2[y] = CUT && z == -INFINITY ? 0.f : exp2_fast(fmaf(z, cf, sub));
                  la[(x + y) & 3] += w2[y];
                }
                b[x / 2] = pack2h(w2[0], w2[1]);
                if constexpr (W::F32) low[x / 2] = pack2h(w2[0] - low_h(b[x / 2]), w2[1] - high_h(b[x / 2]));
              }
              tm_store16(at + 8 * c, b);  // over the scores, which are all in registers
              if constexpr (W::F32) tm_store16(at + 32 + 8 * c, low);
            }
            l += (la[0] + la[1]) + (la[2] + la[3]);
          };
          if (__all_sync(0xffffffffu, vis >= SP)) step(std::false_type());
          else step(std::true_type());
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const uint32_t b0 = says[k & 3].bad[2 * g], b1 = says[k & 3].bad[2 * g + 1];
            if (b0 | b1) {
              const uint32_t v0 = vis >= 32 ? ~0u : vis > 0 ? (1u << vis) - 1 : 0u;
              const uint32_t v1 = vis >= 64 ? ~0u : vis > 32 ? (1u << (vis - 32)) - 1 : 0u;
              bad[g] |= (b0 & v0) || (b1 & v1);
            }
          }
          tm_stored();
        }
        before_sync();
        __syncwarp();
        if (lane == 0) arrive(smem_addr(&p_full[st][tile]));
      }
      // ---- the run's end: this column's sums, dimensions put back in order
      bar_wait(smem_addr(&pv_done[(k - 1) & 1]), ((k - 1) >> 1) & 1, &give_up, p.a.status);
      after_sync();
      const bool whole = run.t0 == 0 && run.t1 == run.nt;
      const float undo = kUnit * exp2f(-e), M = m - kRoom;
      const float f = whole ? (l == 0.f ? 0.f : undo / l) : undo;
      float* part = p.part + ((size_t)part_slot(blockIdx.x, run.t0) * CT + tid) * (HD + 4);
      T* dst = reinterpret_cast<T*>(const_cast<void*>(p.out.p)) + seq * p.out.seq + row * p.out.row + hd * p.out.head;
#pragma unroll 1
      for (int c = 0; c < HD; c += 16) {
        float o[16];
        tm_read16(tm_o + c, o);
        if (!there) continue;
        const bool nan = give_up || (NG == 2 && c >= 64 ? bad[NG - 1] : bad[0]);
#pragma unroll
        for (int x = 0; x < 16; ++x) o[x] = nan ? NAN : o[x] * f;
#pragma unroll
        for (int x = 0; x < 16; x += 8) {  // 0 2 1 3 4 6 5 7
          if (whole && !W::F32) {
            *reinterpret_cast<uint4*>(dst + c + x) = make_uint4(pack2(o[x], o[x + 2]), pack2(o[x + 1], o[x + 3]),
                                                                pack2(o[x + 4], o[x + 6]), pack2(o[x + 5], o[x + 7]));
          } else {
            float* to = whole ? reinterpret_cast<float*>(dst) : part;
            *reinterpret_cast<float4*>(to + c + x) = make_float4(o[x], o[x + 2], o[x + 1], o[x + 3]);
            *reinterpret_cast<float4*>(to + c + x + 4) = make_float4(o[x + 4], o[x + 6], o[x + 5], o[x + 7]);
          }
        }
      }
      if (there) {
        if (!whole) *reinterpret_cast<float2*>(part + HD) = l == 0.f ? make_float2(kLow, 0.f) : make_float2(M, give_up ? NAN : l);
        else if (p.lse)
          p.lse[((size_t)seq * p.a.rows + row) * p.n_heads + hd] =
              l == 0.f ? -INFINITY : (M + log2f(l)) * 0.69314718055994530942f;
      }
      if (tid == 0 && run.t0 == 0)
        p.item[(size_t)run.e * p.a.n_kv_heads + run.head] =
            make_longlong2(whole ? -1 : run.base + (long long)run.head * (run.nt + kOver), blockIdx.x);
      before_sync();  // the next run's products overwrite the sums
    }
  }
  before_sync();
  __syncthreads();
  if (w == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "n"(W::TM * TB));
}

template <int HD, class T, int TB>
WideKernel info() {
  using W = Wide<HD, T, TB>;
  return {reinterpret_cast<const void*>(&k_kv4_wide<HD, T, TB>), W::CT, W::SP, W::SMEM, W::BLOCKS, W::THREADS};
}

}  // namespace

WideKernel kv4_wide_kernel(int head_dim, int dtype) {
  if (dtype == MK_F32) return head_dim == 64 ? info<64, float, 2>() : info<128, float, 2>();
  return head_dim == 64 ? info<64, __nv_bfloat16, 1>() : info<128, __nv_bfloat16, 1>();
}

}  // namespace mk
