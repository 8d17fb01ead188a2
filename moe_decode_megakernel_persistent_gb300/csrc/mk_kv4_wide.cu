// Attention over the 4-bit paged cache for many query columns (prompt chunks):
// tiles of 128 columns on the 5th-generation tensor cores (tcgen05).  The
// mathematics, the split of the work and the join are those of
// mk_kv4_attention.cu; what differs is who does what in a block.
//
//   S_g = Q_g K_g^T   for each group g of 64 dimensions: 128 columns x 64
//                     positions, K = the codes as bf16 subnormals +-m 2^-129 (exact),
//                     Q carrying 2^64; both groups' sums stay apart in TMEM, since
//                     K's scales (one per position and group) multiply them;
//   O_g += P_g V_g    P_g = weight x V's scale in fp16, read from TMEM over S's
//                     place, V = the codes as fp16 subnormals +-m 2^-20.
//
// Warps 0..3: a thread has a query column (a TMEM lane).  It loads its 64 scores,
// applies K's scales, keeps the running maximum and sum, and stores the two
// groups' weights.  Running maxima and the normalisation of V's scales move only
// when they are passed (by 2^8, by the next power of two and 2^3); then the warp
// rescales its sums in TMEM.
// Warps 4..7 unpack the tiles: 16 bytes of codes become four 16-byte words of
// operands (1 instruction a value) in the 128-byte swizzled layout, dimensions
// 0 2 1 3 4 6 5 7 of every eight (q is laid the same, and the sums are put back).
// The next tile's codes are in registers meanwhile.  One lane of warp 4 issues the
// products.
// A block has one tile of S in flight (256 TMEM columns with O); two blocks
// of an SM fill each other's waits.
#include <algorithm>

#include "mk_kv4_att.cuh"

namespace mk {
namespace {

template <int HD>
struct Wide {
  static constexpr int NG = HD / kGroup, CT = 128, SP = kTile;
  static constexpr int QB = NG * CT * 128;          // bytes of q's operand
  static constexpr int KVB = NG * SP * 128;         // of K's (or V's) operand of a step
  static constexpr int SCB = 2 * NG * SP * 4;       // of a step's scales, fp32
  static constexpr int SMEM = 1024 + QB + 2 * (2 * KVB + SCB);
  static constexpr int TM = NG * 128;               // TMEM columns: S [NG][64], O [NG][64]
};

// Shared-memory operand, 128-byte swizzle, rows of 128 bytes in atoms of 8 rows.
__device__ __forceinline__ uint64_t operand(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
               "l"(a), "l"(b), "r"(idesc), "r"(add)
               : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
               "r"(a), "l"(b), "r"(idesc), "r"(add)
               : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_load16(uint32_t at, float (&x)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]), "=f"(x[8]),
        "=f"(x[9]), "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), "=f"(x[14]), "=f"(x[15])
      : "r"(at)
      : "memory");
}
// The loads have landed; x passes through, so that nothing uses it before.
__device__ __forceinline__ void tm_loaded(float (&x)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]), "+f"(x[6]), "+f"(x[7]), "+f"(x[8]),
                 "+f"(x[9]), "+f"(x[10]), "+f"(x[11]), "+f"(x[12]), "+f"(x[13]), "+f"(x[14]), "+f"(x[15])::"memory");
}
__device__ __forceinline__ void tm_store16(uint32_t at, const uint32_t (&x)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]), "r"(x[8]), "r"(x[9]),
      "r"(x[10]), "r"(x[11]), "r"(x[12]), "r"(x[13]), "r"(x[14]), "r"(x[15])
      : "memory");
}
__device__ __forceinline__ void tm_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Four bytes of codes as eight operand values, dimensions 0 2 1 3 4 6 5 7.
__device__ __forceinline__ uint4 unpack(uint32_t w) {
  const uint32_t x = __byte_perm(w, 0, 0x1100), y = __byte_perm(w, 0, 0x3322);
  return make_uint4((x << 4) & kNib, x & kNib, (y << 4) & kNib, y & kNib);
}

constexpr int kFirst = 1 << 8;  // of a step's note: the first of a run (low bits: positions that exist)

template <int HD>
__global__ void __launch_bounds__(256, 2) k_kv4_wide(const __grid_constant__ AttArgs p) {
  using W = Wide<HD>;
  using L = Tile<HD>;
  constexpr int NG = W::NG, CT = W::CT, SP = W::SP;
  extern __shared__ uint8_t sm_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~(uintptr_t)1023);
  __shared__ __align__(8) uint64_t kv_full[2], s_full, p_full, pv_done, q_full;
  __shared__ unsigned long long list[kList];
  __shared__ int note[kList];
  __shared__ float top_vs[2][2];  // the largest V scale of a step, by warp of 32 positions
  __shared__ uint32_t tm_base;
  __shared__ Runs s_run;
  __shared__ volatile int give_up;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  uint8_t* q_op = sm;
  uint8_t* kv_op = sm + W::QB;                                        // [stage][K | V][g][64][128]
  float* scales = reinterpret_cast<float*>(sm + W::QB + 4 * W::KVB);  // [stage][K g.., V g..][64]
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    const uint32_t bars[6] = {smem_addr(&kv_full[0]), smem_addr(&kv_full[1]), smem_addr(&s_full),
                              smem_addr(&p_full), smem_addr(&pv_done), smem_addr(&q_full)};
    const uint32_t n[6] = {4, 4, 1, 4, 1, 4};
    for (int i = 0; i < 6; ++i)
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bars[i]), "r"(n[i]) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    give_up = 0;
  }
  if (w == 0) {
    const Runs r = first_run(p, CT, SP, lane);
    if (lane == 0) s_run = r;
  }
  if (w == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tm_base)), "n"(W::TM)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  before_sync();
  __syncthreads();
  after_sync();
  const uint32_t tm = tm_base;
  Runs run = s_run;
  const Runs mine = run;
  uint32_t n_steps = run.t1 - run.t0;
  if (n_steps)
    for (Runs r = mine; r.next(p, CT, SP);) n_steps += r.t1 - r.t0;

  if (w >= 4) {  // ---- unpacking, and the products
    const int u = tid - 128;
    auto look_up = [&](uint32_t i) {
      Runs r = mine;
      uint32_t before = 0;
      while (i >= before + (r.t1 - r.t0)) {
        before += r.t1 - r.t0;
        if (!r.next(p, CT, SP)) return;
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
    // (the first 64 threads) a position's scales
    uint4 kc[NG], vc[NG];
    uint32_t ks = 0, vs = 0;
    auto fetch = [&](uint32_t i) {
      const uint8_t* src = reinterpret_cast<const uint8_t*>(list[i % kList]);
      const int have = note[i % kList] & (kFirst - 1);
#pragma unroll
      for (int c = 0; c < NG; ++c) {
        kc[c] = src ? __ldg(reinterpret_cast<const uint4*>(src) + u + 128 * c) : make_uint4(0, 0, 0, 0);
        vc[c] = src ? __ldg(reinterpret_cast<const uint4*>(src + L::V) + u + 128 * c) : make_uint4(0, 0, 0, 0);
      }
      ks = vs = 0;
      if (u < have) {  // a slot behind the end may hold anything
        if constexpr (NG == 2) {
          ks = __ldg(reinterpret_cast<const uint32_t*>(src + L::CODES) + u);
          vs = __ldg(reinterpret_cast<const uint32_t*>(src + L::V + L::CODES) + u);
        } else {
          ks = __ldg(reinterpret_cast<const uint16_t*>(src + L::CODES) + u);
          vs = __ldg(reinterpret_cast<const uint16_t*>(src + L::V + L::CODES) + u);
        }
      }
    };
    if (n_steps) fetch(0);
    uint32_t n_runs = 0;
    constexpr uint32_t id_qk = (1u << 4) | (1u << 7) | (1u << 10) | ((SP >> 3) << 17) | ((CT >> 4) << 24);   // bf16
    constexpr uint32_t id_pv = (1u << 4) | (1u << 16) | ((64 >> 3) << 17) | ((CT >> 4) << 24);               // fp16, V by rows
    // the second product of step i, once its weights are there
    auto second = [&](uint32_t i) {
      const bool ok = bar_wait(smem_addr(&p_full), i & 1, &give_up, p.a.status);
      after_sync();
      if (lane == 0 && ok && !give_up) {
        const uint32_t first = note[i % kList] & kFirst, v = smem_addr(kv_op + ((i & 1) * 2 + 1) * W::KVB);
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int kk = 0; kk < SP / 16; ++kk)
            mma_ts(tm + 64 * (NG + g), tm + 32 * g + 8 * kk, operand(v + g * SP * 128 + kk * 16 * 128), id_pv, !first || kk);
        commit(smem_addr(&pv_done));
      }
      __syncwarp();
    };
    for (uint32_t i = 0; i < n_steps; ++i) {
      if (i % (kList / 2) == 0 && i) {
        asm volatile("bar.sync 2, 128;" ::: "memory");
        // (the notes of the last steps are still read: 16 of them stay)
        if (i + kList / 2 - 16 + u < n_steps) look_up(i + kList / 2 - 16 + u);
        asm volatile("bar.sync 2, 128;" ::: "memory");
      }
      const int st = i & 1;
      if (i >= 2) bar_wait(smem_addr(&pv_done), i & 1, &give_up, p.a.status);  // step i - 2 has left the stage
      {
        uint8_t* kd = kv_op + st * 2 * W::KVB;
        uint8_t* vd = kd + W::KVB;
#pragma unroll
        for (int c = 0; c < NG; ++c) {
          const int x = u + 128 * c, r = x / (2 * NG), cc = x % (2 * NG), g = cc / 2;
          const uint32_t kw[4] = {kc[c].x, kc[c].y, kc[c].z, kc[c].w}, vw[4] = {vc[c].x, vc[c].y, vc[c].z, vc[c].w};
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            const int at = g * SP * 128 + r * 128 + ((((cc & 1) * 4 + i4) ^ (r & 7)) << 4);
            *reinterpret_cast<uint4*>(kd + at) = unpack(kw[i4]);
            *reinterpret_cast<uint4*>(vd + at) = unpack(vw[i4]);
          }
        }
        if (u < SP) {
          float* sc = scales + st * 2 * NG * SP + u;
          float top = 0.f;
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const float v = g ? high_f(vs) : low_f(vs);
            sc[g * SP] = (g ? high_f(ks) : low_f(ks)) * p.c;
            sc[(NG + g) * SP] = v;
            top = fmaxf(top, v);
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          if (lane == 0) top_vs[st][w - 4] = top;
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive(smem_addr(&kv_full[st]));
      if (i + 1 < n_steps) fetch(i + 1);
      if (w == 4) {
        // all warps have unpacked step i (and so have passed their wait for step
        // i - 2) before step i - 1's end can be announced
        bool ok = bar_wait(smem_addr(&kv_full[st]), (i >> 1) & 1, &give_up, p.a.status);
        if (i) {
          second(i - 1);
          ok = bar_wait(smem_addr(&pv_done), (i - 1) & 1, &give_up, p.a.status) && ok;  // the weights' place is free
        }
        if (note[i % kList] & kFirst) {
          ok = bar_wait(smem_addr(&q_full), n_runs & 1, &give_up, p.a.status) && ok;
          ++n_runs;
        }
        after_sync();
        if (lane == 0 && ok && !give_up) {
          const uint32_t q = smem_addr(q_op), k = smem_addr(kv_op + st * 2 * W::KVB);
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ss(tm + 64 * g, operand(q + g * CT * 128 + kk * 32), operand(k + g * SP * 128 + kk * 32), id_qk, kk);
          commit(smem_addr(&s_full));
        }
        __syncwarp();
      }
    }
    if (w == 4 && n_steps) second(n_steps - 1);
  } else {  // ---- a query column each
    const uint32_t my = tm + ((uint32_t)(32 * w) << 16);  // this warp's lanes
    uint32_t k = 0;
    for (bool more = n_steps > 0; more; more = run.next(p, CT, SP)) {
      const int seq = p.n_ctiles == 1 ? run.e : run.e / p.n_ctiles, j = run.e - seq * p.n_ctiles;
      const int col = j * CT + tid;
      const bool there = col < p.cols;
      const int row = there ? row_of(p, col) : 0, hd = run.head * p.gqa + (there ? col - row * p.gqa : 0);
      int len, nn;
      seq_extent(p.a, seq, len, nn);
      const int lim = there && row < nn ? max(0, len - nn + row + 1) : 0;  // positions that it sees
      {
        const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(p.q.p) + seq * p.q.seq + row * p.q.row + hd * p.q.head;
#pragma unroll 4
        for (int x = 0; x < HD / 8; ++x) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (there) v = *reinterpret_cast<const uint4*>(src + 8 * x);
          const uint4 y = make_uint4(pack2(low_f(v.x) * kUp, low_f(v.y) * kUp), pack2(high_f(v.x) * kUp, high_f(v.y) * kUp),
                                     pack2(low_f(v.z) * kUp, low_f(v.w) * kUp), pack2(high_f(v.z) * kUp, high_f(v.w) * kUp));
          const int g = x / 8, unit = x % 8;
          *reinterpret_cast<uint4*>(q_op + g * CT * 128 + tid * 128 + ((unit ^ (tid & 7)) << 4)) = y;
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive(smem_addr(&q_full));
      // running maximum (log2) and sum, the sum and the weights times 2^e where
      // V's scales are below cap = 2^(6 - e)
      float m = kLow, l = 0.f, cap = 0.f, e = 0.f;
      for (int t = run.t0; t < run.t1; ++t, ++k) {
        const int st = k & 1;
        bool ok = bar_wait(smem_addr(&kv_full[st]), (k >> 1) & 1, &give_up, p.a.status);
        ok = bar_wait(smem_addr(&s_full), k & 1, &give_up, p.a.status) && ok;
        after_sync();
        if (ok && !give_up) {
          const float* sc = scales + st * 2 * NG * SP;
          const int vis = min(lim - t * SP, note[k % kList] & (kFirst - 1));  // of the step's positions
          auto step = [&](auto cut_) {
            constexpr bool CUT = decltype(cut_)::value;
            float s[SP], mx = -INFINITY;
#pragma unroll
            for (int c = 0; c < SP; c += 16) {
              float a[NG][16];
#pragma unroll
              for (int g = 0; g < NG; ++g) tm_load16(my + 64 * g + c, a[g]);
#pragma unroll
              for (int g = 0; g < NG; ++g) tm_loaded(a[g]);
#pragma unroll
              for (int x = 0; x < 16; x += 4) {
                const float4 k0 = *reinterpret_cast<const float4*>(sc + c + x);
                s[c + x] = a[0][x] * k0.x, s[c + x + 1] = a[0][x + 1] * k0.y;
                s[c + x + 2] = a[0][x + 2] * k0.z, s[c + x + 3] = a[0][x + 3] * k0.w;
                if constexpr (NG == 2) {
                  const float4 k1 = *reinterpret_cast<const float4*>(sc + SP + c + x);
                  s[c + x] = fmaf(a[1][x], k1.x, s[c + x]), s[c + x + 1] = fmaf(a[1][x + 1], k1.y, s[c + x + 1]);
                  s[c + x + 2] = fmaf(a[1][x + 2], k1.z, s[c + x + 2]), s[c + x + 3] = fmaf(a[1][x + 3], k1.w, s[c + x + 3]);
                }
              }
#pragma unroll
              for (int x = 0; x < 16; ++x) {
                if (CUT && c + x >= vis) s[c + x] = -INFINITY;
                mx = fmaxf(mx, s[c + x]);
              }
            }
            const float top = fmaxf(top_vs[st][0], top_vs[st][1]);
            if (__any_sync(0xffffffffu, mx > m + kLazy || top > cap)) {
              float move = 1.f;
              if (top > cap) {  // the next power of two, and 2^3 of room
                const int b = min(max((int)(__float_as_uint(top) >> 23) + 4, 40), 200);  // 2^e stays within 2^+-93
                const float ne = (float)(133 - b);
                move = exp2_fast(ne - e);
                cap = __uint_as_float((uint32_t)b << 23);
                e = ne;
              }
              const float nm = fmaxf(m, mx), f = exp2_fast(m - nm) * move;
              m = nm;
              l *= f;
              if (t > run.t0) {
#pragma unroll 1
                for (int c = 0; c < NG * 64; c += 16) {
                  float o[16];
                  uint32_t b[16];
                  tm_load16(my + 64 * NG + c, o);
                  tm_loaded(o);
#pragma unroll
                  for (int x = 0; x < 16; ++x) b[x] = __float_as_uint(o[x] * f);
                  tm_store16(my + 64 * NG + c, b);
                }
              }
            }
            const float sub = m - e;
#pragma unroll
            for (int c = 0; c < SP; c += 32) {
              uint32_t b[NG][16];
#pragma unroll
              for (int x = 0; x < 32; x += 4) {
                float w4[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  w4[y] = exp2_fast(s[c + x + y] - sub);
                  l += w4[y];
                }
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                  const float4 v = *reinterpret_cast<const float4*>(sc + (NG + g) * SP + c + x);
                  float z[4] = {w4[0] * v.x, w4[1] * v.y, w4[2] * v.z, w4[3] * v.w};
                  if constexpr (CUT) {  // whatever the scale of what is not seen
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                      if (c + x + y >= vis) z[y] = 0.f;
                  }
                  b[g][x / 2] = pack2h(z[0], z[1]);
                  b[g][x / 2 + 1] = pack2h(z[2], z[3]);
                }
              }
#pragma unroll
              for (int g = 0; g < NG; ++g) tm_store16(my + 32 * g + c / 2, b[g]);
            }
          };
          if (__all_sync(0xffffffffu, vis >= SP)) step(std::false_type());
          else step(std::true_type());
          tm_stored();
        }
        before_sync();
        __syncwarp();
        if (lane == 0) arrive(smem_addr(&p_full));
      }
      // ---- the run's end: this column's sums, dimensions put back in order
      bar_wait(smem_addr(&pv_done), (k - 1) & 1, &give_up, p.a.status);
      after_sync();
      const bool whole = run.t0 == 0 && run.t1 == run.nt;
      const float undo = kCode * exp2f(-e);
      float f = whole ? (l == 0.f ? 0.f : kCode / l) : undo;
      if (give_up) f = NAN;
      float* part = p.part + ((size_t)part_slot(blockIdx.x, run.t0) * CT + tid) * (HD + 4);
      __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(const_cast<void*>(p.out.p)) + seq * p.out.seq + row * p.out.row +
                           hd * p.out.head;
#pragma unroll 1
      for (int c = 0; c < HD; c += 16) {
        float o[16];
        tm_load16(my + 64 * NG + c, o);
        tm_loaded(o);
        if (!there) continue;
#pragma unroll
        for (int x = 0; x < 16; ++x) o[x] *= f;
#pragma unroll
        for (int x = 0; x < 16; x += 8) {  // 0 2 1 3 4 6 5 7
          if (whole) {
            *reinterpret_cast<uint4*>(dst + c + x) = make_uint4(pack2(o[x], o[x + 2]), pack2(o[x + 1], o[x + 3]),
                                                                pack2(o[x + 4], o[x + 6]), pack2(o[x + 5], o[x + 7]));
          } else {
            *reinterpret_cast<float4*>(part + c + x) = make_float4(o[x], o[x + 2], o[x + 1], o[x + 3]);
            *reinterpret_cast<float4*>(part + c + x + 4) = make_float4(o[x + 4], o[x + 6], o[x + 5], o[x + 7]);
          }
        }
      }
      const float sum = l * exp2f(-e);
      if (there) {
        if (!whole) *reinterpret_cast<float2*>(part + HD) = make_float2(m, give_up ? NAN : sum);
        else if (p.lse)
          p.lse[((size_t)seq * p.a.rows + row) * p.n_heads + hd] =
              sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.69314718055994530942f;
      }
      if (tid == 0 && run.t0 == 0)
        p.item[(size_t)run.e * p.a.n_kv_heads + run.head] =
            make_longlong2(whole ? -1 : run.base + (long long)run.head * (run.nt + kOver), blockIdx.x);
      before_sync();  // the next run's products overwrite the sums
    }
  }
  before_sync();
  __syncthreads();
  if (w == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "n"(W::TM));
}

template <int HD>
WideKernel info() {
  return {reinterpret_cast<const void*>(&k_kv4_wide<HD>), Wide<HD>::CT, Wide<HD>::SP, Wide<HD>::SMEM, 2, 256};
}

}  // namespace

WideKernel kv4_wide_kernel(int head_dim) { return head_dim == 64 ? info<64>() : info<128>(); }

}  // namespace mk
