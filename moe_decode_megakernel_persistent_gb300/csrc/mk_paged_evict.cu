// Eviction from the 16-bit paged cache: which positions of a (sequence, kv head)
// stay, and their moves.
//
// Which.  The keep - recent largest masses among the others are found by their
// bits (an order-preserving map to unsigned numbers): three passes count the next 11, 11
// and 10 bits of those that agree so far, and the digit is where the count from the top
// passes what is left to take.  That gives the least mass that stays and how many of its
// ties do; ties, free slots and late positions (kept ones at or above `keep`) are then
// numbered in order.  An item is a cluster of blocks, each with a run of the positions, which
// it holds in shared memory (read from the masses again in each pass, an item of 131071 took 64 us),
// and each of its threads a run of that, so that numbers are sums over the threads before (numbers by ballots of
// a warp's 32 positions took ten times the instructions); counts go through distributed shared memory.  Every block passes the same barriers whatever it reads, so that
// lengths written meanwhile give a wrong answer, not a hang.
//
// Moves.  Only late positions move, into free slots: never more rows than it takes, sources
// (>= keep) and destinations (< keep) are apart, and nothing is read after it is written.  The
// item's own blocks make them, from the lists of free slots and late positions in order; where there may be many, a second
// kernel of all SMs does.
//
// Bounds.  16 sequences of 256 to 8448 positions cut to 2048 (4 kv heads of 128) read and write 30 MB of K and V each, with the
// masses 9 us at the memory's rate, and take 30: 17 for the choice, a chain of three passes over shared memory with
// barriers of the cluster between them (28 % of the issue slots), and 10 for the moves.  64 sequences at a budget of 4096 take 15,
// nearly all of it the read of the masses and that chain.
#include <algorithm>
#include <climits>
#include <string>

#include "mk_paged_att.cuh"

namespace mk {
namespace {

constexpr int kSelWarps = 16, kSelThreads = 32 * kSelWarps, kBins = 4 * kSelThreads;  // four bins a thread
constexpr int kMostBlocks = 16;  // of an item's cluster
constexpr int kMostHeld = 96 * kSelThreads;  // positions that a block holds

struct EvictArgs {
  Kv4Args a;
  PagedMass mass, to;
  int32_t keep, recent, in_place;
  int32_t* kept;     // [n_seqs][n_kv_heads][keep]
  int32_t *free, *late;  // workspace, as kept: free slots and late positions in order
  int32_t* counts;   // workspace: moves of each item, where another kernel makes them
  int32_t* lengths;  // new ones
};

__device__ __forceinline__ int held_length(const Kv4Args& a, int s) {
  const int len = a.lengths[s];
  const long long most = (long long)a.max_pages * kPageTokens;
  if (len < 0 || len > most) refuse(a.status);
  return (int)max(0ll, min((long long)len, most));
}
// Unsigned numbers in the order of the masses; NaN above all, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  if (x != x) return 0xFFFFFFFFu;
  return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint32_t peer_addr(const void* p, int rank) {
  uint32_t y;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(y) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return y;
}
__device__ __forceinline__ int peer_load(const void* p, int rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(peer_addr(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ void peer_store(const void* p, int rank, int v) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(peer_addr(p, rank)), "r"(v) : "memory");
}

// Two numbers' sums over all threads of the cluster before this one, and the first one's over all.
struct Before {
  int2 warp[kSelWarps];
  int x, y;  // of the block
};
__device__ __forceinline__ int3 before(Before& b, int x, int y, int rank, int C) {
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int ix = x, iy = y;  // over the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int ux = __shfl_up_sync(0xffffffffu, ix, o), uy = __shfl_up_sync(0xffffffffu, iy, o);
    if (lane >= o) ix += ux, iy += uy;
  }
  if (lane == 31) b.warp[w] = make_int2(ix, iy);
  __syncthreads();
  int2 n = lane < kSelWarps ? b.warp[lane] : make_int2(0, 0);
  if (w == 0) {
    const int sx = __reduce_add_sync(0xffffffffu, n.x), sy = __reduce_add_sync(0xffffffffu, n.y);
    if (lane == 0) b.x = sx, b.y = sy;
  }
  if (C > 1) cluster_sync();
  else __syncthreads();
  if (lane >= w) n = make_int2(0, 0);
  const int px = lane < C ? peer_load(&b.x, lane) : 0;
  if (lane < rank) n.x += px, n.y += peer_load(&b.y, lane);
  return make_int3(__reduce_add_sync(0xffffffffu, n.x) + ix - x, __reduce_add_sync(0xffffffffu, n.y) + iy - y,
                   __reduce_add_sync(0xffffffffu, px));
}

// The moves of an item by warps `first`, `first` + 1 .. of `warps`, MV at a time: K in the first half of the lanes
// that a position's 4 * HD bytes take and V in the second.
template <int HD>
__device__ __forceinline__ void make_moves(const EvictArgs& p, int item, int seq, int head, int moves, int first, int warps) {
  constexpr int LP = HD / 4, LR = LP / 2, MV = 8;
  const int lane = threadIdx.x & 31, mine = lane / LP, word = lane % LR, kv = lane % LP / LR;
  const int half = p.a.n_kv_heads * kPageTokens;  // rows from K to V
  const int positions = p.a.max_pages * kPageTokens, keep = p.keep;
  const float* mass = p.mass.p + seq * p.mass.seq + head * p.mass.head;
  float* to = p.to.p + seq * p.to.seq + head * p.to.head;
  const int *free = p.free + (size_t)item * keep, *late = p.late + (size_t)item * keep;
  for (int r0 = first * MV; r0 < moves; r0 += warps * MV) {
    int from = -1, dst = -1;
    const int r = r0 + lane;
    if (lane < MV && r < moves) {
      const int src = __ldcg(&late[r]), slot = __ldcg(&free[r]);
      if (src >= 0 && src < positions && slot >= 0 && slot < min(keep, positions)) {  // (always, but for lengths that change under the call)
        p.kept[(size_t)item * keep + slot] = src;
        to[slot] = mass[src];
        from = page_of(p.a, seq, src);
        dst = page_of(p.a, seq, slot);
        if (from >= 0 && dst >= 0) {
          from = paged_row(p.a, from, 0, head, src);
          dst = paged_row(p.a, dst, 0, head, slot);
        } else {
          from = -1;
        }
      }
    }
    uint4 x[MV * LP / 32];
    int d[MV * LP / 32];
#pragma unroll
    for (int i = 0; i < MV * LP / 32; ++i) {
      const int pick = i * (32 / LP) + mine, f = __shfl_sync(0xffffffffu, from, pick);
      d[i] = __shfl_sync(0xffffffffu, dst, pick);
      if (f < 0) d[i] = -1;
      else x[i] = reinterpret_cast<const uint4*>(paged_at<HD>(p.a, f + kv * half))[word];
    }
#pragma unroll
    for (int i = 0; i < MV * LP / 32; ++i)
      if (d[i] >= 0) reinterpret_cast<uint4*>(paged_at<HD>(p.a, d[i] + kv * half))[word] = x[i];
  }
}

template <int HD>
__global__ void __launch_bounds__(kSelThreads) k_evict(const __grid_constant__ EvictArgs p, int C) {
  extern __shared__ __align__(16) uint32_t held[];  // of a thread's PT positions: masses as unsigned numbers, later what becomes of them
  __shared__ __align__(16) int hist[2][kBins], total[kBins];
  __shared__ Before cnt[2];
  __shared__ int scan[kSelWarps], s_digit, s_left, s_ties;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int item = blockIdx.x / C, rank = blockIdx.x - item * C;
  const int seq = item / p.a.n_kv_heads, head = item - seq * p.a.n_kv_heads;
  behind();
  const int len = held_length(p.a, seq), keep = p.keep;
  const bool all = len <= keep;
  const int others = max(0, len - p.recent), positions = p.a.max_pages * kPageTokens;
  const float* mass = p.mass.p + seq * p.mass.seq + head * p.mass.head;
  float* to = p.to.p + seq * p.to.seq + head * p.to.head;
  int* kept = p.kept + (size_t)item * keep;
  // Threads have runs of PT positions, PT | 1 words apart (an odd number: 32 threads' words are in 32 banks).
  const int PT = max(4, ((len + C - 1) / C + kSelThreads - 1) / kSelThreads), apart = PT | 1, per = PT * kSelThreads;
  const uint32_t magic = (uint32_t)((0x100000000ull + PT - 1) / PT);  // i / PT for i < 2^16 (PT <= 96)
  auto at = [&](int i) { return i + (int)__umulhi((uint32_t)i, magic) * (apart - PT); };
  const int lo = (int)min((long long)len, (long long)rank * per), n = min(len - lo, per);
  const int i0 = min(n, tid * PT), i1 = min(n, i0 + PT);  // this thread's run
  const uint32_t* mine = held + tid * apart;
#pragma unroll 4
  for (int i = tid; i < n; i += kSelThreads) held[at(i)] = key_of(mass[lo + i]);
  for (int i = tid; i < 2 * kBins; i += kSelThreads) hist[0][i] = 0;
  if (tid == 0) s_digit = s_left = s_ties = 0;
  __syncthreads();

  // ---- the least mass that stays (its bits), and how many of its ties do
  uint32_t least = 0;
  int left = all ? 0 : keep - p.recent;
  const int m_others = min(n, max(0, others - lo));
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    int* h = hist[pass & 1];
#pragma unroll 4
    for (int i = i0; i < min(i1, m_others); ++i) {
      const uint32_t k = mine[i - i0];
      if (pass == 0 || k >> (shift + bits) == least >> (shift + bits)) atomicAdd(&h[k >> shift & ((1u << bits) - 1)], 1);
    }
    // Each block adds a part of the bins over the cluster and gives every block the sums (all bins of all blocks read
    // by every block: 2.4 us a pass in a cluster of 8, 11 in one of 16).
    if (C > 1) {
      cluster_sync();
      const int seg = kBins / C;
      for (int i = rank * seg + tid; i < (rank + 1) * seg; i += kSelThreads) {
        int sum = 0;
        for (int r0 = 0; r0 < C; r0 += 8) {  // (eight reads on their way)
          int v[8];
#pragma unroll
          for (int r = 0; r < 8; ++r) v[r] = r0 + r < C ? peer_load(&h[i], r0 + r) : 0;
#pragma unroll
          for (int r = 0; r < 8; ++r) sum += v[r];
        }
        for (int r = 0; r < C; ++r) peer_store(&total[i], r, sum);
      }
      cluster_sync();
    } else {
      __syncthreads();
    }
    // four bins a thread, from the top
    const int4 c4 = *reinterpret_cast<const int4*>((C > 1 ? total : h) + kBins - 4 - 4 * tid);
    const int c[4] = {c4.w, c4.z, c4.y, c4.x};
    const int sum = (c[0] + c[1]) + (c[2] + c[3]);
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) scan[w] = incl;
    __syncthreads();
    const int whole = lane < w ? scan[lane] : 0;
    incl += __reduce_add_sync(0xffffffffu, whole);
    int above = incl - sum;
    if (above < left && left <= incl) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (above < left && left <= above + c[i]) {
          s_digit = kBins - 1 - 4 * tid - i;
          s_left = left - above;
          s_ties = c[i];
        }
        above += c[i];
      }
    }
    if (pass == 1)  // the third pass counts where the first did, which all blocks have read by now
      for (int i = tid; i < kBins; i += kSelThreads) hist[0][i] = 0;
    __syncthreads();
    least |= (uint32_t)s_digit << shift;
    left = s_left;
  }

  // ---- numbers in order
  // Where all ties stay, or none, they need no number.
  const bool some = left > 0 && left < s_ties;
  int ties = 0;
  if (some)
    for (int i = i0; i < min(i1, m_others); ++i) ties += mine[i - i0] == least;
  const int tie0 = before(cnt[0], ties, 0, rank, C).x;
  const uint32_t above = left > 0 ? least : 0xFFFFFFFFu;  // (left = 0: of the others none stays, whatever its mass)
  auto stays = [&](int i, int& tie) {
    if (all || i >= m_others) return true;
    const uint32_t k = mine[i - i0];
    if (some && k == least) return tie++ < left;
    return left > 0 && k >= above;
  };
  int n_free = 0, n_late = 0, tie = tie0;
  const int below = keep - lo;  // of the block's positions
  for (int i = i0; i < i1; ++i) {
    const bool s = stays(i, tie);
    n_free += i < below && !s;
    n_late += i >= below && s;
  }
  const int3 at0 = before(cnt[1], n_free, n_late, rank, C);
  const int moves = min(at0.z, keep);
  // what becomes of a position: its number among the free slots or late positions, or kStay
  constexpr uint32_t kStay = 0xFFFFFFFFu, kGone = 0xFFFFFFFEu;
  int nf = at0.x, nl = at0.y;
  tie = tie0;
  for (int i = i0; i < i1; ++i) {
    const bool s = stays(i, tie);
    held[tid * apart + i - i0] = i < below ? s ? kStay : (uint32_t)nf++ : s ? (uint32_t)nl++ : kGone;
  }
  __syncthreads();
  int *free = p.free + (size_t)item * keep, *late = p.late + (size_t)item * keep;
#pragma unroll 4
  for (int i = tid; i < n; i += kSelThreads) {
    const int q = lo + i;
    const uint32_t x = held[at(i)];
    if (q < keep) {
      if (x == kStay) {
        kept[q] = q;
        if (!p.in_place) to[q] = mass[q];
      } else if (x < (uint32_t)keep) {
        free[x] = q;
      }
    } else {
      if (x < (uint32_t)keep) late[x] = q;
      if (!p.in_place) to[q] = 0.f;
    }
  }
  for (uint32_t q = len + rank * kSelThreads + tid; q < (uint32_t)keep; q += C * kSelThreads) kept[q] = -1;  // (keep may be 2^31 - 1)
  if (!p.in_place)
    for (int q = len + rank * kSelThreads + tid; q < positions; q += C * kSelThreads) to[q] = 0.f;
  if (C > 1) cluster_sync();  // the lists are whole, and no block reads another's shared memory any more
  else __syncthreads();

  if (p.counts) {  // the moves are another kernel's
    if (rank == 0 && tid == 0) p.counts[item] = moves;
  } else {
    make_moves<HD>(p, item, seq, head, moves, rank * kSelWarps + w, C * kSelWarps);
  }
  if (p.lengths != p.a.lengths && head == 0 && rank == 0 && tid == 0) p.lengths[seq] = min(len, keep);
}

template <int HD>
__global__ void __launch_bounds__(256) k_evict_moves(const __grid_constant__ EvictArgs p, int blocks) {
  behind();
  const int item = blockIdx.x / blocks, seq = item / p.a.n_kv_heads, head = item - seq * p.a.n_kv_heads;
  make_moves<HD>(p, item, seq, head, min(p.counts[item], p.keep), (blockIdx.x - item * blocks) * 8 + (threadIdx.x >> 5), blocks * 8);
}

// New lengths in the place of the old ones, once all blocks have read those.
__global__ void __launch_bounds__(256) k_evict_lengths(const __grid_constant__ EvictArgs p) {
  behind();
  const int s = blockIdx.x * 256 + threadIdx.x;
  if (s < p.a.n_seqs) p.lengths[s] = min(held_length(p.a, s), p.keep);
}

int check(const mk_paged_cache* c, int keep, bool* empty) {
  if (!c) return host_fail(MK_ERR_INVALID_ARG, "cache is NULL");
  mk_paged_cache one = *c;
  one.rows = 1;  // not used
  if (int r = paged_check_cache(&one, empty)) return r;
  if (keep < 1) return host_fail(MK_ERR_INVALID_ARG, "keep must be >= 1");
  if ((long long)c->n_seqs * c->n_kv_heads * keep > INT_MAX)
    return host_fail(MK_ERR_INVALID_ARG, "n_seqs x n_kv_heads x keep passes 31 bits");
  if (c->max_pages > kMostBlocks * kMostHeld / kPageTokens)
    return host_fail(MK_ERR_UNSUPPORTED, "eviction takes tables of at most 6144 pages (786432 positions)");
  return MK_OK;
}

size_t bytes_of(const mk_paged_cache& c, int keep) { return (size_t)c.n_seqs * c.n_kv_heads * (2 * (size_t)keep + 1) * sizeof(int32_t); }

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" MK_API size_t mk_paged_evict_bytes(const mk_paged_cache* c, int32_t keep) {
  bool empty = false;
  return check(c, keep, &empty) || empty ? 0 : bytes_of(*c, keep);
}

extern "C" MK_API int mk_paged_evict(const mk_paged_cache* c, const mk_paged_mass* mass, int32_t keep, int32_t recent,
                                     int32_t* kept, int32_t* new_lengths, const mk_paged_mass* new_mass, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  host_clear_error();
  bool empty = false;
  if (int r = check(c, keep, &empty)) return r;
  if (recent < 0 || recent > keep) return host_fail(MK_ERR_INVALID_ARG, "recent must lie in [0, keep]");
  if (empty) return MK_OK;
  if (int r = paged_check_mass(mass, c, "mass")) return r;
  if (int r = paged_check_mass(new_mass, c, "new_mass")) return r;
  if (!kept || !new_lengths) return host_fail(MK_ERR_INVALID_ARG, "kept or new_lengths is NULL");
  const size_t need = bytes_of(*c, keep);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u) || workspace_bytes < need)
    return host_fail(MK_ERR_INVALID_ARG, "workspace is NULL, not 16-byte aligned or smaller than mk_paged_evict_bytes");
  EvictArgs p;
  p.a = kv4_args(*c);
  p.mass = {mass->data, mass->seq_stride, mass->head_stride, 1.f};
  p.to = {new_mass->data, new_mass->seq_stride, new_mass->head_stride, 1.f};
  p.in_place = mass->data == new_mass->data;
  if (p.in_place && ((c->n_seqs > 1 && mass->seq_stride != new_mass->seq_stride) ||
                     (c->n_kv_heads > 1 && mass->head_stride != new_mass->head_stride)))
    return host_fail(MK_ERR_INVALID_ARG, "new_mass begins with mass but has other strides");
  p.keep = keep;
  p.recent = recent;
  p.kept = kept;
  p.free = static_cast<int32_t*>(workspace);
  p.late = p.free + (size_t)c->n_seqs * c->n_kv_heads * keep;
  p.lengths = new_lengths;
  cudaStream_t st = (cudaStream_t)stream;
  const int items = c->n_seqs * c->n_kv_heads, positions = c->max_pages * kPageTokens;
  if ((long long)items * ((positions + 255) / 256) > INT_MAX || (long long)items * kMostBlocks > INT_MAX)
    return host_fail(MK_ERR_INVALID_ARG, "n_seqs x n_kv_heads x max_pages is too large");
  // Blocks of an item: while they run at once (two an SM) and have 2048 positions each, or until they hold theirs.
  const int sms = device_sms();
  int C = 1;
  while (C < kMostBlocks && (((long long)items * C * 2 <= 2 * sms && positions / (2 * C) >= 2048) || positions > C * kMostHeld)) C *= 2;
  const int PT = std::max(4, ((positions + C - 1) / C + kSelThreads - 1) / kSelThreads);
  const size_t smem = (size_t)kSelThreads * (PT + 1) * sizeof(uint32_t);
  const void* f = c->head_dim == 64 ? reinterpret_cast<const void*>(&k_evict<64>) : reinterpret_cast<const void*>(&k_evict<128>);
  cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelThreads * (kMostHeld / kSelThreads + 1) * 4);
  if (e == cudaSuccess && C > 8) e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  void* args[] = {&p, &C};
  // As many moves as the table and keep allow: few are made by the item's own blocks, many levelled over all SMs by a kernel of
  // their own, unless the items fill the SMs themselves (keep 4096; own blocks and a second kernel, us: 4 items of 256 moves
  // 15.5 and 16.4, 512 17.7 and 16.7; 16 of 512 18.0 and 18.5, 1024 22.1 and 22.2, 2048 30.8 and 22.6; 64 of 1024 26.5 and 28.1,
  // 2048 47.3 and 44.4; 256 of 256 24.1 and 25.9, 2048 110 and 119).
  const int few = items >= sms ? INT_MAX : items >= 16 ? 1024 : 256;
  p.counts = std::min(keep, positions - keep) > few ? p.late + (size_t)items * keep : nullptr;
  if (e == cudaSuccess) e = launch(f, (unsigned)items * C, kSelThreads, smem, st, args, C);
  if (e == cudaSuccess && p.counts) {
    int blocks = (8 * sms + items - 1) / items;
    void* margs[] = {&p, &blocks};
    e = launch(c->head_dim == 64 ? reinterpret_cast<const void*>(&k_evict_moves<64>) : reinterpret_cast<const void*>(&k_evict_moves<128>),
               (unsigned)items * blocks, 256, 0, st, margs);
  }
  if (e == cudaSuccess && new_lengths == c->lengths)
    e = launch(reinterpret_cast<const void*>(&k_evict_lengths), (unsigned)(c->n_seqs + 255) / 256, 256, 0, st, args);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return host_fail(MK_ERR_CUDA, (std::string("paged evict: ") + cudaGetErrorString(e)).c_str());
  }
  return MK_OK;
}
