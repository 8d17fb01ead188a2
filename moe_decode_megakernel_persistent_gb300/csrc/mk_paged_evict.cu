// Eviction from the 16-bit paged cache: which positions of a (sequence, kv head)
// stay, and their moves.
//
// Which.  The keep - recent largest masses among the others are found by their
// bits (an order-preserving map to unsigned numbers): three passes over the masses
// count the next 11, 11 and 10 bits of those that agree so far, and the digit is
// where the count from the top passes what is left to take.  That gives the least
// mass that stays and how many of its ties do; ties, free slots and late positions
// (kept ones at or above `keep`) are then numbered in order.  An item is a cluster
// of blocks, each with a run of the positions and each of its warps a run of that,
// so that numbers are sums over the warps before; counts go through distributed
// shared memory.  Every block passes the same barriers whatever it reads, so that lengths
// written meanwhile give a wrong answer, not a hang.
//
// Moves.  Only late positions move, into free slots: never more rows than it takes, sources
// (>= keep) and destinations (< keep) are apart, and nothing is read after it is written.
#include <algorithm>
#include <climits>
#include <string>

#include "mk_paged.cuh"

namespace mk {
namespace {

constexpr int kSelWarps = 16, kSelThreads = 32 * kSelWarps, kBins = 2048;

struct EvictArgs {
  Kv4Args a;
  PagedMass mass, to;
  int32_t keep, recent, in_place;
  int32_t* kept;     // [n_seqs][n_kv_heads][keep]
  int32_t* late;     // workspace, as kept: late positions in order
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
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
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

// The sum over all warps of the cluster before this one, of a number of each warp.
struct Before {
  int warp[kSelWarps], block;
};
__device__ __forceinline__ int before(Before& b, int n, int rank, int C) {
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) b.warp[w] = n;
  __syncthreads();
  if (threadIdx.x == 0) {
    int s = 0;
    for (int i = 0; i < kSelWarps; ++i) s += b.warp[i];
    b.block = s;
  }
  cluster_sync();
  int s = lane < w ? b.warp[lane] : 0;
  if (lane < rank && lane < C) s += peer_load(&b.block, lane);
  return __reduce_add_sync(0xffffffffu, s);
}

__global__ void __launch_bounds__(kSelThreads) k_evict_select(const __grid_constant__ EvictArgs p, int C) {
  __shared__ int hist[kBins], total[kBins];
  __shared__ Before cnt[3];
  __shared__ int scan[kSelWarps], s_digit, s_left;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int item = blockIdx.x / C, rank = blockIdx.x - item * C;
  const int seq = item / p.a.n_kv_heads, head = item - seq * p.a.n_kv_heads;
  const int len = held_length(p.a, seq), keep = p.keep;
  const bool all = len <= keep;
  const int others = max(0, len - p.recent);
  const float* mass = p.mass.p + seq * p.mass.seq + head * p.mass.head;
  int* kept = p.kept + (size_t)item * keep;
  int* late = p.late + (size_t)item * keep;
  // this warp's run of the positions
  const int per = ((len + C * kSelWarps - 1) / (C * kSelWarps) + 31) & ~31;
  const int lo = (int)min((long long)len, (long long)(rank * kSelWarps + w) * per), hi = min(len, lo + per);

  // ---- the least mass that stays (its bits), and how many of its ties do
  uint32_t least = 0;
  int left = all ? 0 : keep - p.recent;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
    if (tid == 0) s_digit = s_left = 0;
    __syncthreads();
    for (int q = lo + lane; q < hi && q < others; q += 32) {
      const uint32_t k = key_of(mass[q]);
      if (pass == 0 || k >> (shift + bits) == least >> (shift + bits)) atomicAdd(&hist[k >> shift & ((1u << bits) - 1)], 1);
    }
    cluster_sync();
    // each block adds a part of the bins over the cluster and gives every block the sums
    const int seg = kBins / C;
    for (int i = tid; i < seg; i += kSelThreads) {
      int s = 0;
      for (int r = 0; r < C; ++r) s += peer_load(&hist[rank * seg + i], r);
      for (int r = 0; r < C; ++r) peer_store(&total[rank * seg + i], r, s);
    }
    cluster_sync();
    int n[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) sum += n[i] = total[kBins - 1 - 4 * tid - i];
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) scan[w] = incl;
    __syncthreads();
    for (int i = 0; i < w; ++i) incl += scan[i];
    int above = incl - sum;
    if (above < left && left <= incl) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (above < left && left <= above + n[i]) {
          s_digit = kBins - 1 - 4 * tid - i;
          s_left = left - above;
        }
        above += n[i];
      }
    }
    __syncthreads();
    least |= (uint32_t)s_digit << shift;
    left = s_left;
    __syncthreads();
  }

  // ---- numbers in order
  // whether position q stays, of the warp's next 32; `tie`: ties before them
  auto stays = [&](int q, int& tie) {
    bool t = false, s = q < hi;
    if (s && !all && q < others) {
      const uint32_t k = key_of(mass[q]);
      t = k == least;
      s = k > least && p.keep > p.recent;
    }
    const uint32_t ties = __ballot_sync(0xffffffffu, t);
    if (t) s = tie + __popc(ties & ((1u << lane) - 1)) < left;
    tie += __popc(ties);
    return s;
  };
  int n_tie = 0;
  for (int q0 = lo; q0 < hi; q0 += 32) stays(q0 + lane, n_tie);
  const int tie0 = before(cnt[0], n_tie, rank, C);
  int n_free = 0, n_late = 0, tie = tie0;
  for (int q0 = lo; q0 < hi; q0 += 32) {
    const int q = q0 + lane;
    const bool s = stays(q, tie);
    n_free += __popc(__ballot_sync(0xffffffffu, q < hi && q < keep && !s));
    n_late += __popc(__ballot_sync(0xffffffffu, q >= keep && s));
  }
  const int free0 = before(cnt[1], n_free, rank, C), late0 = before(cnt[2], n_late, rank, C);
  tie = tie0;
  for (int q0 = lo, nl = late0; q0 < hi; q0 += 32) {
    const int q = q0 + lane;
    const bool s = stays(q, tie), l = s && q >= keep;
    const uint32_t ls = __ballot_sync(0xffffffffu, l);
    if (s && q < keep) kept[q] = q;
    const int at = nl + __popc(ls & ((1u << lane) - 1));
    if (l && at < keep) late[at] = q;
    nl += __popc(ls);
  }
  for (int q = len + rank * kSelThreads + tid; q < keep; q += C * kSelThreads) kept[q] = -1;
  cluster_sync();
  tie = tie0;
  for (int q0 = lo, nf = free0; q0 < hi && q0 < keep; q0 += 32) {
    const int q = q0 + lane;
    const bool s = stays(q, tie), f = q < hi && q < keep && !s;
    const uint32_t fs = __ballot_sync(0xffffffffu, f);
    const int at = nf + __popc(fs & ((1u << lane) - 1));
    if (f) kept[q] = __ldcg(&late[at]);
    nf += __popc(fs);
  }
  cluster_sync();  // no block leaves while others read its shared memory
}

// A warp takes 32 slots of an item: their masses, then the rows that move, K in the first
// half of the lanes that a position's 4 * HD bytes take and V in the second.
template <int HD>
__global__ void __launch_bounds__(256) k_evict_move(const __grid_constant__ EvictArgs p, int width, int chunks) {
  constexpr int LP = HD / 4, LR = LP / 2;  // lanes of a move, of a row
  const int item = blockIdx.x / chunks, lane = threadIdx.x & 31;
  const int s0 = ((blockIdx.x - item * chunks) * 8 + (threadIdx.x >> 5)) * 32;
  const int seq = item / p.a.n_kv_heads, head = item - seq * p.a.n_kv_heads;
  const int most = p.a.max_pages * kPageTokens;
  if (head == 0 && s0 == 0 && lane == 0) p.lengths[seq] = min(held_length(p.a, seq), p.keep);
  const int slot = s0 + lane;
  int src = slot < p.keep ? p.kept[(size_t)item * p.keep + slot] : -1;
  if (src >= most) src = -1;
  const float* mass = p.mass.p + seq * p.mass.seq + head * p.mass.head;
  float* to = p.to.p + seq * p.to.seq + head * p.to.head;
  if (slot < width && !(p.in_place && (src < 0 || src == slot))) to[slot] = src >= 0 ? mass[src] : 0.f;
  const bool moves = src >= 0 && src != slot && slot < most;
  int from = -1, dst = -1;
  if (moves) {
    from = page_of(p.a, seq, src);
    dst = page_of(p.a, seq, slot);
    if (from < 0 || dst < 0) {
      from = -1;
    } else {
      from = paged_row(p.a, from, 0, head, src);
      dst = paged_row(p.a, dst, 0, head, slot);
    }
  }
  const int half = p.a.n_kv_heads * kPageTokens;  // rows from K to V
  uint32_t todo = __ballot_sync(0xffffffffu, from >= 0);
  const int mine = lane / LP, word = lane % LR, kv = lane % LP / LR;
  while (todo) {
    uint4 x[4];
    int d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int pick = -1;
#pragma unroll
      for (int j = 0; j < 32 / LP; ++j) {
        const int b = __ffs(todo) - 1;
        if (j == mine) pick = b;
        if (b >= 0) todo &= todo - 1;
      }
      const int f = __shfl_sync(0xffffffffu, from, max(pick, 0));
      d[i] = __shfl_sync(0xffffffffu, dst, max(pick, 0));
      if (pick < 0) d[i] = -1;
      else x[i] = reinterpret_cast<const uint4*>(paged_at<HD>(p.a, f + kv * half))[word];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (d[i] >= 0) reinterpret_cast<uint4*>(paged_at<HD>(p.a, d[i] + kv * half))[word] = x[i];
  }
}

int check(const mk_paged_cache* c, int keep, bool* empty) {
  if (!c) return host_fail(MK_ERR_INVALID_ARG, "cache is NULL");
  mk_paged_cache one = *c;
  one.rows = 1;  // not used
  if (int r = paged_check_cache(&one, empty)) return r;
  if (keep < 1) return host_fail(MK_ERR_INVALID_ARG, "keep must be >= 1");
  if ((long long)c->n_seqs * c->n_kv_heads * keep > INT_MAX)
    return host_fail(MK_ERR_INVALID_ARG, "n_seqs x n_kv_heads x keep passes 31 bits");
  if (c->max_pages > INT_MAX / kPageTokens / 2) return host_fail(MK_ERR_INVALID_ARG, "max_pages is too large");
  return MK_OK;
}

size_t bytes_of(const mk_paged_cache& c, int keep) { return (size_t)c.n_seqs * c.n_kv_heads * keep * sizeof(int32_t); }

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
  p.late = static_cast<int32_t*>(workspace);
  p.lengths = new_lengths;
  cudaStream_t st = (cudaStream_t)stream;
  const int items = c->n_seqs * c->n_kv_heads, positions = c->max_pages * kPageTokens;
  int C = 1;
  while (C < 8 && (long long)items * C * 2 <= 304 && positions / (2 * C) >= 2048) C *= 2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)items * C);
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, k_evict_select, p, C);
  if (e == cudaSuccess) {
    const int width = p.in_place ? std::min(keep, positions) : positions;
    const int chunks = (std::max(width, std::min(keep, positions)) + 255) / 256;
    if ((long long)items * chunks > INT_MAX) return host_fail(MK_ERR_INVALID_ARG, "n_seqs x n_kv_heads x max_pages is too large");
    if (c->head_dim == 64) k_evict_move<64><<<(unsigned)items * chunks, 256, 0, st>>>(p, width, chunks);
    else k_evict_move<128><<<(unsigned)items * chunks, 256, 0, st>>>(p, width, chunks);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return host_fail(MK_ERR_CUDA, (std::string("paged evict: ") + cudaGetErrorString(e)).c_str());
  }
  return MK_OK;
}
