// What the operators on the 16-bit paged cache share (mk_paged.cu,
// mk_paged_attention.cu, mk_paged_evict.cu).  Arguments are those of the 4-bit
// cache's calls; a pool of one layer is bf16 [page][K|V][kv head][128][head_dim].
#pragma once
#include "mk_kv4.cuh"

namespace mk {

// Masses of the cached positions: [n_seqs][n_kv_heads][128 * max_pages].
struct PagedMass {
  float* p;
  long long seq, head;  // strides in elements
  float decay;
};

// Row of a page's slot in the pool taken as rows of head_dim (held to 31 bits by the entry points).
__device__ __forceinline__ int paged_row(const Kv4Args& a, int page, int kv, int head, int p) {
  return ((page * 2 + kv) * a.n_kv_heads + head) * kPageTokens + p % kPageTokens;
}
template <int HD>
__device__ __forceinline__ __nv_bfloat16* paged_at(const Kv4Args& a, int row) {
  return reinterpret_cast<__nv_bfloat16*>(a.pool) + (size_t)row * HD;
}

// Every kernel here begins behind the stream's last one as soon as that has no block left to
// start, and waits for its end before it reads or writes memory (so a kernel's start, about 2 us of
// a short call, overlaps what runs before it).  The next one may begin only then: what it reads before its own wait (the
// join reads the lengths) must be final.
__device__ __forceinline__ void behind() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
inline cudaError_t launch(const void* kernel, unsigned grid, int block, size_t smem, cudaStream_t st, void** args, int cluster = 0,
                          unsigned grid_y = 1) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(grid, grid_y);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

// Host checks of a description (*empty: the call has no row), and of masses.
int paged_check_cache(const mk_paged_cache* c, bool* empty);
int paged_check_mass(const mk_paged_mass* m, const mk_paged_cache* c, const char* what);

}  // namespace mk
