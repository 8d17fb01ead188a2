// The 4-bit paged cache's format and arguments, shared by the store and load
// (mk_kv4.cu) and the attention (mk_kv4_attention.cu).
#pragma once
#include <cuda_bf16.h>

#include "mk_kv4_host.h"

namespace mk {

constexpr int kTile = 64;    // positions of a tile
constexpr int kGroup = 64;   // values that share a scale

// A tile of one kv head: K codes, K scales, V codes, V scales.
template <int HD>
struct Tile {
  static constexpr int ROW = HD / 2;             // code bytes of a row
  static constexpr int NG = HD / kGroup;         // scales of a row
  static constexpr int CODES = kTile * ROW;
  static constexpr int SCALES = kTile * NG * 2;
  static constexpr int V = CODES + SCALES;       // offset of the V half
  static constexpr int BYTES = 2 * V;
  static constexpr int RECORD = kPageTokens / kTile * BYTES;
};

__device__ __forceinline__ void refuse(int32_t* status) {
  if (status) atomicCAS(status, 0, MK_ERR_DEVICE_INDEX);
}

// Length and new rows of a sequence, held to what the table and the call can hold.
__device__ __forceinline__ void seq_extent(const Kv4Args& a, int s, int& len, int& nn) {
  len = a.lengths[s];
  nn = a.n_new ? a.n_new[s] : a.rows;
  const long long most = (long long)a.max_pages * kPageTokens;
  if (len < 0 || len > most || nn < 0 || nn > a.rows) refuse(a.status);
  len = (int)max(0ll, min((long long)len, most));
  nn = max(0, min(nn, a.rows));
}

__device__ __forceinline__ const int32_t* table_row(const Kv4Args& a, int s) {
  return a.table + (size_t)(a.slots ? a.slots[s] : s) * a.table_stride;
}

// The page of position p of sequence s, or -1.
__device__ __forceinline__ int page_of(const Kv4Args& a, int s, int p) {
  const int page = table_row(a, s)[p / kPageTokens];
  if (page >= 0 && page < a.n_pages) return page;
  refuse(a.status);
  return -1;
}

template <int HD>
__device__ __forceinline__ uint8_t* tile_of(const Kv4Args& a, int page, int head, int p) {
  return a.pool + ((size_t)page * a.n_kv_heads + head) * Tile<HD>::RECORD + (size_t)(p % kPageTokens / kTile) * Tile<HD>::BYTES;
}

// Host checks shared by the entry points (mk_kv4.cu): of a cache description
// (*empty: the call has no row), and of rows.
int kv4_check_cache(const mk_kv4_cache* c, bool* empty);
int kv4_check_rows(const mk_kv4_rows* r, int dtype, const char* what);
Kv4Args kv4_args(const mk_kv4_cache& c);
Kv4Rows kv4_rows(const mk_kv4_rows& r);

}  // namespace mk
