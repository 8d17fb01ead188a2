// The 4-bit cache and the page moves as the library's own host code calls them.
#pragma once
#include "mk_internal.h"

namespace mk {

// Lengths and block-table rows of a step's sequences, entered in device arrays
// for the 4-bit cache's kernels (mk_kv.cu).
struct StepSeqs {
  int32_t n;
  int32_t len[kMaxBatch], slot[kMaxBatch];
};
int launch_step_seqs(const StepSeqs& a, int32_t* len_dev, int32_t* slot_dev, cudaStream_t st);

// Page moves of every layer of a pool [n_layers][n_pages][page_bytes]
// (mk_pages.cu); the caller has checked that no page is written twice or both
// read and written.
int launch_page_copy(void* pool, int n_layers, int n_pages, size_t page_bytes, const int32_t* src, const int32_t* dst,
                     int n, cudaStream_t st);

// The 4-bit cache (mk_kv4.cu, mk_kv4_attention.cu).  What the C ABI's
// mk_kv4_cache describes, with two things more that a context needs: the rows
// of its block table that the sequences have, and a bound of the lengths below
// the table's width (max_pages pages), which sizes the work.
struct Kv4Args {
  uint8_t* pool;
  const int32_t* table;
  const int32_t* lengths;
  const int32_t* n_new;
  int32_t* status;
  int32_t n_pages, n_kv_heads, n_seqs, max_pages, rows;
  const int32_t* slots;   // device int32 [n_seqs]: rows of the table, or null (row i)
  int32_t table_stride;   // entries of a table row
};
// Rows of heads: strides in elements.  slot: further elements for each position
// within a page (rows that lie where a bf16 page has them), or 0.
struct Kv4Rows {
  const void* p;
  long long seq, row, head, slot;
};
int kv4_store(const Kv4Args& a, int head_dim, const Kv4Rows& k, const Kv4Rows& v, int dtype, cudaStream_t st);
int kv4_load(const Kv4Args& a, int head_dim, const Kv4Rows& k, const Kv4Rows& v, int dtype, cudaStream_t st);
// Workspace of an attention call; false: too large a call.
bool kv4_attention_bytes(const Kv4Args& a, int head_dim, int n_heads, int dtype, size_t* bytes);
int kv4_attention(const Kv4Args& a, int head_dim, int n_heads, const Kv4Rows& q, int dtype, float scale,
                  const Kv4Rows& out, float* lse, void* ws, size_t ws_bytes, cudaStream_t st);

// A chunk's prefill over the 4-bit cache (PrefillArgs::kv null then): its pool
// [layer][page], and the device arrays that hold the chunk's end (start + n) and the
// sequence's block-table row.
struct PrefillKv4 {
  uint8_t* pool = nullptr;
  const int32_t *len = nullptr, *slot = nullptr;
};
int prefill_run(PrefillWork** work, const PrefillArgs& a, const PrefillKv4& kv4, cudaStream_t st);

}  // namespace mk
