// Sequences of the entry points for chunks of new tokens: argument checks, the
// sizes of a sequence, and the even split of the attention's work.
#pragma once
#include <stdint.h>

#include "kv_view.cuh"

namespace spec {

// Device arrays that describe the sequences of a call.
struct ChunkIndex {
  const int32_t* row_start;
  const int32_t* n_new;
  const int32_t* cache_len;
  int n_seq, n_rows, max_new;
  int capacity;                 // positions of a block table's row (or of another array, where that is shorter)
};

// Sequence s as the kernels take it: n positions before the chunk, m tokens in
// rows r0 ..; m = 0 for a padded sequence and for one whose sizes do not fit (bad).
struct ChunkSeq {
  int n, m, r0;
  bool bad;
  __device__ ChunkSeq(const ChunkIndex& X, int s) {
    n = X.cache_len[s];
    m = X.n_new[s];
    r0 = X.row_start[s];
    bad = m != 0 && (m < 0 || m > X.max_new || m > X.n_rows || n < 0 || n > X.capacity - m || r0 < 0 || r0 > X.n_rows - m);
    if (bad) m = 0;
  }
};

inline bool spans_meet(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + nb && y < x + na;
}
inline int64_t cache_bytes(const spec_kv_view& kv) {
  return (int64_t)kv.n_pages * kv.n_layers * kv.n_kv_heads * 2 * kv.page_size * kv.head_dim * (kv.dtype == SPEC_F32 ? 4 : 2);
}

// Host checks that these entry points share.
inline int check_chunks(const spec_kv_view* kv, int n_seq, int n_q_heads) {
  const int rc = check_kv_view(kv, true);
  if (rc) return rc;
  if (n_seq < 1 || n_seq > 65535) return set_last_error(SPEC_ERR_ARG, "1 <= n_seq <= 65535 required");
  if (n_q_heads < 1 || n_q_heads % kv->n_kv_heads)
    return set_last_error(SPEC_ERR_ARG, "n_q_heads must be a multiple of n_kv_heads");
  return SPEC_OK;
}
inline int check_layer_rows(const spec_kv_view* kv, int layer, int n_rows, int max_new) {
  if (layer < 0 || layer >= kv->n_layers) return set_last_error(SPEC_ERR_ARG, "layer out of range");
  if (n_rows < 1 || max_new < 1) return set_last_error(SPEC_ERR_ARG, "n_rows >= 1 and max_new >= 1 required");
  return SPEC_OK;
}

// bf16 chunks of few tokens, by the tree attention's kernel (ops_tree.cu): at most
// SPEC_TREE_MAX_NODES tokens of a sequence and 128 (token, head) rows per kv head. The
// arguments are checked already.
size_t chain_ws_bytes(const spec_kv_view& kv, int max_new, int hq);
int launch_chain_attention(const spec_kv_view& kv, int layer, const void* q, int n_rows, int n_seq, int max_new, int hq,
                           const int32_t* row_start, const int32_t* n_new, const int32_t* cache_len, float scale_l2e,
                           void* out, float* lse, void* ws, int32_t* err, int sms, cudaStream_t st);

}  // namespace spec
