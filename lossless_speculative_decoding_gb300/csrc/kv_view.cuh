// The paged cache of the tree entry points: argument checks, addressing, and
// the ancestors of a drafted tree's nodes.
#pragma once
#include <stdint.h>

#include "common.cuh"
#include "spec.h"

namespace spec {

static_assert(SPEC_DEV_ERR_PAGE == DERR_PAGE && SPEC_DEV_ERR_POS == DERR_POS && SPEC_DEV_ERR_TIMEOUT == DERR_TIMEOUT,
              "device error bits");
constexpr int TREE_N = SPEC_TREE_MAX_NODES;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Host checks shared by the entry points; table: the block table is needed.
inline int check_kv_view(const spec_kv_view* kv, bool table) {
  if (!kv || !kv->kv_dev || (table && !kv->block_table_dev)) return set_last_error(SPEC_ERR_ARG, "null cache view");
  if (kv->dtype != SPEC_F32 && kv->dtype != SPEC_BF16) return set_last_error(SPEC_ERR_UNSUPPORTED, "cache dtype: F32 or BF16");
  if (kv->head_dim != 64 && kv->head_dim != 128) return set_last_error(SPEC_ERR_UNSUPPORTED, "head_dim: 64 or 128");
  if (kv->page_size < 16 || kv->page_size % 16) return set_last_error(SPEC_ERR_ARG, "page_size must be a multiple of 16");
  if (kv->n_pages < 1 || kv->n_layers < 1 || kv->n_kv_heads < 1 || (table && kv->max_pages < 1))
    return set_last_error(SPEC_ERR_ARG, "empty cache view");
  // positions, a page's rows and the cache's (page, layer, head, K | V) planes are counted in 32 bits
  if ((table && (int64_t)kv->max_pages * kv->page_size > (1 << 30)) ||
      (int64_t)kv->n_layers * kv->n_kv_heads * 2 * kv->page_size > (1 << 30) ||
      (int64_t)kv->n_pages * kv->n_layers * kv->n_kv_heads * 2 > (1 << 30))
    return set_last_error(SPEC_ERR_UNSUPPORTED, "cache view too large");
  if (!aligned16(kv->kv_dev)) return set_last_error(SPEC_ERR_ARG, "the cache must be 16-byte aligned");
  return SPEC_OK;
}

// Length and node count of sequence s as the kernels take them: k = 0 for a
// padded sequence and for one whose sizes do not fit (bad).
struct TreeSize {
  int n, k;
  bool bad;
  __device__ TreeSize(const int32_t* cache_len, const int32_t* n_nodes, int s, int max_nodes, int capacity) {
    n = cache_len[s];
    k = n_nodes[s];
    bad = n < 0 || k < 0 || k > max_nodes || n > capacity - max(k, 0);
    if (bad) k = 0;
  }
};

}  // namespace spec
