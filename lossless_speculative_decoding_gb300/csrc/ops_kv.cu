// Kernel-level entry points on the pages of a cache: the commit of a verified
// tree (walk of the agreeing path, accepted rows moved next to the committed
// ones) and copies of whole pages. Both only move bytes. A commit is bound by the
// latency of its dependent loads (sizes and pages, walk, rows) and by rows of 256
// bytes far apart: 32 sequences, 36 layers of 8 heads, 66 MB: 16.6 us, 0.59 of the
// copy rate (the same with registers for all blocks at once); one sequence in 12
// layers 10 to 11 us, most of it the call. Page copies by HBM: 96 pages of 2.4 MB
// 69.6 us, 6.5 TB/s, 0.96 of the copy rate.
#include <cuda_runtime.h>

#include <algorithm>

#include "kv_view.cuh"

namespace spec {
namespace {

constexpr int COMMIT_THREADS = 256;
// Rows a thread holds in flight. Scattered rows of 256 bytes: 32 sequences with
// up to 14 moves in 36 layers took 16.5 us with 4 rows, 17.6 with 8, 22.6 with 16.
constexpr int COMMIT_ROWS = 4;

struct CommitShared {
  int parent[TREE_N], token[TREE_N], target[TREE_N], path[TREE_N];
  int page[TREE_N];                     // of slots n, n + 1, ..
  long long src[TREE_N], dst[TREE_N];   // row offsets (16-byte pieces) of the moves
  int accepted, moves, ok;
};

// Walk of sequence s by warp 0. Lane l looks at nodes l and l + 32; the lowest
// child that agrees is the lowest set bit of the two ballots. A child's index
// is above its parent's, so the walk ends.
__device__ void walk_tree(const spec_kv_view& kv, int n, int k, CommitShared& sh, int32_t* err, bool report) {
  const int lane = threadIdx.x;
  __syncwarp();
  int cur = 0, a = 0;
  if (lane == 0) sh.path[0] = 0;
  for (;;) {
    const int want = sh.target[cur];
    bool hit[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int c = lane + 32 * u;
      hit[u] = c < k && c > cur && sh.parent[c] == cur && sh.token[c] == want;
    }
    const uint32_t b0 = __ballot_sync(0xffffffffu, hit[0]), b1 = __ballot_sync(0xffffffffu, hit[1]);
    if (!(b0 | b1)) break;
    cur = b0 ? __ffs(b0) - 1 : 31 + __ffs(b1);
    ++a;
    if (lane == 0) sh.path[a] = cur;
  }
  __syncwarp();
  // the moves: rows whose slot changes, in path order; the path's other rows need their pages as well
  const int esz = kv.dtype == SPEC_F32 ? 4 : 2;
  const long long row16 = kv.head_dim * esz / 16, page16 = (long long)kv.n_layers * kv.n_kv_heads * 2 * kv.page_size * row16;
  int moves = 0;
  bool fine = true;
  for (int j0 = 0; j0 <= a; j0 += 32) {
    const int j = j0 + lane;
    const bool on = j <= a, mv = on && sh.path[j] != j;
    const uint32_t who = __ballot_sync(0xffffffffu, mv);
    const int gs = on ? sh.page[sh.path[j]] : 0, gd = on ? sh.page[j] : 0;
    fine = fine && gs >= 0 && gs < kv.n_pages && gd >= 0 && gd < kv.n_pages;
    if (mv) {
      const int ps = n + sh.path[j], pd = n + j;
      const int at = moves + __popc(who & ((1u << lane) - 1));
      sh.src[at] = gs * page16 + (ps % kv.page_size) * row16;
      sh.dst[at] = gd * page16 + (pd % kv.page_size) * row16;
    }
    moves += __popc(who);
  }
  fine = __all_sync(0xffffffffu, fine);
  if (lane == 0) {
    sh.accepted = a;
    sh.moves = fine ? moves : 0;
    sh.ok = fine;
    if (!fine && report) atomicOr(err, DERR_PAGE);
  }
}

// grid (blocks over a row's columns, n_seq). A column is one 16-byte piece of
// one (layer, head, K | V) plane; a thread takes whole columns and moves the
// path's rows of each in order, loading up to COMMIT_ROWS rows before it
// stores any. Row j goes to slot n + j <= n + path_j, and a later row j' > j
// comes from n + path_j' >= n + j' > n + j, so no store lands on a row that is
// still to be read.
__global__ void __launch_bounds__(COMMIT_THREADS) k_tree_commit(spec_kv_view kv, int max_nodes, const int32_t* tokens,
                                                                const int32_t* parents, const int32_t* n_nodes,
                                                                const int32_t* target, const int32_t* cache_len,
                                                                int32_t* out_acc, int32_t* out_tok, int32_t* out_path,
                                                                int32_t* out_len, int32_t* err) {
  __shared__ CommitShared sh;
  const int s = blockIdx.y, t = threadIdx.x;
  if (t < max_nodes) {                           // (on their way beside the sizes)
    const size_t e = (size_t)s * max_nodes + t;
    sh.parent[t] = parents[e];
    sh.token[t] = tokens[e];
    sh.target[t] = target[e];
  }
  const TreeSize z(cache_len, n_nodes, s, max_nodes, kv.max_pages * kv.page_size);
  const bool first = blockIdx.x == 0;
  if (z.k == 0) {
    if (first) {
      for (int j = t; j < max_nodes; j += COMMIT_THREADS) out_path[(size_t)s * max_nodes + j] = -1;
      if (t == 0) {
        out_acc[s] = out_tok[s] = -1;
        out_len[s] = z.n;
        if (z.bad) atomicOr(err, DERR_POS);
      }
    }
    return;
  }
  if (t < z.k && first && (sh.parent[t] < -1 || sh.parent[t] >= t)) atomicOr(err, SPEC_DEV_ERR_TREE);
  if (t >= 64 && t < 64 + z.k) sh.page[t - 64] = kv.block_table_dev[(size_t)s * kv.max_pages + (z.n + t - 64) / kv.page_size];
  __syncthreads();
  if (t < 32) walk_tree(kv, z.n, z.k, sh, err, first);
  __syncthreads();
  const int a = sh.accepted;
  if (first) {
    for (int j = t; j < max_nodes; j += COMMIT_THREADS) out_path[(size_t)s * max_nodes + j] = sh.ok && j <= a ? sh.path[j] : -1;
    if (t == 0) {
      out_acc[s] = sh.ok ? a : -1;
      out_tok[s] = sh.ok ? sh.target[sh.path[a]] : -1;
      out_len[s] = sh.ok ? z.n + a + 1 : z.n;
    }
  }
  const int moves = sh.moves;
  if (moves == 0) return;
  const int row16 = kv.head_dim * (kv.dtype == SPEC_F32 ? 4 : 2) / 16;
  const int cols = kv.n_layers * kv.n_kv_heads * 2 * row16;
  uint4* base = static_cast<uint4*>(kv.kv_dev);
  for (int c = blockIdx.x * COMMIT_THREADS + t; c < cols; c += gridDim.x * COMMIT_THREADS) {
    uint4* col = base + (long long)(c / row16) * kv.page_size * row16 + c % row16;
    for (int j0 = 0; j0 < moves; j0 += COMMIT_ROWS) {
      uint4 v[COMMIT_ROWS];
#pragma unroll
      for (int u = 0; u < COMMIT_ROWS; ++u)
        if (j0 + u < moves) v[u] = col[sh.src[j0 + u]];
#pragma unroll
      for (int u = 0; u < COMMIT_ROWS; ++u)
        if (j0 + u < moves) col[sh.dst[j0 + u]] = v[u];
    }
  }
}

constexpr int COPY_THREADS = 256;
constexpr int COPY_UNROLL = 8;          // 16-byte pieces a thread holds in flight

// grid (blocks over a page, pairs).
__global__ void __launch_bounds__(COPY_THREADS) k_copy_pages(uint4* kv, long long page16, int n_pages, const int32_t* src,
                                                             const int32_t* dst, int n, int32_t* err) {
  for (int i = blockIdx.y; i < n; i += gridDim.y) {
    const int a = src[i], b = dst[i];
    if (a == -1 || b == -1 || (a == b && a >= 0 && a < n_pages)) continue;
    if (a < 0 || a >= n_pages || b < 0 || b >= n_pages) {
      if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(err, DERR_PAGE);
      continue;
    }
    const uint4* from = kv + (long long)a * page16;
    uint4* to = kv + (long long)b * page16;
    const long long step = (long long)gridDim.x * COPY_THREADS * COPY_UNROLL;
    for (long long p = (long long)blockIdx.x * COPY_THREADS * COPY_UNROLL + threadIdx.x; p < page16; p += step) {
      uint4 v[COPY_UNROLL];
#pragma unroll
      for (int u = 0; u < COPY_UNROLL; ++u)
        if (p + u * COPY_THREADS < page16) v[u] = ld_stream(from + p + u * COPY_THREADS);
#pragma unroll
      for (int u = 0; u < COPY_UNROLL; ++u)
        if (p + u * COPY_THREADS < page16) to[p + u * COPY_THREADS] = v[u];
    }
  }
}

}  // namespace
}  // namespace spec

using namespace spec;

extern "C" int spec_tree_commit(const spec_kv_view* kv, int n_seq, int max_nodes, const int32_t* tokens_dev,
                                const int32_t* parents_dev, const int32_t* n_nodes_dev, const int32_t* target_dev,
                                const int32_t* cache_len_dev, int32_t* out_accepted_dev, int32_t* out_token_dev,
                                int32_t* out_path_dev, int32_t* out_len_dev, int32_t* err_dev, uintptr_t cuda_stream) {
  const int rc = check_kv_view(kv, true);
  if (rc) return rc;
  if (!tokens_dev || !parents_dev || !n_nodes_dev || !target_dev || !cache_len_dev || !out_accepted_dev ||
      !out_token_dev || !out_path_dev || !out_len_dev || !err_dev)
    return set_last_error(SPEC_ERR_ARG, "null pointer argument");
  if (n_seq < 1 || n_seq > 65535) return set_last_error(SPEC_ERR_ARG, "1 <= n_seq <= 65535 required");
  if (max_nodes < 1 || max_nodes > TREE_N) return set_last_error(SPEC_ERR_ARG, "1 <= max_nodes <= 64 required");
  // a sequence's blocks read the inputs while one of them writes the outputs
  struct Span { const int32_t* p; int64_t n; };
  const int64_t all = (int64_t)n_seq * max_nodes;
  const Span out[4] = {{out_accepted_dev, n_seq}, {out_token_dev, n_seq}, {out_path_dev, all}, {out_len_dev, n_seq}};
  const Span in[5] = {{tokens_dev, all}, {parents_dev, all}, {target_dev, all}, {n_nodes_dev, n_seq}, {cache_len_dev, n_seq}};
  auto meet = [](const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.n * sizeof(int32_t) && y < x + a.n * sizeof(int32_t);
  };
  for (int i = 0; i < 4; ++i) {
    for (const Span& b : in)
      if (meet(out[i], b)) return set_last_error(SPEC_ERR_ARG, "an output overlaps an input");
    for (int j = 0; j < i; ++j)
      if (meet(out[i], out[j])) return set_last_error(SPEC_ERR_ARG, "two outputs overlap");
  }
  const int64_t cols = (int64_t)kv->n_layers * kv->n_kv_heads * 2 * kv->head_dim * (kv->dtype == SPEC_F32 ? 4 : 2) / 16;
  const int blocks = (int)std::min<int64_t>((cols + COMMIT_THREADS - 1) / COMMIT_THREADS, 4096);
  k_tree_commit<<<dim3(blocks, n_seq), COMMIT_THREADS, 0, reinterpret_cast<cudaStream_t>(cuda_stream)>>>(
      *kv, max_nodes, tokens_dev, parents_dev, n_nodes_dev, target_dev, cache_len_dev, out_accepted_dev, out_token_dev,
      out_path_dev, out_len_dev, err_dev);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SPEC_OK : set_last_error(SPEC_ERR_CUDA, cudaGetErrorString(e));
}

extern "C" int spec_kv_copy_pages(const spec_kv_view* kv, const int32_t* src_dev, const int32_t* dst_dev, int n,
                                  int32_t* err_dev, uintptr_t cuda_stream) {
  const int rc = check_kv_view(kv, false);
  if (rc) return rc;
  if (n < 0) return set_last_error(SPEC_ERR_ARG, "n >= 0 required");
  if (n == 0) return SPEC_OK;
  if (!src_dev || !dst_dev || !err_dev) return set_last_error(SPEC_ERR_ARG, "null pointer argument");
  const long long page16 = (long long)kv->n_layers * kv->n_kv_heads * 2 * kv->page_size * kv->head_dim *
                           (kv->dtype == SPEC_F32 ? 4 : 2) / 16;
  const long long per = COPY_THREADS * COPY_UNROLL;
  const int blocks = (int)std::min<long long>((page16 + per - 1) / per, 65535);
  k_copy_pages<<<dim3(blocks, std::min(n, 65535)), COPY_THREADS, 0, reinterpret_cast<cudaStream_t>(cuda_stream)>>>(
      static_cast<uint4*>(kv->kv_dev), page16, kv->n_pages, src_dev, dst_dev, n, err_dev);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SPEC_OK : set_last_error(SPEC_ERR_CUDA, cudaGetErrorString(e));
}
