// Kernel-level entry point: attention of trees of drafted nodes over the paged
// cache.
//
// For node i of a sequence with n committed positions, A(i) the node and those
// above it: out = sum_j w_j V_j over j < n and j in n + A(i), w the softmax of
// scale q.K_j. The node rows of the query heads that share a kv head (row r =
// node r / G, head r % G, G query heads per kv head) meet the same keys, so a
// (sequence, kv head, row tile) reads its keys once for all of its rows.
//
// Work split. Units of tile_k keys are numbered sequence by sequence, row tile
// by row tile, kv head by kv head; block c of G takes units [c U / G, (c + 1)
// U / G) of all U. The blocks stay equally busy whatever the lengths, at most
// two of a block's (sequence, tile, head) segments are shared with other
// blocks, and everything follows from lengths that stay on the device. One
// pass over a segment's keys keeps a running maximum, sum and output (scores
// times log2 e, weights 2^(x - m)). A segment that a block holds alone is
// written as it ends; of a shared one, each block leaves (output, maximum,
// sum) in the workspace and a second launch joins the parts in key order.
#include <cuda_runtime.h>

#include <algorithm>

#include "kv_view.cuh"

namespace spec {
namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr int TREE_MAX_G = 128;                 // query heads per kv head

struct TreeArgs {
  spec_kv_view kv;
  const void* q;
  void* out;
  const int32_t* cache_len;
  const int32_t* n_nodes;
  const int32_t* parents;
  int32_t* err;
  float* part_o;       // [blocks][2][rows][d]: part 0 of a block began in an earlier block, part 1 goes on in the next
  float2* part_ml;     // [blocks][2][rows]: maximum (log2 units), sum
  int4* joint;         // [blocks]: (sequence, row tile, kv head, parts) of the shared segment that starts in a block
  int layer, n_seq, max_nodes, hq, G;
  int rows;            // rows of a tile
  int tile_k;          // keys of a unit
  float scale_l2e;     // scale * log2 e
};

__device__ __forceinline__ TreeSize tree_size(const TreeArgs& A, int s) {
  return TreeSize(A.cache_len, A.n_nodes, s, A.max_nodes, A.kv.max_pages * A.kv.page_size);
}

// Segment: tiles [t0, t1) of nt key tiles of (sequence s, row tile rt, kv head hk).
struct TreeSeg {
  int s, rt, hk, nt, t0, t1;
  int n, k;                                      // committed positions, nodes
};

// A block's walk over its units. All threads of the block call the
// constructor (it has block barriers); next() is free of barriers.
struct TreeWalk {
  long long u, u1, U;                            // units left: [u, u1) of U
  int blocks;                                    // blocks that have units (no more than there are units)
  int s, in;                                     // unit u is number `in` of sequence s
  const TreeArgs* A;

  __device__ static int units_of(const TreeArgs& A, int s) {
    const TreeSize z = tree_size(A, s);
    if (z.k == 0) return 0;
    const int nt = (z.n + z.k + A.tile_k - 1) / A.tile_k, nrt = (z.k * A.G + A.rows - 1) / A.rows;
    return nt * nrt * A.kv.n_kv_heads;           // checked on the host to stay below 2^31
  }
  template <int THREADS>
  __device__ void init(const TreeArgs& args) {
    __shared__ long long w_sum[THREADS / 32];
    __shared__ long long s_start;
    __shared__ int s_seq;
    A = &args;
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    const int per = (args.n_seq + THREADS - 1) / THREADS;
    const int a = min(t * per, args.n_seq), b = min(a + per, args.n_seq);
    long long sum = 0;
    for (int i = a; i < b; ++i) sum += units_of(args, i);
    long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) w_sum[w] = inc;
    __syncthreads();
    long long before = 0, total = 0;
    for (int i = 0; i < THREADS / 32; ++i) {
      if (i < w) before += w_sum[i];
      total += w_sum[i];
    }
    U = total;
    blocks = (int)min((long long)gridDim.x, max(U, 1ll));
    u = U * min((int)blockIdx.x, blocks) / blocks;
    u1 = U * min((int)blockIdx.x + 1, blocks) / blocks;
    long long at = before + inc - sum;
    if (u < u1 && at <= u && u < at + sum) {     // one thread's chunk holds unit u
      int i = a;
      for (int c; at + (c = units_of(args, i)) <= u; ++i) at += c;
      s_seq = i;
      s_start = at;
    }
    __syncthreads();
    if (u < u1) {
      s = s_seq;
      in = (int)(u - s_start);
    }
  }
  __device__ bool next(TreeSeg& g) {
    if (u >= u1) return false;
    TreeSize z = tree_size(*A, s);
    for (;;) {
      if (z.k > 0) {
        g.nt = (z.n + z.k + A->tile_k - 1) / A->tile_k;
        const int nrt = (z.k * A->G + A->rows - 1) / A->rows;
        if (in < g.nt * nrt * A->kv.n_kv_heads) break;
      }
      ++s;
      in = 0;
      z = tree_size(*A, s);
    }
    g.s = s;
    g.n = z.n;
    g.k = z.k;
    const int seg = in / g.nt;
    g.rt = seg / A->kv.n_kv_heads;
    g.hk = seg % A->kv.n_kv_heads;
    g.t0 = in % g.nt;
    g.t1 = (int)min((long long)g.nt, g.t0 + (u1 - u));
    u += g.t1 - g.t0;
    in += g.t1 - g.t0;
    return true;
  }
};

// Bit j of a node's mask: node j is it or above it. A parent outside [-1, i)
// makes a root.
__device__ __forceinline__ unsigned long long ancestors(const int32_t* parents, int i) {
  unsigned long long m = 1ull << i;
  for (;;) {
    const int p = parents[i];
    if (p < 0 || p >= i) return m;
    i = p;
    m |= 1ull << p;
  }
}

// The part of a shared segment that this block leaves: -1 none (the block
// holds the segment alone), 0 or 1.
__device__ __forceinline__ int part_of(const TreeSeg& g) { return g.t0 > 0 ? 0 : (g.t1 < g.nt ? 1 : -1); }

// Number of blocks that hold units of the segment that ends at unit `end`,
// from block `block` on.
__device__ __forceinline__ int parts_until(long long U, int block, int blocks, long long end) {
  int n = 1;
  while (U * (block + n) / blocks < end) ++n;
  return n;
}

// ---------------------------------------------------------------------------
// FMA form. 128 threads, 32 rows and 64 keys at a time, everything in fp32:
// thread (ty, tx) = (t / 16, t % 16) has rows 4 ty .. 4 ty + 3, in the score
// product keys tx + 16 j, in the output product dims 4 tx + 64 j. Rows of K are
// padded by 16 bytes, so eight lanes' reads cover all banks.
constexpr int FM_THREADS = 128;
constexpr int FM_ROWS = 32;
constexpr int FM_KEYS = 64;

template <int D>
struct FmSmem {
  static constexpr int KST = D + 4, PST = FM_KEYS + 4;
  float q[FM_ROWS][D];
  float k[FM_KEYS][KST];
  float v[FM_KEYS][D];
  float p[FM_ROWS][PST];
  unsigned long long mask[TREE_N];
};

template <int D, class KT>
__device__ __forceinline__ float4 load4(const KT* p) {
  if constexpr (sizeof(KT) == 4) {
    return *reinterpret_cast<const float4*>(p);
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xFFFF0000u));
  }
}
template <class KT>
__device__ __forceinline__ void store4(KT* p, float4 v) {
  if constexpr (sizeof(KT) == 4) {
    *reinterpret_cast<float4*>(p) = v;
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(f_to_bf16(v.x) | ((uint32_t)f_to_bf16(v.y) << 16),
                                              f_to_bf16(v.z) | ((uint32_t)f_to_bf16(v.w) << 16));
  }
}

template <int D, class KT>
__global__ void __launch_bounds__(FM_THREADS) k_tree_fma(const __grid_constant__ TreeArgs A) {
  using L = FmSmem<D>;
  extern __shared__ __align__(16) unsigned char sm_raw[];
  L& sm = *reinterpret_cast<L*>(sm_raw);
  constexpr int NV = D / 64;                     // float4 of dims per thread
  const int t = threadIdx.x, tx = t & 15, ty = t >> 4;
  const int P = A.kv.page_size;
  TreeWalk walk;
  walk.init<FM_THREADS>(A);
  if (t == 0) A.joint[blockIdx.x] = make_int4(0, 0, 0, 0);
  if (blockIdx.x == 0)
    for (int s = t; s < A.n_seq; s += FM_THREADS)
      if (tree_size(A, s).bad) atomicOr(A.err, DERR_POS);
  const size_t page_elems = (size_t)A.kv.n_layers * A.kv.n_kv_heads * 2 * P * D;
  TreeSeg g;
  while (walk.next(g)) {
    const int row0 = g.rt * FM_ROWS, nrows = min(FM_ROWS, g.k * A.G - row0);
    const int32_t* bt = A.kv.block_table_dev + (size_t)g.s * A.kv.max_pages;
    const KT* plane = static_cast<const KT*>(A.kv.kv_dev) +
                      (((size_t)A.layer * A.kv.n_kv_heads + g.hk) * 2) * P * D;
    __syncthreads();                             // the last segment's reads of q and mask are done
    if (t < g.k) {
      const int32_t* par = A.parents + (size_t)g.s * A.max_nodes;
      sm.mask[t] = ancestors(par, t);
      if (g.t0 == 0 && (par[t] < -1 || par[t] >= t)) atomicOr(A.err, SPEC_DEV_ERR_TREE);
    }
    for (int i = t; i < FM_ROWS * (D / 4); i += FM_THREADS) {
      const int r = i / (D / 4), c = 4 * (i % (D / 4)), rr = row0 + r;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < nrows) {
        v = load4<D>(static_cast<const KT*>(A.q) +
                     (((size_t)g.s * A.max_nodes + rr / A.G) * A.hq + g.hk * A.G + rr % A.G) * D + c);
        v = make_float4(v.x * A.scale_l2e, v.y * A.scale_l2e, v.z * A.scale_l2e, v.w * A.scale_l2e);
      }
      *reinterpret_cast<float4*>(&sm.q[r][c]) = v;
    }
    float m[4], l[4];
    float4 o[4][NV];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) o[i][j] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int tile = g.t0; tile < g.t1; ++tile) {
      const int k0 = tile * FM_KEYS, nk = min(FM_KEYS, g.n + g.k - k0);
      __syncthreads();                           // the last tile's reads of k, v and p are done
      for (int i = t; i < FM_KEYS * (D / 4); i += FM_THREADS) {
        const int key = i / (D / 4), c = 4 * (i % (D / 4));
        float4 kv4 = make_float4(0.f, 0.f, 0.f, 0.f), vv4 = kv4;     // slots past the last: zeros
        if (key < nk) {
          const int page = bt[(k0 + key) / P];
          if (page < 0 || page >= A.kv.n_pages) {
            atomicOr(A.err, DERR_PAGE);
          } else {
            const KT* e = plane + page * page_elems + (size_t)((k0 + key) % P) * D + c;
            kv4 = load4<D>(e);
            vv4 = load4<D>(e + (size_t)P * D);
          }
        }
        *reinterpret_cast<float4*>(&sm.k[key][c]) = kv4;
        *reinterpret_cast<float4*>(&sm.v[key][c]) = vv4;
      }
      __syncthreads();
      float x[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = 0.f;
#pragma unroll 4
      for (int c = 0; c < D; c += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(&sm.q[4 * ty + i][c]);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(&sm.k[tx + 16 * j][c]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[i][j] = fmaf(a[i].x, b[j].x, x[i][j]);
            x[i][j] = fmaf(a[i].y, b[j].y, x[i][j]);
            x[i][j] = fmaf(a[i].z, b[j].z, x[i][j]);
            x[i][j] = fmaf(a[i].w, b[j].w, x[i][j]);
          }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int node = min(row0 + 4 * ty + i, g.k * A.G - 1) / A.G;
        const unsigned long long mask = sm.mask[node];
        float mt = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = tx + 16 * j, slot = k0 + key - g.n;        // >= 0: a tree slot
          if (key >= nk || (slot >= 0 && !((mask >> slot) & 1))) x[i][j] = -INFINITY;
          mt = fmaxf(mt, x[i][j]);
        }
#pragma unroll
        for (int w = 1; w < 16; w <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, w));
        const float mn = fmaxf(m[i], mt), base = mn == -INFINITY ? 0.f : mn;   // nothing seen yet: weights 0
        const float corr = exp2f(m[i] - base);
        float lt = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = exp2f(x[i][j] - base);
          lt += e;
          sm.p[4 * ty + i][tx + 16 * j] = e;
        }
#pragma unroll
        for (int w = 1; w < 16; w <<= 1) lt += __shfl_xor_sync(0xffffffffu, lt, w);
        l[i] = fmaf(l[i], corr, lt);
        m[i] = mn;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          o[i][j].x *= corr; o[i][j].y *= corr; o[i][j].z *= corr; o[i][j].w *= corr;
        }
      }
      __syncwarp();                              // a row's p is written and read by the same half warp
#pragma unroll 2
      for (int key = 0; key < FM_KEYS; key += 4) {
        float4 pr[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) pr[i] = *reinterpret_cast<const float4*>(&sm.p[4 * ty + i][key]);
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            const float4 vv = *reinterpret_cast<const float4*>(&sm.v[key + u][4 * tx + 64 * j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float w = u == 0 ? pr[i].x : u == 1 ? pr[i].y : u == 2 ? pr[i].z : pr[i].w;
              o[i][j].x = fmaf(w, vv.x, o[i][j].x);
              o[i][j].y = fmaf(w, vv.y, o[i][j].y);
              o[i][j].z = fmaf(w, vv.z, o[i][j].z);
              o[i][j].w = fmaf(w, vv.w, o[i][j].w);
            }
          }
      }
    }
    const int part = part_of(g);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * ty + i, rr = row0 + r;
      if (r >= nrows) continue;
      if (part < 0) {
        KT* og = static_cast<KT*>(A.out) +
                 (((size_t)g.s * A.max_nodes + rr / A.G) * A.hq + g.hk * A.G + rr % A.G) * D;
        const float inv = 1.f / l[i];
#pragma unroll
        for (int j = 0; j < NV; ++j)
          store4<KT>(og + 4 * tx + 64 * j, make_float4(o[i][j].x * inv, o[i][j].y * inv, o[i][j].z * inv, o[i][j].w * inv));
      } else {
        const size_t pr = ((size_t)blockIdx.x * 2 + part) * A.rows + r;
#pragma unroll
        for (int j = 0; j < NV; ++j) *reinterpret_cast<float4*>(A.part_o + pr * D + 4 * tx + 64 * j) = o[i][j];
        if (tx == 0) A.part_ml[pr] = make_float2(m[i], l[i]);
      }
    }
    if (part == 1 && t == 0)
      A.joint[blockIdx.x] = make_int4(g.s, g.rt, g.hk, parts_until(walk.U, blockIdx.x, walk.blocks, walk.u1 + g.nt - g.t1));
  }
}

// Joins the parts of the segment that starts in block blockIdx.x and ends in a
// later one: M = max m_c, out = sum_c o_c 2^(m_c - M) / sum_c l_c 2^(m_c - M),
// parts in key order. One warp per row.
constexpr int JOIN_WARPS = 8;

template <int D, class KT>
__global__ void __launch_bounds__(JOIN_WARPS * 32) k_tree_join(const __grid_constant__ TreeArgs A) {
  const int4 jt = A.joint[blockIdx.x];
  const int r = blockIdx.y * JOIN_WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int parts = jt.w;
  if (parts == 0) return;
  const int s = jt.x, rr = jt.y * A.rows + r;
  if (r >= A.rows || rr >= tree_size(A, s).k * A.G) return;
  // part 0 of the join is this block's part 1, then part 0 of the blocks after it
  auto at = [&](int c) { return ((size_t)(blockIdx.x + c) * 2 + (c == 0 ? 1 : 0)) * A.rows + r; };
  float M = -INFINITY;
  for (int c = lane; c < parts; c += 32) M = fmaxf(M, A.part_ml[at(c)].x);
  M = warp_max(M);
  constexpr int NV = D / 32;
  float o[NV], l = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) o[i] = 0.f;
  for (int c = 0; c < parts; ++c) {
    const float2 ml = A.part_ml[at(c)];
    const float w = exp2f(ml.x - M);
    l = fmaf(ml.y, w, l);
    const float* v = A.part_o + at(c) * D + NV * lane;
#pragma unroll
    for (int i = 0; i < NV; ++i) o[i] = fmaf(v[i], w, o[i]);
  }
  KT* og = static_cast<KT*>(A.out) + (((size_t)s * A.max_nodes + rr / A.G) * A.hq + jt.z * A.G + rr % A.G) * D + NV * lane;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if constexpr (sizeof(KT) == 4) og[i] = o[i] / l;
    else reinterpret_cast<uint16_t*>(og)[i] = f_to_bf16(o[i] / l);
  }
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n;
}

constexpr int FM_PER_SM = 2;
// blocks of the largest grid any device of this kind gives
constexpr int TREE_MAX_BLOCKS = 512;

struct TreeWs {
  size_t o, ml, joint, total;
  TreeWs(int rows, int d) {
    o = 0;
    ml = o + (size_t)TREE_MAX_BLOCKS * 2 * rows * d * sizeof(float);
    joint = ml + (size_t)TREE_MAX_BLOCKS * 2 * rows * sizeof(float2);
    total = joint + (size_t)TREE_MAX_BLOCKS * sizeof(int4);
  }
};

int check_tree(const spec_kv_view* kv, int n_seq, int max_nodes, int hq) {
  const int rc = check_kv_view(kv, true);
  if (rc) return rc;
  if (n_seq < 1 || n_seq > 65535) return set_last_error(SPEC_ERR_ARG, "1 <= n_seq <= 65535 required");
  if (max_nodes < 1 || max_nodes > TREE_N) return set_last_error(SPEC_ERR_ARG, "1 <= max_nodes <= 64 required");
  if (hq < 1 || hq % kv->n_kv_heads) return set_last_error(SPEC_ERR_ARG, "n_q_heads must be a multiple of n_kv_heads");
  if (hq / kv->n_kv_heads > TREE_MAX_G) return set_last_error(SPEC_ERR_UNSUPPORTED, "more than 128 query heads per kv head");
  // a sequence's units are counted in 32 bits
  if ((double)kv->max_pages * kv->page_size / FM_KEYS * ((double)max_nodes * hq / FM_ROWS + kv->n_kv_heads) > 2e9)
    return set_last_error(SPEC_ERR_UNSUPPORTED, "block table too long for this many heads");
  return SPEC_OK;
}

}  // namespace
}  // namespace spec

using namespace spec;

extern "C" int64_t spec_tree_attention_ws_bytes(const spec_kv_view* kv, int n_seq, int max_nodes, int n_q_heads) {
  const int rc = check_tree(kv, n_seq, max_nodes, n_q_heads);
  if (rc) return rc;
  return (int64_t)TreeWs(FM_ROWS, kv->head_dim).total;
}

extern "C" int spec_tree_attention(const spec_kv_view* kv, int layer, const void* q_dev, int n_seq, int max_nodes,
                                   int n_q_heads, const int32_t* cache_len_dev, const int32_t* n_nodes_dev,
                                   const int32_t* parents_dev, float scale, void* out_dev, void* ws_dev,
                                   size_t ws_bytes, int32_t* err_dev, uintptr_t cuda_stream) {
  const int rc = check_tree(kv, n_seq, max_nodes, n_q_heads);
  if (rc) return rc;
  if (!q_dev || !out_dev || !cache_len_dev || !n_nodes_dev || !parents_dev || !ws_dev || !err_dev)
    return set_last_error(SPEC_ERR_ARG, "null pointer argument");
  if (layer < 0 || layer >= kv->n_layers) return set_last_error(SPEC_ERR_ARG, "layer out of range");
  if (!(scale > 0.f) || !(scale < INFINITY)) return set_last_error(SPEC_ERR_ARG, "scale must be positive");
  if (!aligned16(q_dev) || !aligned16(out_dev) || !aligned16(ws_dev))
    return set_last_error(SPEC_ERR_ARG, "q, out and the workspace must be 16-byte aligned");
  const int d = kv->head_dim;
  const TreeWs ws(FM_ROWS, d);
  if (ws_bytes < ws.total) return set_last_error(SPEC_ERR_ARG, "workspace too small");
  const int sms = sm_count();
  if (sms < 1) return set_last_error(SPEC_ERR_CUDA, "no device");
  char* w = static_cast<char*>(ws_dev);
  TreeArgs A{*kv, q_dev, out_dev, cache_len_dev, n_nodes_dev, parents_dev, err_dev,
             reinterpret_cast<float*>(w + ws.o), reinterpret_cast<float2*>(w + ws.ml),
             reinterpret_cast<int4*>(w + ws.joint), layer, n_seq, max_nodes, n_q_heads, n_q_heads / kv->n_kv_heads,
             FM_ROWS, FM_KEYS, scale * LOG2E};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
  const int blocks = std::min(FM_PER_SM * sms, TREE_MAX_BLOCKS);
  const dim3 jgrid(blocks, (FM_ROWS + JOIN_WARPS - 1) / JOIN_WARPS);
  cudaError_t e = cudaSuccess;
#define TREE_FMA(D, KT)                                                                   \
  if ((e = allow_dyn_smem(k_tree_fma<D, KT>)) == cudaSuccess) {                           \
    k_tree_fma<D, KT><<<blocks, FM_THREADS, sizeof(FmSmem<D>), st>>>(A);                  \
    k_tree_join<D, KT><<<jgrid, JOIN_WARPS * 32, 0, st>>>(A);                             \
  }
  if (kv->dtype == SPEC_F32) {
    if (d == 128) { TREE_FMA(128, float) } else { TREE_FMA(64, float) }
  } else {
    if (d == 128) { TREE_FMA(128, bf16_t) } else { TREE_FMA(64, bf16_t) }
  }
#undef TREE_FMA
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? SPEC_OK : set_last_error(SPEC_ERR_CUDA, cudaGetErrorString(e));
}
