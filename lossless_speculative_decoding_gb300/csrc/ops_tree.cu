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
// by row tile, kv head by kv head; block c of B takes units [c U / B, (c + 1)
// U / B) of all U. The blocks stay equally busy whatever the lengths, at most
// two of a block's (sequence, tile, head) segments are shared with other
// blocks, and everything follows from lengths that stay on the device. One
// pass over a segment's keys keeps a running maximum, sum and output (scores
// times log2 e, weights 2^(x - m)). A segment that a block holds alone is
// written as it ends; of a shared one, each block leaves (output, maximum,
// sum) in the workspace and a second launch joins the parts in key order.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

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
  int4* joint;         // [blocks]: (sequence, row tile, kv head, parts and rows) of the shared segment that starts in a block
  int layer, n_seq, max_nodes, hq, G;
  int rows;            // rows of a tile
  int q_box;           // rows of a box of the query's tensor map (tensor-core form)
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

// A block's walk over its units. All threads of the block call init (it has
// block barriers); next() is called by whole warps.
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
    const int a = min(t * per, args.n_seq), a1 = min(a + per, args.n_seq);
    long long sum = 0;
    for (int i = a; i < a1; ++i) sum += units_of(args, i);
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
    // floor(U b / blocks) = (U / blocks) b + floor((U % blocks) b / blocks)
    const long long each = U / blocks;
    const int rest = (int)(U - each * blocks), b = min((int)blockIdx.x, blocks), b1 = min((int)blockIdx.x + 1, blocks);
    u = each * b + rest * b / blocks;
    u1 = each * b1 + rest * b1 / blocks;
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
      in = 0;                                    // the next sequence that is not padded, of 32 at a time
      for (++s;; s += 32) {
        if (s >= A->n_seq) return false;         // (only if the lengths changed meanwhile)
        const int i = s + (threadIdx.x & 31);
        const uint32_t live = __ballot_sync(0xffffffffu, i < A->n_seq && tree_size(*A, i).k > 0);
        if (live) {
          s += __ffs(live) - 1;
          break;
        }
      }
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
// from block `block` on (unit u is in block floor(((u + 1) blocks - 1) / U)).
__device__ __forceinline__ int parts_until(long long U, int block, int blocks, long long end) {
  return (int)((end * blocks - 1) / U) - block + 1;
}

// ---------------------------------------------------------------------------
// FMA form (f32 cache). 128 threads, 32 rows and 64 keys at a time, everything in
// fp32 (the matrix instructions round their operands). Bound: FMA and the shared
// memory that feeds it, 16 bytes read for each 8 FMAs; a few short sequences by
// latency (4 of up to 200 positions, 8 nodes, 4 heads of 64: 11.8 us with the join).
// Thread (ty, tx) = (t / 16, t % 16) has rows 4 ty .. 4 ty + 3, in the score
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
  int parent[TREE_N], page[FM_KEYS];
};

__device__ __forceinline__ void cp_async16(void* smem, const void* gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(gmem) : "memory");
}

template <int D>
__global__ void __launch_bounds__(FM_THREADS) k_tree_fma(const __grid_constant__ TreeArgs A) {
  using L = FmSmem<D>;
  extern __shared__ __align__(16) unsigned char sm_raw[];
  L& sm = *reinterpret_cast<L*>(sm_raw);
  constexpr int NV = D / 64;                     // float4 of dims per thread
  const int t = threadIdx.x, tx = t & 15, ty = t >> 4;
  const int P = A.kv.page_size;
  pdl_wait();
  pdl_trigger();
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
    const float* plane = static_cast<const float*>(A.kv.kv_dev) +
                      (((size_t)A.layer * A.kv.n_kv_heads + g.hk) * 2) * P * D;
    __syncthreads();                             // the last segment's reads of q and mask are done
    if (t < g.k) {
      const int par = A.parents[(size_t)g.s * A.max_nodes + t];
      sm.parent[t] = par;
      if (g.t0 == 0 && (par < -1 || par >= t)) atomicOr(A.err, SPEC_DEV_ERR_TREE);
    }
    for (int i = t; i < FM_ROWS * (D / 4); i += FM_THREADS) {
      const int r = i / (D / 4), c = 4 * (i % (D / 4)), rr = row0 + r;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < nrows) {
        v = *reinterpret_cast<const float4*>(static_cast<const float*>(A.q) +
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
      if (t < FM_KEYS) {
        int page = -1;                           // slots past the last, and bad pages: zeros
        if (t < nk) {
          page = bt[(k0 + t) / P];
          if (page < 0 || page >= A.kv.n_pages) {
            page = -1;
            atomicOr(A.err, DERR_PAGE);
          }
        }
        sm.page[t] = page;
      }
      __syncthreads();
      if (tile == g.t0 && t < g.k) sm.mask[t] = ancestors(sm.parent, t);   // (read after the next barrier)
#pragma unroll 4
      for (int i = t; i < FM_KEYS * (D / 4); i += FM_THREADS) {
        const int key = i / (D / 4), c = 4 * (i % (D / 4)), page = sm.page[key];
        float *kd = &sm.k[key][c], *vd = &sm.v[key][c];
        if (page >= 0) {
          const float* e = plane + page * page_elems + (size_t)((k0 + key) % P) * D + c;
          cp_async16(kd, e);
          cp_async16(vd, e + (size_t)P * D);
        } else {
          *reinterpret_cast<float4*>(kd) = *reinterpret_cast<float4*>(vd) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
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
        float* og = static_cast<float*>(A.out) +
                 (((size_t)g.s * A.max_nodes + rr / A.G) * A.hq + g.hk * A.G + rr % A.G) * D;
        const float inv = 1.f / l[i];
#pragma unroll
        for (int j = 0; j < NV; ++j)
          *reinterpret_cast<float4*>(og + 4 * tx + 64 * j) =
              make_float4(o[i][j].x * inv, o[i][j].y * inv, o[i][j].z * inv, o[i][j].w * inv);
      } else {
        const size_t pr = ((size_t)blockIdx.x * 2 + part) * A.rows + r;
#pragma unroll
        for (int j = 0; j < NV; ++j) *reinterpret_cast<float4*>(A.part_o + pr * D + 4 * tx + 64 * j) = o[i][j];
        if (tx == 0) A.part_ml[pr] = make_float2(m[i], l[i]);
      }
    }
    if (part == 1 && t == 0)
      A.joint[blockIdx.x] = make_int4(g.s, g.rt, g.hk, parts_until(walk.U, blockIdx.x, walk.blocks, walk.u1 + g.nt - g.t1) << 16 | nrows);
  }
}

// ---------------------------------------------------------------------------
// Tensor-core form (bf16 cache). One block per SM, eleven warps: a TMA producer,
// an MMA issuer, a loader (the next segment's sizes, queries and masks) and two
// softmax groups of four warps. Keys come in tiles of 128. S = Q K^T (M = 128
// rows, N = 128 keys) goes to tensor memory; a softmax thread owns one TMEM lane,
// reads its scores 32 at a time, and writes the weights over them as bf16, and
// what that rounding leaves as bf16 too (hi = bf16(p), lo = bf16(p - hi): 16 bits,
// so that the result is as near as the one rounding of the output lets it be);
// O += hi V + lo V takes them from TMEM as the A operand and V as an MN-major B
// operand. Instead of the running maximum, weights 2^(x - m) are taken against a
// whole number m, set 24 above the first scores' maximum and again when a score
// passes m + 8: the weights are floats, whose precision another m leaves as it is,
// so one pass over the scores serves, and the rare step rescales O and the tile's
// earlier weights by an exact power of two. (Weights stay below 2^8, so that large
// values keep their range, and those that float cannot hold are below 2^-100 of the
// largest; a row of values all below 2^-100 would lose bits of its sums. With m
// the maximum itself and moved from 8 above it: 61 us for 57, 170 for 168.)
// Above 2^24 float does not hold every whole number, and a rounded m is soon off by
// more than an exponent's range. A warp that meets such a score takes its chunks
// from there on through a second copy of the loop, out of line, in which such a
// lane subtracts its largest score, s0, from all of them. (The test in the one loop:
// 58 us for 56, 170 for 166; the second copy in line: 57.5.) What lanes, slots and
// blocks are joined by is s0 in units of m, rounded: equal largest scores stay
// equal, others are told apart as far as the rounding of a score of their size.
//
// The two softmax groups have a buffer for S and an accumulator for O ("slot")
// each, take the segment's tiles in turn, so that one's exponentials run beside
// the other's MMAs, and join their results at its end. Up to 64 rows would leave
// half of the lanes idle: the rows are repeated, the upper 64 lanes holding the lo
// parts of the weights where the lower ones hold the hi parts, which saves the
// second MMA; up to 32 rows are repeated once more, and repetition p of two takes
// keys 64 p .. 64 p + 63 of each tile alone, with weights 0 for the others (the
// MMA has M = 128 in any case, and sums each lane apart).
//
// Bound. An MMA of 128 x 128 x 16 takes 64 cycles (measured), so a tile takes the
// tensor cores 1,024 cycles with the hi parts alone and 1,536 with both; its 64 KB
// take 2,800 at an SM's share of the measured copy rate. So HBM, where a tile's
// keys are read for one row tile: 64 sequences of 336 to 5,236 positions and 17 to
// 32 nodes, 10 heads, 0.93 GB: 168 us with the join, 5.5 TB/s, 0.82 of the copy
// rate; two of up to 65,521 positions, 21 nodes, 32 on 8 heads: 74 us, 0.71. With
// two row tiles (8 sequences of 64 nodes, 32 on 8 heads) the chain S, softmax, P V
// of a slot: 2,400 cycles a tile, 57 us with the start (5) and the join (12).
// (Row tiles of 256, each slot with 128 rows of its own, read keys once for all of
// them, but took 59.5 us there, 176 and 79 above: less room for keys, twice the
// bytes of parts to join, more code. Scores 64 at a time: 55.7 and 168. A next
// chunk's scores on their way beside the exponentials: 67 and 178. All 128 in
// registers: 68 and 243. The loops are better short. Weights handed to P V in two
// halves of a tile: 57.5 and 171.)
constexpr int TT_KEYS = 128;
constexpr int TT_THREADS = 352;
constexpr int TT_HALF = 128 * 128;               // bytes of 64 dims of 128 rows of Q
constexpr int TT_OCOL = 256;                     // TMEM columns: S of a slot at 128 slot, its O behind at TT_OCOL + D slot
constexpr float TT_GROW = 8.f, TT_AHEAD = 24.f;  // m moves when a score passes m + 8, to that score + 24
constexpr float TT_FAR = 16777216.f;             // scores up to here go by m alone
constexpr int TT_STAGE = 2 * 128 * 64;           // staged output: two groups x 128 lanes x 16 columns

template <int D>
struct TtCfg {
  static constexpr int BUF = TT_KEYS * D * 2;    // K or V of a tile
  static constexpr int Q = 128 * D * 2;          // 128 rows of Q
  static constexpr int TAIL = 5120;              // alignment slack and the header
  static constexpr int NBUF = (232448 - 512 - TAIL - Q - TT_STAGE) / BUF;
  static constexpr int SMEM = NBUF * BUF + Q + TT_STAGE + TAIL;
};

template <int NBUF>
struct TtHeader {
  uint64_t kv_full[NBUF], kv_empty[NBUF], s_full[2], p_full[2], o_done[2], seg_full[2], seg_free[2], mask_full[2];
  uint64_t q_full, q_free, fin;
  uint32_t tmem;
  int abort;
  TreeSeg seg[2];                                // nt = 0: no more
  int parent[TREE_N];
  unsigned long long mask[2][TREE_N];
  float2 ml[2][128];                             // the lanes' (maximum, sum) in both slots
};

__device__ __forceinline__ uint32_t sm_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 32 (16) columns of this warp's lanes; the values are there when it returns.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_ld16x2(uint32_t a0, uint32_t a1, uint32_t (&r)[16], uint32_t (&q)[16]) {
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7]),
        "=&r"(r[8]), "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]), "=&r"(r[12]), "=&r"(r[13]), "=&r"(r[14]), "=&r"(r[15]),
        "=&r"(q[0]), "=&r"(q[1]), "=&r"(q[2]), "=&r"(q[3]), "=&r"(q[4]), "=&r"(q[5]), "=&r"(q[6]), "=&r"(q[7]),
        "=&r"(q[8]), "=&r"(q[9]), "=&r"(q[10]), "=&r"(q[11]), "=&r"(q[12]), "=&r"(q[13]), "=&r"(q[14]), "=&r"(q[15])
      : "r"(a0), "r"(a1) : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  __syncwarp();
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
}
// (the first 16 values)
template <int N>
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[N]) {
  __syncwarp();
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  __syncwarp();
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// 1 in one lane of the (converged) warp.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r;
}
// Issued by the lanes with one != 0: D (+)= A B with A in shared memory (ss) or
// in tensor memory (ts); the barrier arrival when all MMAs so far are done.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc, uint32_t one) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %5, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc), "r"(one) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc, uint32_t one) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %5, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc), "r"(one) : "memory");
}
__device__ __forceinline__ void tc_commit(uint32_t bar, uint32_t one) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar), "r"(one) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
// A wait that was not over at once, out of line: the waits are many, the code of
// the roles is better short.
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, int* abort, int32_t* err) {
  if (mbar_wait_deadline(bar, parity, abort)) return true;
  *reinterpret_cast<volatile int*>(abort) = DERR_TIMEOUT;
  atomicOr(err, DERR_TIMEOUT);
  return false;
}
__device__ __forceinline__ void mbar_init(const uint64_t* bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(sm_addr(bar)), "r"(count));
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// The same, true when v holds in every thread of it.
__device__ __forceinline__ bool named_sync_and(int id, int threads, bool v) {
  uint32_t r;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}\n"
               : "=r"(r) : "r"((uint32_t)v), "r"(id), "r"(threads) : "memory");
  return r != 0;
}
// Shared-memory matrix descriptor, 128-byte swizzle. sbo: bytes between 8-row
// groups; lbo: bytes between 64-element groups of the leading dimension (an
// MN-major operand; unused for a K-major one).
__device__ __forceinline__ uint64_t tt_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// bf16 pair (a in the low half).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
// Two fp32 values in a register pair, for the packed instructions.
__device__ __forceinline__ unsigned long long pair(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 halves(unsigned long long v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Rows of a segment and how they lie on the 128 lanes of a slot. Queries
// come in boxes of whole nodes, so a few rows behind the segment's may be there
// too; nothing is made of them.
struct TtRows {
  int row0, rows, boxes;       // first row, rows, boxes of queries
  int rpp, kparts;             // lanes of a repetition, parts of a tile's keys
  bool hl;                     // hi parts on the lower lanes, lo parts on the upper ones
  __device__ TtRows(const TreeArgs& A, const TreeSeg& g) {
    row0 = g.rt * A.rows;
    rows = min(A.rows, g.k * A.G - row0);
    boxes = (rows + A.q_box - 1) / A.q_box;
    const int lie = boxes * A.q_box;
    hl = lie <= 64;
    rpp = lie <= 32 ? 32 : lie <= 64 ? 64 : 128;
    kparts = lie <= 32 ? 2 : 1;
  }
};

// A lane's row of a segment so far: weights are 2^(sc (S - s0) - m), l their sum. s0
// is 0, or the largest score (m = TT_AHEAD).
struct TtLane {
  float m, l, s0;
};
// Its scores of a tile.
struct TtTile {
  uint32_t s, o;               // tensor memory of S and O
  unsigned long long mask;     // tree slots it may see
  int slot0, c0;               // tree slot of the tile's first key; the lane's first chunk
  float sc;                    // scale * log2 e
  bool first, live, low, hl;   // no O yet; a row; the lo parts' lane; lo parts on lanes of their own
};

// Chunks c .. c1 - 1 of 32 keys: weights in the place of scores. Without WIDE it
// stops at a chunk with a score beyond TT_FAR, which is as it was; returns the
// chunk it ended before.
template <int D, bool WIDE>
__device__ __forceinline__ int tt_chunks(const TtTile& T, int c, int c1, TtLane& a) {
  const unsigned long long sc2 = pair(T.sc, T.sc);
#pragma unroll 1
  for (; c < c1; ++c) {
    uint32_t v[32];
    tmem_ld32(T.s + 32 * c, v);
    const int sh = T.slot0 + 32 * c;             // tree slot of the chunk's first key
    if (sh > -32) {                              // tree slots, or slots past the last
      uint32_t bits = 0u;
      if (sh < 0) bits = (uint32_t)(T.mask << -sh) | ((1u << -sh) - 1);
      else if (sh < TREE_N) bits = (uint32_t)(T.mask >> sh);
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (!((bits >> i) & 1)) v[i] = 0xff800000u;
    }
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < 32; i += 8)
#pragma unroll
      for (int u = 0; u < 4; ++u) mx[u] = max3(mx[u], __uint_as_float(v[i + 2 * u]), __uint_as_float(v[i + 2 * u + 1]));
    const float mv = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]), mt = (WIDE ? mv - a.s0 : mv) * T.sc;
    const bool grow = T.live && (WIDE && a.s0 != 0.f ? mv > a.s0 : mt > a.m + TT_GROW);
    if (__any_sync(0xffffffffu, grow)) {
      // a larger score: the lane's weights and sums so far are of another m
      const bool away = grow && (WIDE && a.s0 != 0.f || !(fabsf(mt) <= TT_FAR));
      if (!WIDE && __any_sync(0xffffffffu, away)) return c;
      float corr = 1.f;
      if (WIDE && away) {                        // (the score itself, so that equal ones differ by 0)
        corr = ex2(a.m - mt - TT_AHEAD);
        a.m = TT_AHEAD;
        a.s0 = mv;
      } else if (grow) {
        const float to = ceilf(mt) + TT_AHEAD, by = to - a.m;
        corr = by < 127.f ? __uint_as_float((127 - (int)by) << 23) : 0.f;    // 2^-by, exact
        a.m = to;
      }
      a.l *= corr;
      tmem_wait_st();                            // the chunks' weights are read back
      if (!T.first) {                            // (S of this tile came after the slot's last P V)
#pragma unroll 1
        for (int i = 0; i < D; i += 16) {
          uint32_t o[16];
          tmem_ld16(T.o + i, o);
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * corr);
          tmem_st16(T.o + i, o);
        }
      }
#pragma unroll 1
      for (int i = 32 * T.c0; i < 32 * c; i += 16) {
        uint32_t w[16];
        tmem_ld16(T.s + i, w);
#pragma unroll
        for (int j = 0; j < 16; ++j)
          w[j] = pack_bf16(__uint_as_float(w[j] << 16) * corr, __uint_as_float(w[j] & 0xFFFF0000u) * corr);
        tmem_st16(T.s + i, w);
      }
    }
    if constexpr (WIDE) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) - a.s0);
    }
    const float mb = a.m == -INFINITY ? 0.f : a.m;
    const unsigned long long nm2 = pair(-mb, -mb);
    unsigned long long sum[2] = {0, 0};
    uint32_t w[32];
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const float2 y = halves(fma2(pair(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), sc2, nm2));
      const float p0 = ex2(y.x), p1 = ex2(y.y);
      const unsigned long long p2 = pair(p0, p1);
      sum[i / 2 & 1] = add2(sum[i / 2 & 1], p2);
      const uint32_t hi = pack_bf16(p0, p1);
      const float2 e = halves(add2(p2, pair(-__uint_as_float(hi << 16), -__uint_as_float(hi & 0xFFFF0000u))));
      const uint32_t lo = pack_bf16(e.x, e.y);
      w[i / 2] = T.low ? lo : hi;
      w[16 + i / 2] = lo;
    }
    if (T.hl) tmem_st16(T.s + 32 * c, w);
    else tmem_st32(T.s + 32 * c, w);
    const float2 s2 = halves(add2(sum[0], sum[1]));
    a.l += s2.x + s2.y;
  }
  return c;
}
// Out of line: rare, and the loops around it are better without it.
template <int D>
__device__ __noinline__ TtLane tt_chunks_wide(TtTile T, int c, int c1, TtLane a) {
  tt_chunks<D, true>(T, c, c1, a);
  return a;
}

template <int D>
__global__ void __launch_bounds__(TT_THREADS, 1)
    k_tree_tc(const __grid_constant__ CUtensorMap kvmap, const __grid_constant__ CUtensorMap qmap,
              const __grid_constant__ TreeArgs A, int kb) {
  using C = TtCfg<D>;
  constexpr int HALVES = D / 64, NBUF = C::NBUF;
  // a K or V tile lies as [8 keys][64-dim half][key][64 dims], as a box of whole pages brings it
  constexpr int GROUP = 1024 * HALVES;
  extern __shared__ unsigned char tt_raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(tt_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* qsm = base + NBUF * C::BUF;
  unsigned char* stg = qsm + C::Q;
  TtHeader<NBUF>& H = *reinterpret_cast<TtHeader<NBUF>*>(stg + TT_STAGE);
  static_assert(sizeof(TtHeader<NBUF>) + 1024 <= C::TAIL, "header and alignment slack");
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const uint32_t bufs = sm_addr(base), q_addr = sm_addr(qsm);
  if (t == 0) {
    for (int i = 0; i < NBUF; ++i) {
      mbar_init(H.kv_full + i, 1);
      mbar_init(H.kv_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(H.s_full + i, 1);
      mbar_init(H.p_full + i, 4);
      mbar_init(H.o_done + i, 1);
      mbar_init(H.seg_full + i, 1);
      mbar_init(H.mask_full + i, 1);
      mbar_init(H.seg_free + i, 8);              // the softmax warps
    }
    mbar_init(&H.q_full, 1);
    mbar_init(&H.q_free, 1);                     // a segment's last S
    mbar_init(&H.fin, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    H.abort = 0;
  }
  if (t == 32) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kvmap)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&qmap)) : "memory");
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sm_addr(&H.tmem)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_wait();
  pdl_trigger();
  if (t == 0) A.joint[blockIdx.x] = make_int4(0, 0, 0, 0);
  if (blockIdx.x == 0)
    for (int s = t; s < A.n_seq; s += TT_THREADS)
      if (tree_size(A, s).bad) atomicOr(A.err, DERR_POS);
  TreeWalk walk;
  tc_fence_before();
  walk.init<TT_THREADS>(A);                      // two block barriers
  tc_fence_after();
  const uint32_t tmem = H.tmem;
  // A wait that runs out raises the block's abort flag, which ends its other
  // waits at once: the producer and the issuer stop, the softmax groups finish
  // the segment without a result and stop, and so does the loader where a
  // segment's place is not free.
  auto wait = [&](const uint64_t* bar, uint32_t parity) {
    return mbar_try(sm_addr(bar), parity & 1) || wait_long(sm_addr(bar), parity & 1, &H.abort, A.err);
  };
  const int P = A.kv.page_size;

  if (warp == 8) {
    // ---- producer: K and V of every tile, a box for each kb keys of a page ----
    const int nbox = TT_KEYS / kb, j = lane;
    int b = 0;
    uint32_t turn = 0;                           // passes over the ring
    bool ok = true;
    TreeSeg g;
    while (ok && walk.next(g)) {
      const int32_t* bt = A.kv.block_table_dev + (size_t)g.s * A.kv.max_pages;
      const int planes = A.kv.n_layers * A.kv.n_kv_heads * 2, plane = (A.layer * A.kv.n_kv_heads + g.hk) * 2;
      auto page_of = [&](int tile) {             // of this lane's box; -1 reads zeros
        const int key = tile * TT_KEYS + kb * j;
        int page = -1;
        if (lane < nbox && tile < g.t1 && key < g.n + g.k) {
          page = bt[key / P];
          if (page < 0 || page >= A.kv.n_pages) {
            page = -1;
            atomicOr(A.err, DERR_PAGE);
          }
        }
        return page;
      };
      int page = page_of(g.t0), last = -1, next = page_of(g.t0 + 1);   // of the newest tile, the one before, the one after
      for (int i = 0, n = 2 * (g.t1 - g.t0); ok && i < n; ++i) {
        // in the order of their use: K, then K V K V .. V V, a tile's K before the V of the tile ahead of it
        const bool v = i == n - 1 || (i > 0 && i % 2 == 0);
        const int tile = g.t0 + (v ? (i == n - 1 ? n / 2 - 1 : i / 2 - 1) : (i + 1) / 2);
        if (!v && i > 0) {                       // a new tile's K: its pages
          last = page;
          page = next;
          next = page_of(tile + 1);
        }
        const int pg = v && i < n - 1 ? last : page, key = tile * TT_KEYS + kb * j;
        if (turn > 0 && !__all_sync(0xffffffffu, wait(H.kv_empty + b, turn - 1))) { ok = false; break; }
        const uint32_t full = sm_addr(H.kv_full + b);
        if (lane == 0)
          asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full), "r"((uint32_t)C::BUF) : "memory");
        __syncwarp();
        if (lane < nbox)
          asm volatile(
              "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3, %4}], [%5];"
              ::"r"(bufs + b * C::BUF + j * kb * D * 2), "l"(reinterpret_cast<uint64_t>(&kvmap)), "r"(0), "r"(key % P / 8),
                "r"(pg < 0 ? -1 : pg * planes + plane + (v ? 1 : 0)), "r"(full)
              : "memory");
        if (++b == NBUF) { b = 0; ++turn; }
      }
    }
    // shared memory outlives the copies (over, unless the issuer gave up a wait): each buffer's last one
    for (int i = 0; i < NBUF; ++i) mbar_wait_deadline(sm_addr(H.kv_full + i), (i < b ? turn : turn - 1) & 1, nullptr);
  } else if (warp == 9) {
    // ---- MMA issuer: S of a job, then P V of the job before it. The whole
    // warp runs the loop on values that are the same in every lane, so that the
    // descriptors stay in uniform registers; one lane issues (an issue from
    // divergent code takes some 85 cycles, as long as the MMA itself).
    // instruction descriptors: bf16 x bf16 -> f32, M = 128; V is MN-major
    const uint32_t id_s = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(TT_KEYS >> 3) << 17) | (8u << 24);
    const uint32_t id_o = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | (8u << 24);
    const uint32_t one = elect_one(), tm = __shfl_sync(0xffffffffu, tmem, 0);
    auto same = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    auto waitw = [&](const uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
    uint32_t n0 = 0, n1 = 0;                     // jobs of the slots
    int rbuf = 0, rturn = 0;                     // ring position of the next load
    auto step = [&]() {
      if (++rbuf == NBUF) { rbuf = 0; ++rturn; }
    };
    bool ok = true;
    // the tile whose P V is due: slot, tile of the slot, 16-key steps, first of
    // the slot's segment, lo parts apart
    struct Job { int slot; uint32_t k; int steps; bool first, lo; } q{};
    bool due = false;
    auto pv = [&]() {
      due = false;
      const int vbuf = rbuf;
      bool go = waitw(H.kv_full + vbuf, rturn);
      step();
      if (go) go = waitw(H.p_full + q.slot, q.k);
      if (!go) return false;
      tc_fence_after();
      const uint32_t d = tm + TT_OCOL + q.slot * D, a = tm + q.slot * 128;
      const uint64_t bd = tt_desc(bufs + vbuf * C::BUF, 1024, GROUP);
      // 16 keys a step: their hi weights lie in columns 32 (k / 2) + 8 (k % 2) .., the lo ones 16 behind
      auto part = [&](int k, int at, bool acc) { mma_ts(d, a + 32 * (k / 2) + 8 * (k & 1) + at, bd + (uint64_t)(k * 2 * GROUP >> 4), id_o, acc, one); };
      part(0, 0, !q.first);
      if (q.steps == TT_KEYS / 16) {
        if (q.lo) {
          part(0, 16, true);
#pragma unroll
          for (int k = 1; k < TT_KEYS / 16; ++k) {
            part(k, 0, true);
            part(k, 16, true);
          }
        } else {
#pragma unroll
          for (int k = 1; k < TT_KEYS / 16; ++k) part(k, 0, true);
        }
      } else {
        if (q.lo) part(0, 16, true);
#pragma unroll 1
        for (int k = 1; k < q.steps; ++k) {
          part(k, 0, true);
          if (q.lo) part(k, 16, true);
        }
      }
      tc_commit(sm_addr(H.o_done + q.slot), one);
      tc_commit(sm_addr(H.kv_empty + vbuf), one);
      return true;
    };
    for (uint32_t seg = 0; ok; ++seg) {
      const int sb = seg & 1;
      if (!(ok = waitw(H.seg_full + sb, seg >> 1))) break;
      TreeSeg g = H.seg[sb];
      g.nt = same(g.nt); g.t0 = same(g.t0); g.t1 = same(g.t1); g.n = same(g.n); g.k = same(g.k); g.rt = same(g.rt);
      if (g.nt == 0) break;
      const TtRows R(A, g);
      const int nt = g.t1 - g.t0;
      if (!(ok = waitw(&H.q_full, seg))) break;
      for (int ti = 0; ok && ti < nt; ++ti) {
        const int slot = ti & 1, kbuf = rbuf;
        const uint32_t k = slot ? n1++ : n0++;
        // S goes over the slot's last weights: their P V is done
        ok = waitw(H.kv_full + kbuf, rturn);
        step();
        if (ok && k > 0) ok = waitw(H.o_done + slot, k - 1);
        if (!ok) break;
        tc_fence_after();
        const uint64_t ad = tt_desc(q_addr, 16, 1024), bd = tt_desc(bufs + kbuf * C::BUF, 16, GROUP);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          mma_ss(tm + slot * 128, ad + (uint64_t)(((i & 3) * 32 + (i >> 2) * TT_HALF) >> 4),
                 bd + (uint64_t)(((i & 3) * 32 + (i >> 2) * 1024) >> 4), id_s, i > 0, one);
        tc_commit(sm_addr(H.s_full + slot), one);
        tc_commit(sm_addr(H.kv_empty + kbuf), one);
        if (ti == nt - 1) tc_commit(sm_addr(&H.q_free), one);
        if (due) ok = pv();
        q = Job{slot, k, (min(TT_KEYS, g.n + g.k - (g.t0 + ti) * TT_KEYS) + 15) / 16, ti < 2, !R.hl};
        due = true;
      }
      if (ok && due) ok = pv();
    }
    // everything issued is done before TMEM is freed (also after an abort)
    tc_commit(sm_addr(&H.fin), one);
    mbar_wait_deadline(sm_addr(&H.fin), 0, nullptr);
  } else if (warp == 10) {
    // ---- loader: the segments' sizes, queries (repeated down the lanes) and masks ----
    TreeSeg g;
    uint32_t asked = 0;                          // segments whose queries were asked for
    for (uint32_t seg = 0;; ++seg) {
      const int sb = seg & 1;
      const bool have = walk.next(g);
      // (not free: aborted. The softmax warps may still read this place; the others' waits for it end as well)
      if (seg >= 2 && !__all_sync(0xffffffffu, wait(H.seg_free + sb, (seg >> 1) - 1))) break;
      if (!have) g.nt = 0;
      if (lane == 0) {
        H.seg[sb] = g;
        mbar_arrive(sm_addr(H.seg_full + sb));
      }
      if (!have) break;
      const TtRows R(A, g);
      const bool tree = g.t1 * TT_KEYS > g.n;    // the segment reaches the tree's slots
      const int32_t* par = A.parents + (size_t)g.s * A.max_nodes;
      int p[2] = {-1, -1};
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (tree && lane + 32 * u < g.k) p[u] = par[lane + 32 * u];
      if (seg > 0 && !__all_sync(0xffffffffu, wait(&H.q_free, seg - 1))) continue;   // (aborted: no more copies)
      const int nrep = 128 / R.rpp, copies = R.boxes * nrep * HALVES;
      if (lane == 0)
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;"
                     ::"r"(sm_addr(&H.q_full)), "r"((uint32_t)(copies * A.q_box * 128)) : "memory");
      __syncwarp();
      ++asked;
      for (int i = lane; i < copies; i += 32) {
        const int half = i % HALVES, x = i / HALVES % R.boxes, rp = i / HALVES / R.boxes;
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
            ::"r"(q_addr + half * TT_HALF + (x * A.q_box + rp * R.rpp) * 128),
              "l"(reinterpret_cast<uint64_t>(&qmap)), "r"(0), "r"(half), "r"(g.hk * A.G),
              "r"(g.s * A.max_nodes + (R.row0 + x * A.q_box) / A.G), "r"(sm_addr(&H.q_full))
            : "memory");
      }
      if (tree) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int i = lane + 32 * u;
          if (i < g.k) {
            H.parent[i] = p[u];
            if (g.t1 == g.nt && (p[u] < -1 || p[u] >= i)) atomicOr(A.err, SPEC_DEV_ERR_TREE);
          }
        }
        __syncwarp();
#pragma unroll 1
        for (int i = lane; i < g.k; i += 32) H.mask[sb][i] = ancestors(H.parent, i);
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(sm_addr(H.mask_full + sb));
    }
    if (asked > 0) mbar_wait_deadline(sm_addr(&H.q_full), (asked - 1) & 1, nullptr);   // (over, unless aborted)
  } else {
    // ---- softmax groups ----
    const int slot = warp >> 2, r = t & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t oT = tmem + lanes + TT_OCOL + slot * D;
    uint32_t jobs = 0, tiles = 0;                // of this slot; of the block
    for (uint32_t seg = 0;; ++seg) {
      const int sb = seg & 1;
      // all eight warps together: O and the staging bytes of the last segment
      // are free, and either all of them or none go on after an abort
      if (!named_sync_and(1, 256, wait(H.seg_full + sb, seg >> 1))) break;
      const TreeSeg g = H.seg[sb];
      if (g.nt == 0) break;
      const TtRows R(A, g);
      const int nt = g.t1 - g.t0;
      const int rep = r / R.rpp, lr = r % R.rpp;
      const int kpart = R.kparts == 2 ? rep & 1 : 0;
      const bool live = lr < R.rows, low = R.hl && r >= 64;
      const bool any_live = __any_sync(0xffffffffu, live);
      unsigned long long mask = 0;
      if (g.t1 * TT_KEYS > g.n) {
        wait(H.mask_full + sb, seg >> 1);
        if (live) mask = H.mask[sb][(R.row0 + lr) / A.G];
      }
      TtLane st{-INFINITY, 0.f, 0.f};
      bool far = false;                          // a lane of the warp has met a score beyond TT_FAR
      for (int ti = slot; ti < nt; ti += 2) {
        const int k0 = (g.t0 + ti) * TT_KEYS;
        const bool first = ti < 2;
        const uint32_t k = jobs++, sT = tmem + lanes + slot * 128;
        wait(H.s_full + slot, k);
        tc_fence_after();
        if (any_live) {
          // this lane's chunks of 32 keys: all four, or a key part's two
          const int c0 = 2 * kpart, c1 = R.kparts == 2 ? c0 + 2 : 4;
          const TtTile T{sT, oT, mask, k0 - g.n, c0, A.scale_l2e, first, live, low, R.hl};
          const int c = far ? c0 : tt_chunks<D, false>(T, c0, c1, st);
          if (c < c1) {
            far = true;
            st = tt_chunks_wide<D>(T, c, c1, st);
          }
          if (R.kparts == 2) {                   // the other part's keys: weights 0
            uint32_t x[32];
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = 0u;
            tmem_st16(sT + 32 * (2 - c0), x);
            tmem_st16(sT + 32 * (3 - c0), x);
          }
          tmem_wait_st();
        }
        // slots past the last node may hold anything: their V rows become zeros
        const int nk = g.n + g.k - k0;
        if (nk < TT_KEYS) {
          const uint32_t vi = 2 * (tiles + nt) - 1;            // (the segment's last tile: its last load)
          wait(H.kv_full + vi % NBUF, vi / NBUF);
          unsigned char* vb = base + (vi % NBUF) * C::BUF;
          for (int i = r; i < (TT_KEYS - nk) * HALVES * 8; i += 128) {
            const int key = nk + i / (HALVES * 8), hf = i / 8 % HALVES;
            *reinterpret_cast<uint4*>(vb + key / 8 * GROUP + hf * 1024 + key % 8 * 128 + (i % 8) * 16) = make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sm_addr(H.p_full + slot));
      }
      tiles += nt;

      // ---- the segment's end ----
      const int wpart = part_of(g);
      // where row x goes: the result, or this block's part of it
      auto out_row = [&](int x) -> unsigned char* {
        const int rr = R.row0 + x, node = rr / A.G;
        if (wpart < 0)
          return static_cast<unsigned char*>(A.out) +
                 (((size_t)g.s * A.max_nodes + node) * A.hq + g.hk * A.G + rr - node * A.G) * D * 2;
        return reinterpret_cast<unsigned char*>(A.part_o + (((size_t)blockIdx.x * 2 + wpart) * A.rows + x) * D);
      };
      auto emit4 = [&](unsigned char* o, int col, float4 v) {
        if (wpart < 0) *reinterpret_cast<uint2*>(o + col * 2) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
        else *reinterpret_cast<float4*>(o + col * 4) = v;
      };
      // each group waits for its own slot's last P V; the barriers pass that on
      if (slot < nt) wait(H.o_done + slot, jobs - 1);
      const bool both = nt > 1;                  // slot 1 had tiles
      const float ref = fmaf(st.s0, A.scale_l2e, st.m);      // (finite, whatever the scores)
      H.ml[slot][r] = make_float2(live ? fminf(fmaxf(ref, -3e38f), 3e38f) : -INFINITY, live ? st.l : 0.f);
      tc_fence_before();
      named_sync(1, 256);
      tc_fence_after();
      float M = -INFINITY, L = 0.f;
      for (int p = 0; p < R.kparts; ++p) {       // (the upper lanes repeat the lower ones' statistics)
        const float2 a = H.ml[0][p * R.rpp + lr], b = H.ml[1][p * R.rpp + lr];
        const float mn = max3(M, a.x, b.x), mb = mn == -INFINITY ? 0.f : mn;
        L = L * ex2(M - mb) + a.y * ex2(a.x - mb) + b.y * ex2(b.x - mb);
        M = mn;
      }
      // the weight of this lane's O in slot 0, in slot 1
      const float Mb = M == -INFINITY ? 0.f : M, inv = wpart < 0 ? 1.f / L : 1.f;
      const float w0 = ex2(H.ml[0][r].x - Mb) * inv, w1 = ex2(H.ml[1][r].x - Mb) * inv;
      if (wpart >= 0 && slot == 0 && live && rep == 0)
        A.part_ml[((size_t)blockIdx.x * 2 + wpart) * A.rows + lr] = make_float2(M, L);
      // 16 columns at a time through shared memory: a row's repetitions are
      // summed, and four lanes write 64 bytes of a row together. Each group takes
      // half of the columns, of both slots.
      const int nrep = 128 / R.rpp, col0 = slot * (D / 2);
      const uint32_t o0 = tmem + lanes + TT_OCOL + col0, o1 = o0 + D;
      float4* stage = reinterpret_cast<float4*>(stg + slot * (TT_STAGE / 2));   // [128 lanes][16 columns]
      unsigned char* og[4];                      // the rows whose columns 4 (r % 4) .. this thread writes
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int y = r / 4 + 32 * u;
        og[u] = u * nrep < 4 && y < R.rows ? out_row(y) : nullptr;
      }
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[16], x[16];
        if (both) tmem_ld16x2(o0 + 16 * c, o1 + 16 * c, v, x);
        else tmem_ld16(o0 + 16 * c, v);
        float y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = __uint_as_float(v[i]) * w0;
        if (both) {
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i] = fmaf(__uint_as_float(x[i]), w1, y[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          stage[r * 4 + (i ^ ((r >> 1) & 3))] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
        named_sync(2 + slot, 128);
        float4 z[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int ln = r / 4 + 32 * u;
          z[u] = stage[ln * 4 + ((r & 3) ^ ((ln >> 1) & 3))];
        }
        auto add = [](float4& a, const float4& b) { a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w; };
        if (nrep == 4) add(z[0], z[1]);
        if (nrep == 4) add(z[0], z[2]);
        if (nrep == 4) add(z[0], z[3]);
        if (nrep == 2) add(z[0], z[2]);
        if (nrep == 2) add(z[1], z[3]);
        const int col = col0 + 16 * c + 4 * (r & 3);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (og[u]) emit4(og[u], col, z[u]);
        named_sync(2 + slot, 128);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sm_addr(H.seg_free + sb));
      if (wpart == 1 && t == 0)
        A.joint[blockIdx.x] = make_int4(g.s, g.rt, g.hk, parts_until(walk.U, blockIdx.x, walk.blocks, walk.u1 + g.nt - g.t1) << 16 | R.rows);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

// ---------------------------------------------------------------------------
// Joins the parts of the segment that starts in block blockIdx.x and ends in a
// later one: M = max m_c, out = sum_c o_c 2^(m_c - M) / sum_c l_c 2^(m_c - M),
// parts in key order. One warp per row; a row's statistics and its first eight
// parts are on their way together, so that the launch is two round trips to L2
// (the description, the parts) long: under the profiler 7 us behind the 64
// sequences, 12 where parts of 17 MB are joined (8 sequences of 256 rows a head).
// (A last block that joins within the one launch would need counters at zero: this
// entry point takes its workspace as it comes.)
constexpr int JOIN_WARPS = 8;

template <int D, class KT>
__global__ void __launch_bounds__(JOIN_WARPS * 32) k_tree_join(const __grid_constant__ TreeArgs A) {
  pdl_wait();
  pdl_trigger();
  const int4 jt = __ldcg(A.joint + blockIdx.x);
  const int r = blockIdx.y * JOIN_WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int parts = jt.w >> 16, rr = jt.y * A.rows + r;
  if (r >= (jt.w & 0xFFFF)) return;
  // part 0 of the join is this block's part 1, then part 0 of the blocks after it
  auto at = [&](int c) { return ((size_t)(blockIdx.x + c) * 2 + (c == 0 ? 1 : 0)) * A.rows + r; };
  constexpr int NV = D / 32, FLY = 8;            // values a lane; parts in flight at once
  float v[FLY][NV];
  auto fetch = [&](int c0) {
#pragma unroll
    for (int c = 0; c < FLY; ++c) {
      const float* p = A.part_o + at(c0 + c < parts ? c0 + c : c0) * D + NV * lane;
      if constexpr (NV == 4) {
        const float4 f = __ldcg(reinterpret_cast<const float4*>(p));
        v[c][0] = f.x; v[c][1] = f.y; v[c][2] = f.z; v[c][3] = f.w;
      } else {
        const float2 f = __ldcg(reinterpret_cast<const float2*>(p));
        v[c][0] = f.x; v[c][1] = f.y;
      }
    }
  };
  fetch(0);
  float M = -INFINITY, l = 0.f, o[NV];
  for (int c = lane; c < parts; c += 32) M = fmaxf(M, __ldcg(A.part_ml + at(c)).x);
  M = warp_max(M);
#pragma unroll
  for (int i = 0; i < NV; ++i) o[i] = 0.f;
  for (int c0 = 0;;) {
    // lane c has the weight of part c0 + c
    const float2 ml = c0 + (lane & 7) < parts ? __ldcg(A.part_ml + at(c0 + (lane & 7))) : make_float2(-INFINITY, 0.f);
    const float wl = exp2f(ml.x - M);
#pragma unroll
    for (int c = 0; c < FLY; ++c) {
      const float w = __shfl_sync(0xffffffffu, wl, c);
      l = fmaf(__shfl_sync(0xffffffffu, ml.y, c), w, l);
#pragma unroll
      for (int i = 0; i < NV; ++i) o[i] = fmaf(v[c][i], w, o[i]);
    }
    if ((c0 += FLY) >= parts) break;
    fetch(c0);
  }
  KT* og = static_cast<KT*>(A.out) + (((size_t)jt.x * A.max_nodes + rr / A.G) * A.hq + jt.z * A.G + rr % A.G) * D + NV * lane;
  const float inv = 1.f / l;
#pragma unroll
  for (int i = 0; i < NV; ++i) o[i] *= inv;
  if constexpr (sizeof(KT) == 4) {
#pragma unroll
    for (int i = 0; i < NV; ++i) og[i] = o[i];
  } else {
#pragma unroll
    for (int i = 0; i < NV; i += 2) reinterpret_cast<uint32_t*>(og)[i / 2] = pack_bf16(o[i], o[i + 1]);
  }
}

// Shape of a launch, from sizes and types alone.
struct TreePlan {
  bool tc;                  // bf16 cache: the tensor-core form
  int rows, tile_k;
  int q_box;                // rows of a box of queries, whole nodes
  int max_blocks;           // of any grid (the workspace is sized without a device)
  size_t ml, joint, total;  // workspace: outputs at 0, statistics, joints
  TreePlan(const spec_kv_view& kv, int max_nodes, int hq) {
    const int G = hq / kv.n_kv_heads;
    tc = kv.dtype == SPEC_BF16;
    if (tc) {
      // tiles of at most 128 rows, whole nodes, as even as they come
      const int most = std::max(1, 128 / G), nrt = (max_nodes + most - 1) / most;
      int nodes = (max_nodes + nrt - 1) / nrt, box = 8;
      while (box > 1 && box / 2 * G % 8 == 0) box /= 2;
      // boxes start at multiples of 8 rows (the swizzle's period), up to 32 rows
      // each where that many nodes do; one box when the tile has no more nodes,
      // or when whole boxes would go past 128 rows
      box *= std::max(1, 32 / (box * G));
      if (box >= nodes || (nodes + box - 1) / box * box * G > 128) box = nodes;
      q_box = box * G;
      rows = nodes * G;
      tile_k = TT_KEYS;
      max_blocks = 160;     // one block per SM
    } else {
      rows = FM_ROWS;
      q_box = 0;
      tile_k = FM_KEYS;
      max_blocks = 320;     // two blocks per SM
    }
    ml = (size_t)max_blocks * 2 * rows * kv.head_dim * sizeof(float);
    joint = (ml + (size_t)max_blocks * 2 * rows * sizeof(float2) + 15) / 16 * 16;
    total = joint + (size_t)max_blocks * sizeof(int4);
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
  if (((double)kv->max_pages * kv->page_size / FM_KEYS + 1) * ((double)max_nodes * hq / FM_ROWS + kv->n_kv_heads) > 2e9)
    return set_last_error(SPEC_ERR_UNSUPPORTED, "block table too long for this many heads");
  return SPEC_OK;
}

template <int D, class KT>
cudaError_t join(const TreeArgs& A, int blocks, cudaStream_t st) {
  return launch_k(k_tree_join<D, KT>, dim3(blocks, (A.rows + JOIN_WARPS - 1) / JOIN_WARPS), dim3(JOIN_WARPS * 32), 0, st, A);
}

template <int D>
cudaError_t launch_fma(const TreeArgs& A, int blocks, cudaStream_t st) {
  cudaError_t e = allow_dyn_smem_once<k_tree_fma<D>>();
  if (e == cudaSuccess) e = launch_k(k_tree_fma<D>, dim3(blocks), dim3(FM_THREADS), sizeof(FmSmem<D>), st, A);
  return e == cudaSuccess ? join<D, float>(A, blocks, st) : e;
}

template <int D>
cudaError_t launch_tc(const TreeArgs& A, const CUtensorMap& map, const CUtensorMap& qmap, int kb, int blocks, cudaStream_t st) {
  cudaError_t e = allow_dyn_smem_once<k_tree_tc<D>>();
  if (e == cudaSuccess)
    e = launch_k(k_tree_tc<D>, dim3(blocks), dim3(TT_THREADS), TtCfg<D>::SMEM, st, map, qmap, A, kb);
  return e == cudaSuccess ? join<D, bf16_t>(A, blocks, st) : e;
}

}  // namespace
}  // namespace spec

using namespace spec;

extern "C" int64_t spec_tree_attention_ws_bytes(const spec_kv_view* kv, int n_seq, int max_nodes, int n_q_heads) {
  const int rc = check_tree(kv, n_seq, max_nodes, n_q_heads);
  if (rc) return rc;
  return (int64_t)TreePlan(*kv, max_nodes, n_q_heads).total;
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
  if (!(scale > 0.f) || !(scale * LOG2E < INFINITY)) return set_last_error(SPEC_ERR_ARG, "scale must be positive, and finite times log2 e");
  if (!aligned16(q_dev) || !aligned16(out_dev) || !aligned16(ws_dev))
    return set_last_error(SPEC_ERR_ARG, "q, out and the workspace must be 16-byte aligned");
  const int d = kv->head_dim;
  const TreePlan plan(*kv, max_nodes, n_q_heads);
  if (ws_bytes < plan.total) return set_last_error(SPEC_ERR_ARG, "workspace too small");
  const int sms = sm_count_once();
  if (sms < 1) return set_last_error(SPEC_ERR_CUDA, "no device");
  char* w = static_cast<char*>(ws_dev);
  const TreeArgs A{*kv, q_dev, out_dev, cache_len_dev, n_nodes_dev, parents_dev, err_dev, reinterpret_cast<float*>(w),
                   reinterpret_cast<float2*>(w + plan.ml), reinterpret_cast<int4*>(w + plan.joint), layer, n_seq,
                   max_nodes, n_q_heads, n_q_heads / kv->n_kv_heads, plan.rows, plan.q_box, plan.tile_k, scale * LOG2E};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
  const int blocks = std::min((plan.tc ? 1 : 2) * sms, plan.max_blocks);
  cudaError_t e;
  if (plan.tc) {
    // a box never straddles pages: the largest power of two up to a tile that divides a page
    int kb = 16;
    while (kb < TT_KEYS && kv->page_size % (2 * kb) == 0) kb *= 2;
    CUtensorMap map, qmap;
    if (q_make_map(&qmap, q_dev, d, n_q_heads, (uint64_t)n_seq * max_nodes, A.G, plan.q_box / A.G) ||
        kv_make_group_map(&map, kv->kv_dev, d, kv->page_size, (uint64_t)kv->n_pages * kv->n_layers * kv->n_kv_heads * 2, kb))
      return set_last_error(SPEC_ERR_UNSUPPORTED, "tensor map encoding failed");
    e = d == 128 ? launch_tc<128>(A, map, qmap, kb, blocks, st) : launch_tc<64>(A, map, qmap, kb, blocks, st);
  } else {
    e = d == 128 ? launch_fma<128>(A, blocks, st) : launch_fma<64>(A, blocks, st);
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? SPEC_OK : set_last_error(SPEC_ERR_CUDA, cudaGetErrorString(e));
}
