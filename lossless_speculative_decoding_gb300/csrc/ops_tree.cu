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
// FMA form (f32 cache). 128 threads, 32 rows and 64 keys at a time, everything in fp32:
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
      const int32_t* par = A.parents + (size_t)g.s * A.max_nodes;
      sm.mask[t] = ancestors(par, t);
      if (g.t0 == 0 && (par[t] < -1 || par[t] >= t)) atomicOr(A.err, SPEC_DEV_ERR_TREE);
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
      for (int i = t; i < FM_KEYS * (D / 4); i += FM_THREADS) {
        const int key = i / (D / 4), c = 4 * (i % (D / 4));
        float4 kv4 = make_float4(0.f, 0.f, 0.f, 0.f), vv4 = kv4;     // slots past the last: zeros
        if (key < nk) {
          const int page = bt[(k0 + key) / P];
          if (page < 0 || page >= A.kv.n_pages) {
            atomicOr(A.err, DERR_PAGE);
          } else {
            const float* e = plane + page * page_elems + (size_t)((k0 + key) % P) * D + c;
            kv4 = *reinterpret_cast<const float4*>(e);
            vv4 = *reinterpret_cast<const float4*>(e + (size_t)P * D);
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
      A.joint[blockIdx.x] = make_int4(g.s, g.rt, g.hk, parts_until(walk.U, blockIdx.x, walk.blocks, walk.u1 + g.nt - g.t1));
  }
}

// ---------------------------------------------------------------------------
// Tensor-core form (bf16 cache). One block per SM, ten warps: a TMA producer,
// an MMA issuer and two softmax groups of four warps. Keys come in tiles of
// 128. S = Q K^T (M = 128 rows, N = 128 keys) goes to tensor memory; a softmax
// thread owns one TMEM lane, reads its scores, and writes the weights over
// them as two bf16 parts (hi = bf16(p), lo = bf16(p - hi): 16 bits, so that the
// result is as near as the one rounding of the output lets it be); O += hi V +
// lo V takes them from TMEM as the A operand and V as an MN-major B operand.
// The running maximum moves, and O is rescaled, only when a tile's maximum is
// more than 8 (a factor of 256) above it.
//
// The two softmax groups work on two (S, O) slots in turn, so one group's
// exponentials overlap the other slot's MMAs. More than 128 rows: slot i has
// rows 128 i .. 128 i + 127 and both use every key tile. Up to 128 rows: the
// slots take the segment's tiles alternately and their results are joined at
// its end. Up to 64 (32) rows would leave most lanes idle, so the rows are
// repeated 2 (4) times down the 128 lanes and repetition p takes the keys 128 /
// nq p .. of each tile alone, with weights 0 for the others: the MMA, which has
// M = 128 in any case, sums each repetition apart.
//
// Bound: HBM for up to some 128 rows (two MMAs of 128 x 128 x 128 and one more
// for the low part take about 1,540 cycles a tile, the tile's 64 KB some 2,800
// at an SM's share of the measured copy rate), the tensor cores above that.
constexpr int TT_KEYS = 128;
constexpr int TT_THREADS = 320;
constexpr int TT_HALF = TT_KEYS * 128;           // bytes of 64 dims of a tile
constexpr int TT_MAXBUF = 12;

template <int D>
struct TtCfg {
  static constexpr int BUF = TT_KEYS * D * 2;    // K or V of a tile, and Q of a slot
  // Q (one slot, or two for more than 128 rows); at a segment's end the same
  // bytes hold the statistics and the staged output (32 KB)
  static constexpr int q_bytes(bool two) { return (two ? 2 : 1) * BUF < 32768 ? 32768 : (two ? 2 : 1) * BUF; }
  static constexpr int TAIL = 2048;              // alignment slack and the header
  static constexpr int nbuf(bool two) {
    return (232448 - 512 - TAIL - q_bytes(two)) / BUF < TT_MAXBUF ? (232448 - 512 - TAIL - q_bytes(two)) / BUF : TT_MAXBUF;
  }
  static constexpr int smem(bool two) { return nbuf(two) * BUF + q_bytes(two) + TAIL; }
};

struct TtHeader {
  uint64_t kv_full[TT_MAXBUF], kv_empty[TT_MAXBUF], s_full[2], p_full[2], o_done[2], q_full, fin;
  uint32_t tmem;
  int abort;
  int parent[TREE_N];
};
static_assert(sizeof(TtHeader) <= 1024, "header and alignment slack share 2 KB");

__device__ __forceinline__ uint32_t sm_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 32 columns of this warp's lanes; the values are there when it returns.
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
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_init(const uint64_t* bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(sm_addr(bar)), "r"(count));
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Shared-memory matrix descriptor, 128-byte swizzle, 8-row groups 1024 bytes
// apart. lbo: bytes between 64-element groups of the leading dimension (an
// MN-major operand; unused for a K-major one).
__device__ __forceinline__ uint64_t tt_desc(uint32_t saddr, uint32_t lbo) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
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

// Rows of a segment and how they lie on the 128 lanes of the two slots.
struct TtRows {
  int row0, rows, nq, rpp;     // first row, rows, repetitions, lanes of one
  bool two;                    // slots split the rows, not the key tiles
  __device__ TtRows(const TreeArgs& A, const TreeSeg& g) {
    row0 = g.rt * A.rows;
    rows = min(A.rows, g.k * A.G - row0);
    two = rows > 128;
    nq = rows <= 32 ? 4 : rows <= 64 ? 2 : 1;
    rpp = 128 / nq;
  }
};

template <int D>
__global__ void __launch_bounds__(TT_THREADS, 1)
    k_tree_tc(const __grid_constant__ CUtensorMap kvmap, const __grid_constant__ TreeArgs A, int nbuf, int q_bytes, int kb) {
  using C = TtCfg<D>;
  constexpr int HALVES = D / 64, OCOL = 256;
  extern __shared__ unsigned char tt_raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(tt_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* qsm = base + nbuf * C::BUF;
  TtHeader& H = *reinterpret_cast<TtHeader*>(qsm + q_bytes);
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const uint32_t bufs = sm_addr(base), q_addr = sm_addr(qsm);
  if (t == 0) {
    for (int i = 0; i < nbuf; ++i) {
      mbar_init(H.kv_full + i, 1);
      mbar_init(H.kv_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(H.s_full + i, 1);
      mbar_init(H.p_full + i, 4);
      mbar_init(H.o_done + i, 1);
    }
    mbar_init(&H.q_full, 8);
    mbar_init(&H.fin, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    H.abort = 0;
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
  // waits at once: the producer and the issuer stop, the softmax groups go on
  // through their barriers without results.
  auto wait = [&](const uint64_t* bar, uint32_t parity) {
    if (mbar_wait_deadline(sm_addr(bar), parity & 1, &H.abort)) return true;
    *reinterpret_cast<volatile int*>(&H.abort) = DERR_TIMEOUT;
    atomicOr(A.err, DERR_TIMEOUT);
    return false;
  };
  TreeSeg g;
  const int P = A.kv.page_size;

  if (warp == 8) {
    // ---- producer: K and V of every tile, boxes of kb keys x 64 dims ----
    const int nbox = TT_KEYS / kb, j = lane % nbox, half = lane / nbox;
    int b = 0;
    uint32_t turn = 0;                           // passes over the ring
    bool ok = true;
    while (ok && walk.next(g)) {
      const int32_t* bt = A.kv.block_table_dev + (size_t)g.s * A.kv.max_pages;
      const int plane = (A.layer * A.kv.n_kv_heads + g.hk) * 2;
      for (int tile = g.t0; ok && tile < g.t1; ++tile) {
        const int key = tile * TT_KEYS + kb * j;
        int page = -1;                           // reads zeros
        if (lane < nbox * HALVES && key < g.n + g.k) {
          page = bt[key / P];
          if (page < 0 || page >= A.kv.n_pages) {
            page = -1;
            atomicOr(A.err, DERR_PAGE);
          }
        }
        for (int kv = 0; kv < 2; ++kv) {
          if (turn > 0 && !wait(H.kv_empty + b, turn - 1)) { ok = false; break; }
          const uint32_t full = sm_addr(H.kv_full + b);
          if (lane == 0)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full), "r"((uint32_t)C::BUF) : "memory");
          __syncwarp();
          if (lane < nbox * HALVES)
            asm volatile(
                "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
                ::"r"(bufs + b * C::BUF + half * TT_HALF + j * kb * 128), "l"(reinterpret_cast<uint64_t>(&kvmap)), "r"(0),
                  "r"(key % P), "r"(half), "r"(plane + kv), "r"(page), "r"(full)
                : "memory");
          if (++b == nbuf) { b = 0; ++turn; }
        }
      }
    }
    if (!ok)                                     // shared memory outlives the copies in flight
      for (int i = 0; i < nbuf; ++i) mbar_wait_deadline(sm_addr(H.kv_full + i), (i < b ? turn : turn - 1) & 1, nullptr);
  } else if (warp == 9) {
    if (lane == 0) {
      // ---- MMA issuer: S of a job, then P V of the job before it ----
      // instruction descriptors: bf16 x bf16 -> f32, M = 128; V is MN-major
      const uint32_t id_s = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(TT_KEYS >> 3) << 17) | (8u << 24);
      const uint32_t id_o = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | (8u << 24);
      uint32_t jobs[2] = {0, 0}, tiles = 0, segs = 0;
      bool ok = true;
      struct { int slot, steps; bool first, last; uint32_t v; } pend = {0, 0, false, false, 0};   // v: index of the V load
      bool have = false;
      auto buf_of = [&](uint32_t idx) { return bufs + (idx % nbuf) * C::BUF; };
      auto pv = [&]() {
        have = false;
        if (!wait(H.p_full + pend.slot, jobs[pend.slot] - 1) || !wait(H.kv_full + pend.v % nbuf, pend.v / nbuf)) return false;
        tc_fence_after();
        const uint32_t d = tmem + OCOL + pend.slot * D, a = tmem + pend.slot * TT_KEYS;
        const uint64_t bd = tt_desc(buf_of(pend.v), TT_HALF);
        uint32_t acc = pend.first ? 0u : 1u;
        for (int k = 0; k < pend.steps; ++k) {
#pragma unroll
          for (int part = 0; part < 2; ++part) {   // the hi, then the lo weights of 16 keys
            asm volatile(
                "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
                ::"r"(d), "r"(a + 32 * (k / 2) + 8 * (k & 1) + 16 * part), "l"(bd + (uint64_t)(k * (2048 >> 4))), "r"(id_o), "r"(acc));
            acc = 1u;
          }
        }
        tc_commit(sm_addr(H.o_done + pend.slot));
        if (pend.last) tc_commit(sm_addr(H.kv_empty + pend.v % nbuf));
        return true;
      };
      while (ok && walk.next(g)) {
        const TtRows R(A, g);
        const int nt = g.t1 - g.t0, nj = R.two ? 2 * nt : nt;
        ok = wait(&H.q_full, segs++);
        for (int jb = 0; ok && jb < nj; ++jb) {
          const int slot = jb & 1, ti = R.two ? jb >> 1 : jb;
          const uint32_t kidx = 2 * (tiles + ti);
          // the slot's weights are read: the P V of its last job is done
          ok = wait(H.kv_full + kidx % nbuf, kidx / nbuf) && (jobs[slot] == 0 || wait(H.o_done + slot, jobs[slot] - 1));
          if (!ok) break;
          tc_fence_after();
          const uint64_t ad = tt_desc(q_addr + (R.two ? slot * C::BUF : 0), 16), bd = tt_desc(buf_of(kidx), 16);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint64_t off = (uint64_t)(((k >> 2) * TT_HALF + (k & 3) * 32) >> 4);
            asm volatile(
                "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n"
                ::"r"(tmem + slot * TT_KEYS), "l"(ad + off), "l"(bd + off), "r"(id_s), "r"(k ? 1u : 0u));
          }
          const bool last = !R.two || slot == 1;
          tc_commit(sm_addr(H.s_full + slot));
          if (last) tc_commit(sm_addr(H.kv_empty + kidx % nbuf));
          if (have) ok = pv();
          ++jobs[slot];
          pend = {slot, (min(TT_KEYS, g.n + g.k - (g.t0 + ti) * TT_KEYS) + 15) / 16, ti == (R.two ? 0 : slot), last, kidx + 1};
          have = true;
        }
        if (ok && have) ok = pv();
        tiles += nt;
      }
      // everything issued is done before TMEM is freed (also after an abort)
      tc_commit(sm_addr(&H.fin));
      mbar_wait_deadline(sm_addr(&H.fin), 0, nullptr);
    }
  } else {
    // ---- softmax groups ----
    const int slot = warp >> 2, r = t & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t sT = tmem + lanes + slot * TT_KEYS, oT = tmem + lanes + OCOL + slot * D;
    uint32_t jobs = 0, tiles = 0;                // of this slot; of the block
    while (walk.next(g)) {
      const TtRows R(A, g);
      const int nt = g.t1 - g.t0;
      const int part = R.two ? 0 : r / R.rpp, lr = R.two ? slot * 128 + r : r % R.rpp;
      const bool live = lr < R.rows;
      // Q rows, repeated nq times down the lanes, and the nodes' masks
      for (int i = t; i < R.rows * (D / 8); i += 256) {
        const int x = i / (D / 8), c = i % (D / 8), rr = R.row0 + x;
        const uint4 v = *reinterpret_cast<const uint4*>(
            static_cast<const bf16_t*>(A.q) +
            (((size_t)g.s * A.max_nodes + rr / A.G) * A.hq + g.hk * A.G + rr % A.G) * D + 8 * c);
        unsigned char* dst = qsm + (R.two ? (x >> 7) * C::BUF : 0) + (c >> 3) * TT_HALF;
        for (int p = 0; p < R.nq; ++p) {
          const int y = (x & 127) + p * R.rpp;
          *reinterpret_cast<uint4*>(dst + y * 128 + (((c & 7) ^ (y & 7)) << 4)) = v;
        }
      }
      const bool tree = g.t1 * TT_KEYS > g.n;    // the segment reaches the tree's slots
      if (tree && t < g.k) {
        const int par = A.parents[(size_t)g.s * A.max_nodes + t];
        H.parent[t] = par;
        if (g.t1 == g.nt && (par < -1 || par >= t)) atomicOr(A.err, SPEC_DEV_ERR_TREE);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(sm_addr(&H.q_full));
      unsigned long long mask = 0;
      if (tree) {
        named_sync(1, 256);
        if (live) mask = ancestors(H.parent, (R.row0 + lr) / A.G);
      }
      float m = -INFINITY, l = 0.f;
      const bool any_live = __any_sync(0xffffffffu, live);
      const int nc = 4 / R.nq, c_lo = part * nc;  // this repetition's 32-key chunks of a tile
      for (int ti = R.two ? 0 : slot; ti < nt; ti += R.two ? 1 : 2) {
        const int k0 = (g.t0 + ti) * TT_KEYS;
        const bool first = ti == (R.two ? 0 : slot);
        wait(H.s_full + slot, jobs++);
        tc_fence_after();
        if (any_live) {
          const bool edge = k0 + TT_KEYS > g.n;
          auto bits_of = [&](int c) {            // visible keys of chunk c, for an edge tile
            const int sh = k0 + 32 * c - g.n;    // tree slot of the chunk's first key
            if (!live) return 0u;
            if (sh <= -32) return 0xffffffffu;
            if (sh < 0) return (uint32_t)(mask << -sh) | ((1u << -sh) - 1);
            return sh < TREE_N ? (uint32_t)(mask >> sh) : 0u;
          };
          float mt = -INFINITY;
          for (int c = c_lo; c < c_lo + nc; ++c) {
            uint32_t v[32];
            tmem_ld32(sT + 32 * c, v);
            const uint32_t bits = edge ? bits_of(c) : 0xffffffffu;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if ((bits >> i) & 1) mt = fmaxf(mt, __uint_as_float(v[i]));
          }
          mt *= A.scale_l2e;
          if (first) {
            m = mt;
          } else {
            const bool grow = live && mt > m + 8.f;
            if (__any_sync(0xffffffffu, grow)) {
              const float corr = grow ? ex2(m - mt) : 1.f;
              if (grow) m = mt;
              l *= corr;
              for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32];
                tmem_ld32(oT + 32 * c, v);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * corr);
                tmem_st32(oT + 32 * c, v);
              }
            }
          }
          const float mb = m == -INFINITY ? 0.f : m;
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            if (c >= c_lo && c < c_lo + nc) {    // warp-uniform: a warp's lanes lie in one repetition
              tmem_ld32(sT + 32 * c, v);
              const uint32_t bits = edge ? bits_of(c) : 0xffffffffu;
              uint32_t w[32];
              float s0 = 0.f, s1 = 0.f;
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                float p0 = ex2(fmaf(__uint_as_float(v[i]), A.scale_l2e, -mb));
                float p1 = ex2(fmaf(__uint_as_float(v[i + 1]), A.scale_l2e, -mb));
                if (!((bits >> i) & 1)) p0 = 0.f;
                if (!((bits >> (i + 1)) & 1)) p1 = 0.f;
                s0 += p0;
                s1 += p1;
                const uint32_t hi = pack_bf16(p0, p1);
                w[i / 2] = hi;
                w[16 + i / 2] = pack_bf16(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xFFFF0000u));
              }
              l += s0 + s1;
              tmem_st32(sT + 32 * c, w);
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = 0u;
              tmem_st32(sT + 32 * c, v);
            }
          }
          __syncwarp();
          tmem_wait_st();
        }
        // slots past the last node may hold anything: their V rows become zeros
        const int nk = g.n + g.k - k0;
        if (nk < TT_KEYS) {
          const uint32_t vi = 2 * (tiles + ti) + 1;
          wait(H.kv_full + vi % nbuf, vi / nbuf);
          unsigned char* vb = base + (vi % nbuf) * C::BUF;
          for (int i = r; i < (TT_KEYS - nk) * HALVES * 8; i += 128) {
            const int hf = i / ((TT_KEYS - nk) * 8), e = i % ((TT_KEYS - nk) * 8);
            *reinterpret_cast<uint4*>(vb + hf * TT_HALF + (nk + e / 8) * 128 + (e % 8) * 16) = make_uint4(0, 0, 0, 0);
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
      // 4 output values of row x (final ones where the block holds the segment alone), columns col .. col + 3
      auto emit4 = [&](int x, int col, float4 v) {
        if (wpart < 0) {
          const int rr = R.row0 + x;
          bf16_t* og = static_cast<bf16_t*>(A.out) +
                       (((size_t)g.s * A.max_nodes + rr / A.G) * A.hq + g.hk * A.G + rr % A.G) * D + col;
          *reinterpret_cast<uint2*>(og) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
        } else {
          *reinterpret_cast<float4*>(A.part_o + (((size_t)blockIdx.x * 2 + wpart) * A.rows + x) * D + col) = v;
        }
      };
      auto emit_ml = [&](int x, float mm, float ll) {
        if (wpart >= 0) A.part_ml[((size_t)blockIdx.x * 2 + wpart) * A.rows + x] = make_float2(mm, ll);
      };
      // each group waits for its own slot's last P V; the barriers pass that on
      if (R.two || slot < nt) wait(H.o_done + slot, jobs - 1);
      if (R.two) {
        tc_fence_after();
        const float w = wpart < 0 ? 1.f / l : 1.f;
        if (any_live) {
          for (int c = 0; c < D / 32; ++c) {
            uint32_t v[32];
            tmem_ld32(oT + 32 * c, v);
            if (live) {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                emit4(lr, 32 * c + i, make_float4(__uint_as_float(v[i]) * w, __uint_as_float(v[i + 1]) * w,
                                                  __uint_as_float(v[i + 2]) * w, __uint_as_float(v[i + 3]) * w));
            }
          }
          if (live) emit_ml(lr, m, l);
        }
      } else {
        const bool both = nt > 1;                // slot 1 had tiles
        // statistics of the row's repetitions in both slots, in Q's bytes: a slot's last P V comes after every S but
        // the one of a single tile, which slot 1 has not waited for
        if (!both) named_sync(1, 256);
        float2* ml = reinterpret_cast<float2*>(qsm);
        ml[slot * 128 + r] = make_float2(live ? m : -INFINITY, live ? l : 0.f);
        tc_fence_before();
        named_sync(1, 256);
        tc_fence_after();
        float M = -INFINITY, L = 0.f;
        for (int p = 0; p < R.nq; ++p)
          M = fmaxf(M, fmaxf(ml[p * R.rpp + r % R.rpp].x, ml[128 + p * R.rpp + r % R.rpp].x));
        const float Mb = M == -INFINITY ? 0.f : M;
        for (int p = 0; p < R.nq; ++p) {
          const float2 a = ml[p * R.rpp + r % R.rpp], b = ml[128 + p * R.rpp + r % R.rpp];
          L += a.y * ex2(a.x - Mb) + b.y * ex2(b.x - Mb);
        }
        const float inv = wpart < 0 ? 1.f / L : 1.f;
        const float w0 = ex2(ml[r].x - Mb) * inv, w1 = ex2(ml[128 + r].x - Mb) * inv;
        named_sync(1, 256);                      // the staged output takes the same bytes
        if (slot == 0 && live && part == 0) emit_ml(lr, M, L);
        // group `slot` has columns slot D / 2 .. of both slots' outputs
        const uint32_t o0 = tmem + lanes + OCOL + slot * (D / 2), o1 = o0 + D;
        float4* stage = reinterpret_cast<float4*>(qsm + slot * 16384);   // [128 lanes][32 columns]
        for (int c = 0; c < D / 64; ++c) {
          uint32_t v[32], u[32];
          tmem_ld32(o0 + 32 * c, v);
          if (both) tmem_ld32(o1 + 32 * c, u);
          float4 x[8];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float y = __uint_as_float(v[i]) * w0;
            if (both) y = fmaf(__uint_as_float(u[i]), w1, y);
            reinterpret_cast<float*>(x)[i] = y;
          }
          const int col = slot * (D / 2) + 32 * c;
          if (R.nq == 1) {
            if (live)
#pragma unroll
              for (int i = 0; i < 8; ++i) emit4(lr, col + 4 * i, x[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) stage[r * 8 + (i ^ (r & 7))] = x[i];
            named_sync(2 + slot, 128);
            for (int i = r; i < R.rows * 8; i += 128) {
              const int y = i / 8, pc = i % 8;
              float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
              for (int p = 0; p < R.nq; ++p) {
                const int ln = p * R.rpp + y;
                const float4 z = stage[ln * 8 + (pc ^ (ln & 7))];
                a.x += z.x; a.y += z.y; a.z += z.z; a.w += z.w;
              }
              emit4(y, col + 4 * pc, a);
            }
            named_sync(2 + slot, 128);
          }
        }
      }
      tc_fence_before();
      named_sync(1, 256);                        // O, Q and the statistics are free
      if (wpart == 1 && t == 0)
        A.joint[blockIdx.x] = make_int4(g.s, g.rt, g.hk, parts_until(walk.U, blockIdx.x, walk.blocks, walk.u1 + g.nt - g.t1));
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
// parts in key order. One warp per row.
constexpr int JOIN_WARPS = 8;

template <int D, class KT>
__global__ void __launch_bounds__(JOIN_WARPS * 32) k_tree_join(const __grid_constant__ TreeArgs A) {
  pdl_wait();
  pdl_trigger();
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

// Shape of a launch, from sizes and types alone.
struct TreePlan {
  bool tc;                  // bf16 cache: the tensor-core form
  int rows, tile_k;
  int max_blocks;           // of any grid (the workspace is sized without a device)
  size_t ml, joint, total;  // workspace: outputs at 0, statistics, joints
  TreePlan(const spec_kv_view& kv, int max_nodes, int hq) {
    const int G = hq / kv.n_kv_heads;
    tc = kv.dtype == SPEC_BF16;
    if (tc) {
      // tiles of at most 256 rows, whole nodes, as even as they come
      const int most = std::max(1, 256 / G), nrt = (max_nodes + most - 1) / most;
      rows = (max_nodes + nrt - 1) / nrt * G;
      tile_k = TT_KEYS;
      max_blocks = 160;     // one block per SM
    } else {
      rows = FM_ROWS;
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
  if ((double)kv->max_pages * kv->page_size / FM_KEYS * ((double)max_nodes * hq / FM_ROWS + kv->n_kv_heads) > 2e9)
    return set_last_error(SPEC_ERR_UNSUPPORTED, "block table too long for this many heads");
  return SPEC_OK;
}

template <int D, class KT>
cudaError_t join(const TreeArgs& A, int blocks, cudaStream_t st) {
  return launch_k(k_tree_join<D, KT>, dim3(blocks, (A.rows + JOIN_WARPS - 1) / JOIN_WARPS), dim3(JOIN_WARPS * 32), 0, st, A);
}

template <int D>
cudaError_t launch_fma(const TreeArgs& A, int blocks, cudaStream_t st) {
  cudaError_t e = allow_dyn_smem(k_tree_fma<D>);
  if (e == cudaSuccess) e = launch_k(k_tree_fma<D>, dim3(blocks), dim3(FM_THREADS), sizeof(FmSmem<D>), st, A);
  return e == cudaSuccess ? join<D, float>(A, blocks, st) : e;
}

template <int D>
cudaError_t launch_tc(const TreeArgs& A, const CUtensorMap& map, int kb, int blocks, cudaStream_t st) {
  using C = TtCfg<D>;
  const bool two = A.rows > 128;
  cudaError_t e = allow_dyn_smem(k_tree_tc<D>);
  if (e == cudaSuccess)
    e = launch_k(k_tree_tc<D>, dim3(blocks), dim3(TT_THREADS), C::smem(two), st, map, A, C::nbuf(two), C::q_bytes(two), kb);
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
  if (!(scale > 0.f) || !(scale < INFINITY)) return set_last_error(SPEC_ERR_ARG, "scale must be positive");
  if (!aligned16(q_dev) || !aligned16(out_dev) || !aligned16(ws_dev))
    return set_last_error(SPEC_ERR_ARG, "q, out and the workspace must be 16-byte aligned");
  const int d = kv->head_dim;
  const TreePlan plan(*kv, max_nodes, n_q_heads);
  if (ws_bytes < plan.total) return set_last_error(SPEC_ERR_ARG, "workspace too small");
  const int sms = sm_count();
  if (sms < 1) return set_last_error(SPEC_ERR_CUDA, "no device");
  char* w = static_cast<char*>(ws_dev);
  const TreeArgs A{*kv, q_dev, out_dev, cache_len_dev, n_nodes_dev, parents_dev, err_dev, reinterpret_cast<float*>(w),
                   reinterpret_cast<float2*>(w + plan.ml), reinterpret_cast<int4*>(w + plan.joint), layer, n_seq,
                   max_nodes, n_q_heads, n_q_heads / kv->n_kv_heads, plan.rows, plan.tile_k, scale * LOG2E};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
  const int blocks = std::min((plan.tc ? 1 : 2) * sms, plan.max_blocks);
  cudaError_t e;
  if (plan.tc) {
    // a box never straddles pages: the largest power of two up to a tile that divides a page
    int kb = 16;
    while (kb < TT_KEYS && kv->page_size % (2 * kb) == 0) kb *= 2;
    CUtensorMap map;
    if (kv_make_half_map(&map, kv->kv_dev, d, kv->page_size, kv->n_layers * kv->n_kv_heads * 2, kv->n_pages,
                         (size_t)kv->n_layers * kv->n_kv_heads * 2 * kv->page_size * d, kb))
      return set_last_error(SPEC_ERR_UNSUPPORTED, "tensor map encoding failed");
    e = d == 128 ? launch_tc<128>(A, map, kb, blocks, st) : launch_tc<64>(A, map, kb, blocks, st);
  } else {
    e = d == 128 ? launch_fma<128>(A, blocks, st) : launch_fma<64>(A, blocks, st);
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? SPEC_OK : set_last_error(SPEC_ERR_CUDA, cudaGetErrorString(e));
}
