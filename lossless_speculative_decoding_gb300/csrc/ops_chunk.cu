// Kernel-level entry point: attention of chunks of new tokens over the paged cache.
//
// For token i of a sequence with n positions before the chunk: out = sum_j w_j V_j
// over j <= n + i, w the softmax of scale q.K_j, and lse = log sum_j exp(scale q.K_j).
// The rows of the query heads that share a kv head (row r = token r / G, head r % G,
// G query heads per kv head) meet the same keys, so a (sequence, row tile, kv head)
// reads its keys, those up to its last token's position, once for all of its rows.
//
// Work split. Units of tile_k keys are numbered sequence by sequence, row tile by row
// tile, kv head by kv head; block c of B takes units [c U / B, (c + 1) U / B) of all U,
// whatever the lengths, which stay on the device. At most two of a block's (sequence,
// tile, head) segments are shared with other blocks: of a shared one, each block
// leaves (output, maximum, sum) in the workspace and a second launch joins the parts
// in key order.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "chunk.cuh"
#include "tc_attn.cuh"

namespace spec {
namespace {

constexpr int CH_MAX_G = 128;                    // query heads per kv head

struct ChunkArgs {
  spec_kv_view kv;
  ChunkIndex ix;
  const void* q;
  void* out;
  float* lse;
  int32_t* err;
  float* part_o;       // [blocks][2][rows][d]: part 0 of a block began in an earlier block, part 1 goes on in the next
  float2* part_ml;     // [blocks][2][rows]: maximum (log2 units), sum
  int4* joint;         // [blocks]: (first row, row tile, kv head, parts and rows) of the shared segment that starts in a block
  int layer, hq, G;
  int rows;            // rows of a tile
  int tile_k;          // keys of a unit
  float scale_l2e;     // scale * log2 e
};

// Segment: tiles [t0, t1) of nt key tiles of (sequence s, row tile rt, kv head hk).
struct ChunkSeg {
  int s, rt, hk, nt, t0, t1;
  int n, m, r0;                                  // positions before the chunk, its tokens, its first row
};

// Key tiles of row tile rt: up to the position of its last token.
__device__ __forceinline__ int chunk_tiles(const ChunkArgs& A, int n, int m, int rt) {
  const int last = min(m - 1, (int)(((long long)(rt + 1) * A.rows - 1) / A.G));
  return (n + last + A.tile_k) / A.tile_k;
}
__device__ __forceinline__ int chunk_row_tiles(const ChunkArgs& A, int m) {
  return (int)(((long long)m * A.G + A.rows - 1) / A.rows);
}

// A block's walk over its units. All threads of the block call init (it has
// block barriers); next() is called by whole warps.
struct ChunkWalk {
  long long u, u1, U;                            // units left: [u, u1) of U
  int blocks;                                    // blocks that have units (no more than there are units)
  int s, rt, in;                                 // unit u is number `in` of row tile rt (of all heads) of sequence s
  const ChunkArgs* A;

  __device__ static long long units_of(const ChunkArgs& A, int s) {
    const ChunkSeq z(A.ix, s);
    long long sum = 0;
    for (int rt = 0, nrt = chunk_row_tiles(A, z.m); rt < nrt; ++rt) sum += chunk_tiles(A, z.n, z.m, rt);
    return sum * A.kv.n_kv_heads;
  }
  template <int THREADS>
  __device__ void init(const ChunkArgs& args) {
    __shared__ long long w_sum[THREADS / 32];
    __shared__ int s_seq, s_rt, s_in;
    A = &args;
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    const int per = (args.ix.n_seq + THREADS - 1) / THREADS;
    const int a = min(t * per, args.ix.n_seq), a1 = min(a + per, args.ix.n_seq);
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
    if (u < u1 && at <= u && u < at + sum) {     // one thread's sequences hold unit u
      int i = a, r = 0;
      for (long long c; at + (c = units_of(args, i)) <= u; ++i) at += c;
      const ChunkSeq z(args.ix, i);
      for (long long c; at + (c = (long long)chunk_tiles(args, z.n, z.m, r) * args.kv.n_kv_heads) <= u; ++r) at += c;
      s_seq = i;
      s_rt = r;
      s_in = (int)(u - at);
    }
    __syncthreads();
    if (u < u1) {
      s = s_seq;
      rt = s_rt;
      in = s_in;
    }
  }
  __device__ bool next(ChunkSeg& g) {
    if (u >= u1) return false;
    ChunkSeq z(A->ix, s);
    for (;;) {
      if (rt < chunk_row_tiles(*A, z.m)) {
        g.nt = chunk_tiles(*A, z.n, z.m, rt);
        if (in < g.nt * A->kv.n_kv_heads) break;
        in = 0;
        ++rt;
        continue;
      }
      in = rt = 0;                               // the next sequence that is not padded, of 32 at a time
      for (++s;; s += 32) {
        if (s >= A->ix.n_seq) return false;      // (only if the lengths changed meanwhile)
        const int i = s + (threadIdx.x & 31);
        const uint32_t live = __ballot_sync(0xffffffffu, i < A->ix.n_seq && ChunkSeq(A->ix, i).m > 0);
        if (live) {
          s += __ffs(live) - 1;
          break;
        }
      }
      z = ChunkSeq(A->ix, s);
    }
    g.s = s;
    g.n = z.n;
    g.m = z.m;
    g.r0 = z.r0;
    g.rt = rt;
    g.hk = in / g.nt;
    g.t0 = in - g.hk * g.nt;
    g.t1 = (int)min((long long)g.nt, g.t0 + (u1 - u));
    u += g.t1 - g.t0;
    in += g.t1 - g.t0;
    return true;
  }
};

// Part of a shared segment that this block leaves: -1 none (the block holds the
// segment alone), 0 or 1.
__device__ __forceinline__ int part_of(const ChunkSeg& g) { return g.t0 > 0 ? 0 : (g.t1 < g.nt ? 1 : -1); }

// Description of the shared segment that starts in this block (the walk is behind
// its first part): the blocks up to that of its last unit have parts of it (unit u
// is in block floor(((u + 1) blocks - 1) / U)).
__device__ __forceinline__ int4 joint_of(const ChunkWalk& w, const ChunkSeg& g, int rows) {
  const long long end = w.u1 + g.nt - g.t1;
  const int parts = (int)((end * w.blocks - 1) / w.U) - (int)blockIdx.x + 1;
  return make_int4(g.r0, g.rt, g.hk, parts << 16 | rows);
}

// ---------------------------------------------------------------------------
// FMA form. 128 threads, 32 rows and 64 keys at a time, everything in fp32 (the
// matrix instructions round their operands). Thread (ty, tx) = (t / 16, t % 16) has
// rows 4 ty .. 4 ty + 3, in the score product keys tx + 16 j, in the output product
// dims 4 tx + 64 j. Rows of K are padded by 16 bytes, so eight lanes' reads cover
// all banks.
constexpr int CF_THREADS = 128;
constexpr int CF_ROWS = 32;
constexpr int CF_KEYS = 64;

template <int D>
struct CfSmem {
  static constexpr int KST = D + 4, PST = CF_KEYS + 4;
  float q[CF_ROWS][D];
  float k[CF_KEYS][KST];
  float v[CF_KEYS][D];
  float p[CF_ROWS][PST];
  int page[CF_KEYS];
};

template <class KT>
__device__ __forceinline__ float4 load4(const void* base, size_t e) {
  if constexpr (sizeof(KT) == 4) {
    return *reinterpret_cast<const float4*>(static_cast<const float*>(base) + e);
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + e);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u));
  }
}

template <class KT, int D>
__global__ void __launch_bounds__(CF_THREADS) k_chunk_fma(const __grid_constant__ ChunkArgs A) {
  using L = CfSmem<D>;
  extern __shared__ __align__(16) unsigned char sm_raw[];
  L& sm = *reinterpret_cast<L*>(sm_raw);
  constexpr int NV = D / 64;                     // float4 of dims per thread
  const int t = threadIdx.x, tx = t & 15, ty = t >> 4;
  const int P = A.kv.page_size;
  pdl_wait();
  pdl_trigger();
  ChunkWalk walk;
  walk.init<CF_THREADS>(A);
  if (t == 0) A.joint[blockIdx.x] = make_int4(0, 0, 0, 0);
  if (blockIdx.x == 0)
    for (int s = t; s < A.ix.n_seq; s += CF_THREADS)
      if (ChunkSeq(A.ix, s).bad) atomicOr(A.err, DERR_POS);
  const size_t page_elems = (size_t)A.kv.n_layers * A.kv.n_kv_heads * 2 * P * D;
  ChunkSeg g;
  while (walk.next(g)) {
    const int row0 = g.rt * CF_ROWS, nrows = min(CF_ROWS, g.m * A.G - row0);
    const int32_t* bt = A.kv.block_table_dev + (size_t)g.s * A.kv.max_pages;
    const size_t plane = (((size_t)A.layer * A.kv.n_kv_heads + g.hk) * 2) * P * D;
    auto q_at = [&](int r) {                     // of row r of the tile
      const int rr = row0 + r;
      return (((size_t)g.r0 + rr / A.G) * A.hq + g.hk * A.G + rr % A.G) * D;
    };
    __syncthreads();                             // the last segment's reads of q are done
    for (int i = t; i < CF_ROWS * (D / 4); i += CF_THREADS) {
      const int r = i / (D / 4), c = 4 * (i % (D / 4));
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < nrows) {
        v = load4<KT>(A.q, q_at(r) + c);
        v = make_float4(v.x * A.scale_l2e, v.y * A.scale_l2e, v.z * A.scale_l2e, v.w * A.scale_l2e);
      }
      *reinterpret_cast<float4*>(&sm.q[r][c]) = v;
    }
    float m[4], l[4];
    float4 o[4][NV];
    int seen[4];                                 // positions that the row sees
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
      seen[i] = g.n + min(row0 + 4 * ty + i, g.m * A.G - 1) / A.G + 1;
#pragma unroll
      for (int j = 0; j < NV; ++j) o[i][j] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int tile = g.t0; tile < g.t1; ++tile) {
      const int k0 = tile * CF_KEYS, nk = min(CF_KEYS, g.n + g.m - k0);
      __syncthreads();                           // the last tile's reads of k, v and p are done
      if (t < CF_KEYS) {
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
#pragma unroll 4
      for (int i = t; i < CF_KEYS * (D / 4); i += CF_THREADS) {
        const int key = i / (D / 4), c = 4 * (i % (D / 4)), page = sm.page[key];
        float4 kk = make_float4(0.f, 0.f, 0.f, 0.f), vv = kk;
        if (page >= 0) {
          const size_t e = page * page_elems + plane + (size_t)((k0 + key) % P) * D + c;
          kk = load4<KT>(A.kv.kv_dev, e);
          vv = load4<KT>(A.kv.kv_dev, e + (size_t)P * D);
        }
        *reinterpret_cast<float4*>(&sm.k[key][c]) = kk;
        *reinterpret_cast<float4*>(&sm.v[key][c]) = vv;
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
        float mt = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (k0 + tx + 16 * j >= seen[i]) x[i][j] = -INFINITY;
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
      for (int key = 0; key < CF_KEYS; key += 4) {
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
      const int r = 4 * ty + i;
      if (r >= nrows) continue;
      if (part < 0) {
        const float inv = 1.f / l[i];
        const size_t e = q_at(r);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const float4 y = make_float4(o[i][j].x * inv, o[i][j].y * inv, o[i][j].z * inv, o[i][j].w * inv);
          if constexpr (sizeof(KT) == 4)
            *reinterpret_cast<float4*>(static_cast<float*>(A.out) + e + 4 * tx + 64 * j) = y;
          else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(A.out) + e + 4 * tx + 64 * j) =
                make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
        }
        if (A.lse && tx == 0) A.lse[e / D] = (m[i] + log2f(l[i])) * LN2;
      } else {
        const size_t pr = ((size_t)blockIdx.x * 2 + part) * A.rows + r;
#pragma unroll
        for (int j = 0; j < NV; ++j) *reinterpret_cast<float4*>(A.part_o + pr * D + 4 * tx + 64 * j) = o[i][j];
        if (tx == 0) A.part_ml[pr] = make_float2(m[i], l[i]);
      }
    }
    if (part == 1 && t == 0) A.joint[blockIdx.x] = joint_of(walk, g, nrows);
  }
}

// ---------------------------------------------------------------------------
// Joins the parts of the segment that starts in block blockIdx.x and ends in a
// later one: M = max m_c, out = sum_c o_c 2^(m_c - M) / sum_c l_c 2^(m_c - M),
// parts in key order. One warp per row; a row's statistics and its first eight
// parts are on their way together. (A part may have seen nothing of a row: m = -inf,
// l = 0; the one with the row's first key has not.)
constexpr int CJ_WARPS = 8;

template <int D, class KT>
__global__ void __launch_bounds__(CJ_WARPS * 32) k_chunk_join(const __grid_constant__ ChunkArgs A) {
  pdl_wait();
  pdl_trigger();
  const int4 jt = __ldcg(A.joint + blockIdx.x);
  const int r = blockIdx.y * CJ_WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
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
  const size_t row = ((size_t)jt.x + rr / A.G) * A.hq + jt.z * A.G + rr % A.G;
  KT* og = static_cast<KT*>(A.out) + row * D + NV * lane;
  const float inv = 1.f / l;
  if (A.lse && lane == 0) A.lse[row] = (M + log2f(l)) * LN2;
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
struct ChunkPlan {
  int rows, tile_k;
  int max_blocks;           // of any grid (the workspace is sized without a device)
  size_t ml, joint, total;  // workspace: outputs at 0, statistics, joints
  bool chain;               // few tokens: the tree attention's kernel, each node the next one's parent
  ChunkPlan(const spec_kv_view& kv, int max_new, int hq) {
    chain = kv.dtype == SPEC_BF16 && max_new <= SPEC_TREE_MAX_NODES && max_new * (hq / kv.n_kv_heads) <= 128;
    if (chain) {
      total = chain_ws_bytes(kv, max_new, hq);
      return;
    }
    rows = CF_ROWS;
    tile_k = CF_KEYS;
    max_blocks = 320;       // two blocks per SM
    ml = (size_t)max_blocks * 2 * rows * kv.head_dim * sizeof(float);
    joint = (ml + (size_t)max_blocks * 2 * rows * sizeof(float2) + 15) / 16 * 16;
    total = joint + (size_t)max_blocks * sizeof(int4);
  }
};

int check_attention(const spec_kv_view* kv, int n_seq, int max_new, int hq) {
  const int rc = check_chunks(kv, n_seq, hq);
  if (rc) return rc;
  if (max_new < 1) return set_last_error(SPEC_ERR_ARG, "max_new >= 1 required");
  if (hq / kv->n_kv_heads > CH_MAX_G) return set_last_error(SPEC_ERR_UNSUPPORTED, "more than 128 query heads per kv head");
  // a row tile's units, and a sequence's rows of a kv head, are counted in 32 bits
  if ((double)kv->max_pages * kv->page_size / CF_KEYS * kv->n_kv_heads > 2e9 ||
      (double)std::min<int64_t>(max_new, (int64_t)kv->max_pages * kv->page_size) * (hq / kv->n_kv_heads) > 2e9)
    return set_last_error(SPEC_ERR_UNSUPPORTED, "block table too long for this many heads");
  return SPEC_OK;
}

template <int D, class KT>
cudaError_t launch_fma(const ChunkArgs& A, int blocks, cudaStream_t st) {
  cudaError_t e = allow_dyn_smem_once<k_chunk_fma<KT, D>>();
  if (e == cudaSuccess) e = launch_k(k_chunk_fma<KT, D>, dim3(blocks), dim3(CF_THREADS), sizeof(CfSmem<D>), st, A);
  if (e != cudaSuccess) return e;
  return launch_k(k_chunk_join<D, KT>, dim3(blocks, (A.rows + CJ_WARPS - 1) / CJ_WARPS), dim3(CJ_WARPS * 32), 0, st, A);
}

}  // namespace
}  // namespace spec

using namespace spec;

extern "C" int64_t spec_chunk_attention_ws_bytes(const spec_kv_view* kv, int n_seq, int max_new, int n_q_heads) {
  const int rc = check_attention(kv, n_seq, max_new, n_q_heads);
  if (rc) return rc;
  return (int64_t)ChunkPlan(*kv, max_new, n_q_heads).total;
}

extern "C" int spec_chunk_attention(const spec_kv_view* kv, int layer, const void* q_dev, int n_rows, int n_seq, int max_new,
                                    int n_q_heads, const int32_t* row_start_dev, const int32_t* n_new_dev,
                                    const int32_t* cache_len_dev, float scale, void* out_dev, float* out_lse_dev,
                                    void* ws_dev, size_t ws_bytes, int32_t* err_dev, uintptr_t cuda_stream) {
  int rc = check_attention(kv, n_seq, max_new, n_q_heads);
  if (rc == SPEC_OK) rc = check_layer_rows(kv, layer, n_rows, max_new);
  if (rc) return rc;
  if (!q_dev || !out_dev || !row_start_dev || !n_new_dev || !cache_len_dev || !ws_dev || !err_dev)
    return set_last_error(SPEC_ERR_ARG, "null pointer argument");
  if (!(scale > 0.f) || !(scale * LOG2E < INFINITY)) return set_last_error(SPEC_ERR_ARG, "scale must be positive, and finite times log2 e");
  if (!aligned16(q_dev) || !aligned16(out_dev) || !aligned16(ws_dev))
    return set_last_error(SPEC_ERR_ARG, "q, out and the workspace must be 16-byte aligned");
  const int d = kv->head_dim;
  const int64_t bytes = (int64_t)n_rows * n_q_heads * d * (kv->dtype == SPEC_F32 ? 4 : 2);
  if (out_dev != q_dev && spans_meet(out_dev, bytes, q_dev, bytes))
    return set_last_error(SPEC_ERR_ARG, "out overlaps q without being the same array");
  const ChunkPlan plan(*kv, max_new, n_q_heads);
  if (ws_bytes < plan.total) return set_last_error(SPEC_ERR_ARG, "workspace too small");
  const int sms = sm_count_once();
  if (sms < 1) return set_last_error(SPEC_ERR_CUDA, "no device");
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
  if (plan.chain)
    return launch_chain_attention(*kv, layer, q_dev, n_rows, n_seq, max_new, n_q_heads, row_start_dev, n_new_dev, cache_len_dev,
                                  scale * LOG2E, out_dev, out_lse_dev, ws_dev, err_dev, sms, st);
  char* w = static_cast<char*>(ws_dev);
  const ChunkArgs A{*kv, ChunkIndex{row_start_dev, n_new_dev, cache_len_dev, n_seq, n_rows, max_new, kv->max_pages * kv->page_size},
                    q_dev, out_dev, out_lse_dev, err_dev, reinterpret_cast<float*>(w), reinterpret_cast<float2*>(w + plan.ml),
                    reinterpret_cast<int4*>(w + plan.joint), layer, n_q_heads, n_q_heads / kv->n_kv_heads, plan.rows,
                    plan.tile_k, scale * LOG2E};
  const int blocks = std::min(2 * sms, plan.max_blocks);
  cudaError_t e;
  if (kv->dtype == SPEC_F32) e = d == 128 ? launch_fma<128, float>(A, blocks, st) : launch_fma<64, float>(A, blocks, st);
  else e = d == 128 ? launch_fma<128, bf16_t>(A, blocks, st) : launch_fma<64, bf16_t>(A, blocks, st);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? SPEC_OK : set_last_error(SPEC_ERR_CUDA, cudaGetErrorString(e));
}
