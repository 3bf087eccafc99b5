// Kernel-level entry point: attention of chunks of new tokens over the paged cache.
//
// For token i of a sequence with n positions before the chunk: out = sum_j w_j V_j
// over j <= n + i, w the softmax of scale q.K_j, and lse = log sum_j exp(scale q.K_j).
// The rows of the query heads that share a kv head (row r = token r / G, head r % G,
// G query heads per kv head) meet the same keys, so a (sequence, row tile, kv head)
// reads its keys, those up to its last token's position, once for all of its rows. A
// row tile has whole tokens; where one token's heads are too many for it (FMA form),
// the heads of a kv head are several parts, each of which counts as a kv head.
//
// Work split. Units of 64 or 128 keys are numbered sequence by sequence, row tile by row
// tile, kv head by kv head; block c of B takes units [c U / B, (c + 1) U / B) of all U,
// whatever the lengths, which stay on the device. At most two of a block's (sequence,
// tile, head) segments are shared with other blocks: of a shared one, each block
// leaves (output, maximum, sum) in the workspace and a second launch joins the parts
// in key order. A segment begins with a few units without keys, for what its start and
// its end take.
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
  int layer, hq;
  int G;               // heads of a part
  int parts, heads;    // parts of a kv head's heads; kv heads x parts
  int tok;             // tokens of a row tile
  int rows;            // tok G
  int key_bits;        // log2 of a unit's keys
  int extra;           // units without keys of a segment
  float scale_l2e;     // scale * log2 e
  __device__ int deadlines() const { return segment_deadlines(ix.capacity); }
};

// Segment: tiles [t0, t1) of nt key tiles of (sequence s, row tile rt, head part hk).
struct ChunkSeg {
  int s, rt, hk, nt, t0, t1;
  int n, m, r0;                                  // positions before the chunk, its tokens, its first row
};

// Key tiles of row tile rt: up to the position of its last token.
__device__ __forceinline__ int chunk_tiles(const ChunkArgs& A, int n, int m, int rt) {
  return (n + min(m, (rt + 1) * A.tok) + (1 << A.key_bits) - 1) >> A.key_bits;
}
__device__ __forceinline__ int chunk_row_tiles(const ChunkArgs& A, int m) { return (m + A.tok - 1) / A.tok; }

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
    for (int rt = 0, nrt = chunk_row_tiles(A, z.m); rt < nrt; ++rt) sum += chunk_tiles(A, z.n, z.m, rt) + A.extra;
    return sum * A.heads;
  }
  // Inclusive prefix sum over a warp.
  __device__ static long long scan(long long v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, v, o);
      if ((threadIdx.x & 31) >= o) v += x;
    }
    return v;
  }
  // This block's share of U units.
  __device__ void share(long long total) {
    U = total;
    blocks = (int)min((long long)gridDim.x, max(U, 1ll));
    // floor(U b / blocks) = (U / blocks) b + floor((U % blocks) b / blocks)
    const long long each = U / blocks;
    const int rest = (int)(U - each * blocks), b = min((int)blockIdx.x, blocks), b1 = min((int)blockIdx.x + 1, blocks);
    u = each * b + rest * b / blocks;
    u1 = each * b1 + rest * b1 / blocks;
  }
  // The row tile of sequence s, whose units start at `at`, that has unit u; by a warp.
  __device__ void find_tile(long long at) {
    const int lane = threadIdx.x & 31;
    const ChunkSeq z(A->ix, s);
    for (rt = 0;; rt += 32) {
      const int r = rt + lane;
      const long long mine = r < chunk_row_tiles(*A, z.m) ? (long long)(chunk_tiles(*A, z.n, z.m, r) + A->extra) * A->heads : 0;
      const long long end = at + scan(mine);
      const uint32_t past = __ballot_sync(0xffffffffu, end > u);
      if (past) {
        const int l = __ffs(past) - 1;
        in = (int)(u - __shfl_sync(0xffffffffu, end - mine, l));
        rt += l;
        return;
      }
      at = __shfl_sync(0xffffffffu, end, 31);
      if (rt > chunk_row_tiles(*A, z.m)) return;   // (only if the lengths changed meanwhile)
    }
  }
  template <int THREADS>
  __device__ void init(const ChunkArgs& args) {
    __shared__ long long w_sum[32];
    __shared__ long long s_at;
    __shared__ int s_seq;
    A = &args;
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    s = rt = in = 0;
    if (args.ix.n_seq <= 32) {
      // few sequences: a warp adds up the row tiles of one
      for (int i = w; i < args.ix.n_seq; i += THREADS / 32) {
        const ChunkSeq z(args.ix, i);
        long long sum = 0;
        for (int r = lane, nrt = chunk_row_tiles(args, z.m); r < nrt; r += 32) sum += chunk_tiles(args, z.n, z.m, r) + args.extra;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) w_sum[i] = sum * args.heads;
      }
      __syncthreads();
      const long long mine = lane < args.ix.n_seq ? w_sum[lane] : 0, end = scan(mine);
      share(__shfl_sync(0xffffffffu, end, 31));
      if (u < u1) {
        s = __ffs(__ballot_sync(0xffffffffu, end > u)) - 1;
        find_tile(__shfl_sync(0xffffffffu, end - mine, s));
      }
      return;
    }
    // many: a thread adds up the sequences of its share
    const int per = (args.ix.n_seq + THREADS - 1) / THREADS;
    const int a = min(t * per, args.ix.n_seq), a1 = min(a + per, args.ix.n_seq);
    long long sum = 0;
    for (int i = a; i < a1; ++i) sum += units_of(args, i);
    const long long inc = scan(sum);
    if (lane == 31) w_sum[w] = inc;
    __syncthreads();
    long long before = 0, total = 0;
    for (int i = 0; i < THREADS / 32; ++i) {
      if (i < w) before += w_sum[i];
      total += w_sum[i];
    }
    share(total);
    long long at = before + inc - sum;
    if (u < u1 && at <= u && u < at + sum) {     // one thread's sequences hold unit u
      int i = a;
      for (long long c; at + (c = units_of(args, i)) <= u; ++i) at += c;
      s_seq = i;
      s_at = at;
    }
    __syncthreads();
    if (u < u1) {
      s = s_seq;
      find_tile(s_at);
    }
  }
  __device__ bool next(ChunkSeg& g) {
    ChunkSeq z(A->ix, u < u1 ? s : 0);
    while (u < u1) {
      if (rt >= chunk_row_tiles(*A, z.m)) {
        in = rt = 0;                             // the next sequence that is not padded, of 32 at a time
        for (++s;; s += 32) {
          if (s >= A->ix.n_seq) return false;    // (only if the lengths changed meanwhile)
          const int i = s + (threadIdx.x & 31);
          const uint32_t live = __ballot_sync(0xffffffffu, i < A->ix.n_seq && ChunkSeq(A->ix, i).m > 0);
          if (live) {
            s += __ffs(live) - 1;
            break;
          }
        }
        z = ChunkSeq(A->ix, s);
        continue;
      }
      g.nt = chunk_tiles(*A, z.n, z.m, rt);
      const int len = g.nt + A->extra;
      if (in >= len * A->heads) {
        in = 0;
        ++rt;
        continue;
      }
      g.hk = in / len;
      const int from = in - g.hk * len, take = (int)min((long long)(len - from), u1 - u);
      u += take;
      in += take;
      g.t0 = max(0, from - A->extra);
      g.t1 = from + take - A->extra;
      if (g.t1 <= g.t0) continue;                // (none with keys)
      g.s = s;
      g.n = z.n;
      g.m = z.m;
      g.r0 = z.r0;
      g.rt = rt;
      return true;
    }
    return false;
  }
};

// Part of a shared segment that this block leaves: -1 none (the block holds the
// segment alone), 0 or 1.
__device__ __forceinline__ int part_of(const ChunkSeg& g) { return g.t0 > 0 ? 0 : (g.t1 < g.nt ? 1 : -1); }

// Of a row: its place in rows of [token][query head]; x = its number in the segment's tile.
__device__ __forceinline__ size_t row_at(const ChunkArgs& A, int r0, int rt, int hk, int x) {
  return ((size_t)r0 + (size_t)rt * A.tok + x / A.G) * A.hq + hk * A.G + x % A.G;
}

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
constexpr int CF_KEYS = 64;                      // 2^6 (key_bits)

template <int D>
struct CfSmem {
  static constexpr int KST = D + 4, PST = CF_KEYS + 4;
  float q[CF_ROWS][D];
  float k[CF_KEYS][KST];
  float v[CF_KEYS][D];
  float p[CF_ROWS][PST];
  int page[CF_KEYS];
};

template <int D>
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
    const int ntok = min(A.tok, g.m - g.rt * A.tok), nrows = ntok * A.G;
    const int32_t* bt = A.kv.block_table_dev + (size_t)g.s * A.kv.max_pages;
    const size_t plane = (((size_t)A.layer * A.kv.n_kv_heads + g.hk / A.parts) * 2) * P * D;
    auto q_at = [&](int r) { return row_at(A, g.r0, g.rt, g.hk, r) * D; };
    __syncthreads();                             // the last segment's reads of q are done
    for (int i = t; i < CF_ROWS * (D / 4); i += CF_THREADS) {
      const int r = i / (D / 4), c = 4 * (i % (D / 4));
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < nrows) v = *reinterpret_cast<const float4*>(static_cast<const float*>(A.q) + q_at(r) + c);
      *reinterpret_cast<float4*>(&sm.q[r][c]) = v;
    }
    float m[4], l[4];
    float4 o[4][NV];
    int seen[4];                                 // positions that the row sees
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
      seen[i] = g.n + g.rt * A.tok + min(4 * ty + i, nrows - 1) / A.G + 1;
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
          const float* e = static_cast<const float*>(A.kv.kv_dev) + page * page_elems + plane + (size_t)((k0 + key) % P) * D + c;
          kk = *reinterpret_cast<const float4*>(e);
          vv = *reinterpret_cast<const float4*>(e + (size_t)P * D);
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
          // (the product takes the scale: scale * q may be past the largest float where scale * q.K is not)
          x[i][j] = k0 + tx + 16 * j < seen[i] ? x[i][j] * A.scale_l2e : -INFINITY;
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
          *reinterpret_cast<float4*>(static_cast<float*>(A.out) + e + 4 * tx + 64 * j) = y;
        }
        if (A.lse && tx == 0) A.lse[e / D] = (m[i] + log2f(l[i])) * LN2;
      } else {
        const size_t pr = ((size_t)blockIdx.x * 2 + part) * CF_ROWS + r;
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

template <int D>
__global__ void __launch_bounds__(CJ_WARPS * 32) k_chunk_join(const __grid_constant__ ChunkArgs A) {
  pdl_wait();
  pdl_trigger();
  const int4 jt = __ldcg(A.joint + blockIdx.x);
  const int r = blockIdx.y * CJ_WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int parts = jt.w >> 16;
  if (r >= (jt.w & 0xFFFF)) return;
  // part 0 of the join is this block's part 1, then part 0 of the blocks after it
  auto at = [&](int c) { return ((size_t)(blockIdx.x + c) * 2 + (c == 0 ? 1 : 0)) * CF_ROWS + r; };
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
  const size_t row = row_at(A, jt.x, jt.y, jt.z, r);
  float* og = static_cast<float*>(A.out) + row * D + NV * lane;
  const float inv = 1.f / l;
  if (A.lse && lane == 0) A.lse[row] = (M + log2f(l)) * LN2;
#pragma unroll
  for (int i = 0; i < NV; ++i) og[i] = o[i] * inv;
}

// ---------------------------------------------------------------------------
// Tensor-core form (bf16 cache). One block per SM, eleven warps: a TMA producer of
// keys and values, an MMA issuer, a loader (segments and their queries) and two
// softmax groups of four warps. A tile has two groups of up to 128 rows (whole
// tokens), which share each tile of 128 keys. S = Q K^T (128 x 128) of a group goes to
// its half of tensor memory; a softmax thread owns a row (a TMEM lane), reads its
// scores 32 at a time and writes the weights over them as bf16; O += P V takes them
// from there, V as an MN-major operand. In issue order
//   P V of group 0, tile i - 1; S of group 0, tile i; the same of group 1; ..
// so that one group's exponentials run beside the other's MMAs. MMAs of one thread
// execute in the order of their issue: S may go over the weights that the P V before
// it reads, and a barrier that S completes tells that this P V is over too.
//
// A weight is 2^(x - m) with a whole number m, set 24 above the first scores' maximum:
// weights are floats, whose precision another m leaves as it is, so no maximum is
// looked for afterwards. A tile whose weights sum past 2^9 (a score grew by some 30
// binary orders), or to no number, is done again by ch_slow, which moves m and rescales
// O and the tile's earlier weights. Scores beyond 2^24, above which float
// does not hold every whole number, are taken against the row's largest score itself,
// also there. Rounding a weight to bf16 costs at most 2^-8 relative in each term, as
// rounding the result does: 0.0023 in all against 64 bits, 0.0017 with the result's
// alone; a second bf16 part would be half of the MMAs again. The sum of weights is of
// the fp32 values.
//
// Bound by the MMAs and what feeds them: an iteration's two S and two P V are 2,048 cycles
// of tensor cores, and as many of the shared memory's port (an S MMA reads 8 KB in its
// 64 cycles, all that the port gives, and 64 KB of keys and values come in beside it);
// with the issuer's waits it takes 2,600. (168 registers a thread and 16 bytes of
// spills; with 72 the chunks took 142 us for 139.) Without the exponentials the kernel takes as long,
// without any of the softmax's arithmetic 7% less. Measured, L2 cold, 32 on 8 heads of 128: a
// chunk of 1,021 tokens behind 65,521 720 us (0.78 of the MMA rate; 780 to 810 where the
// clocks have come down to the power cap's), a prompt of 5,288 174 us (0.67), eight chunks
// of 17 to 701 behind 1,288 to 5,288 139 us (0.64): a segment's switch is 10,000 cycles from its
// last S to the next one's first weights (last weights and P V 3,000, results 3,500, the
// next queries and S). Slower: an issuer for each group (951 us where one had 798), sixteen
// softmax warps, scores summed one by one, the sum of the rounded weights; barriers for
// each buffer in place of each iteration's (750 where this has 735); each lane its own
// row's results (prompt 189, chunks 142); the next segment's S before the results are out
// (chunks 150). No faster: scores asked for two loads ahead, the next queries into L2.
constexpr int CT_KEYS = 128;                     // 2^7 (key_bits)
constexpr int CT_THREADS = 352;
constexpr int CT_RING = 16;                      // iterations whose barriers are told apart
constexpr int CT_EXTRA = 2;                      // units' time that a segment's start and end take
constexpr int CT_HALF = 128 * 128;               // bytes of 64 dims of 128 rows of Q
constexpr int CT_OCOL = 256;                     // TMEM columns: S of a group at 128 g, its O behind at CT_OCOL + D g
constexpr float CT_AHEAD = 24.f;                 // m is set to a score + 24
constexpr float CT_MUCH = 512.f;                 // a tile's weights sum to less while m stays
constexpr float CT_GROW = 8.f;                   // and m moves where a score passes m - 24 + 32
constexpr float CT_FAR = 16777216.f;             // scores up to here go by m alone

template <int D>
struct CtCfg {
  static constexpr int BUF = CT_KEYS * D * 2;    // K or V of a tile
  static constexpr int Q = 128 * D * 2;          // a group's queries
  static constexpr int TAIL = 2048;              // alignment slack and the header
  static constexpr int NBUF = (232448 - 512 - TAIL - 2 * Q) / BUF < 8 ? (232448 - 512 - TAIL - 2 * Q) / BUF : 8;
  static constexpr int SMEM = NBUF * BUF + 2 * Q + TAIL;
};

struct CtHeader {
  uint64_t full[CT_RING], done[CT_RING], s_full[2], p_full[2], o_done[2], seg_full[2], seg_free[2];
  uint64_t q_full, q_free, fin;
  uint32_t tmem;
  int abort;
  ChunkSeg seg[2];                               // nt = 0: no more
};

// Rows of group g of a segment, and the key tiles from t0 on that one of them sees.
struct CtGroup {
  int row0, rows, tiles, end;                    // first row in the tile, rows, tiles, positions that the last row sees
  __device__ CtGroup(const ChunkArgs& A, const ChunkSeg& s, int g) {
    const int half = A.tok / 2, tok0 = s.rt * A.tok + g * half, n = max(0, min(half, s.m - tok0));
    row0 = g * half * A.G;
    rows = n * A.G;
    end = n ? s.n + tok0 + n : 0;
    tiles = max(0, min(s.t1, (end + CT_KEYS - 1) / CT_KEYS) - s.t0);
  }
};

// A lane's row of a segment so far: weights are 2^(sc (S - s0) - m), l their sum. s0
// is 0, or the largest score (m = CT_AHEAD).
struct CtLane {
  float m, l, s0;
};
// Its scores of a tile.
struct CtTile {
  uint32_t s, o;               // tensor memory of S and O
  float sc;                    // scale * log2 e
  int seen;                    // keys of the tile that the row sees
  bool first, live;            // no O yet; a row
};

// (The volatile statement keeps it behind its branch: predicated, it is half of a tile's instructions.)
__device__ __forceinline__ void ct_mask(uint32_t (&v)[32], int seen) {
  asm volatile("" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (i >= seen) v[i] = 0xff800000u;
}

// Weights of one chunk of 32 scores, whatever they are. Out of line and rare.
template <int D>
__device__ __noinline__ CtLane ch_slow(CtTile T, int c, CtLane a) {
  uint32_t v[32];
  tmem_ld32(T.s + 32 * c, v);
  ct_mask(v, T.seen - 32 * c);
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < 32; i += 2) mx = max3(mx, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
  const float mt = (mx - a.s0) * T.sc;
  const bool far = a.s0 != 0.f, grow = T.live && (far ? mx > a.s0 : mt > a.m + CT_GROW);
  if (__any_sync(0xffffffffu, grow)) {
    float corr = 1.f;
    if (grow && (far || !(fabsf(mt) <= CT_FAR))) {   // (the score itself, so that equal ones differ by 0)
      corr = ex2(a.m - mt - CT_AHEAD);
      a.m = CT_AHEAD;
      a.s0 = mx;
    } else if (grow) {
      const float to = ceilf(mt) + CT_AHEAD, by = to - a.m;
      corr = by < 127.f ? __uint_as_float((127 - (int)by) << 23) : 0.f;    // 2^-by, exact
      a.m = to;
    }
    a.l *= corr;
    tmem_wait_st();                              // the chunks' weights are read back
    if (!T.first) {                              // (the tile's S came after the group's last P V)
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
    for (int i = 0; i < c; ++i) {
      uint32_t w[16];
      tmem_ld16(T.s + 16 * i, w);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        w[j] = pack_bf16(__uint_as_float(w[j] << 16) * corr, __uint_as_float(w[j] & 0xFFFF0000u) * corr);
      tmem_st16(T.s + 16 * i, w);
    }
  }
  const float mb = a.m == -INFINITY ? 0.f : a.m;
  float sum = 0.f;
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const float p0 = ex2(fmaf(__uint_as_float(v[i]) - a.s0, T.sc, -mb)), p1 = ex2(fmaf(__uint_as_float(v[i + 1]) - a.s0, T.sc, -mb));
    sum += p0 + p1;
    w[i / 2] = pack_bf16(p0, p1);
  }
  tmem_st16(T.s + 16 * c, w);                    // (over scores that are read already)
  a.l += sum;
  return a;
}

// Weights 2^(sc v - m) of 32 scores as bf16 pairs, w[AT] .. w[AT + 15], and their sums.
template <int AT>
__device__ __forceinline__ void ch_weights(const uint32_t (&v)[32], uint32_t (&w)[64], unsigned long long sc2,
                                           unsigned long long nm2, unsigned long long (&sum)[2]) {
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const float2 y = halves(fma2(pair(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), sc2, nm2));
    const float p0 = ex2(y.x), p1 = ex2(y.y);
    sum[i / 2 & 1] = add2(sum[i / 2 & 1], pair(p0, p1));
    w[AT + i / 2] = pack_bf16(p0, p1);
  }
}

template <int D>
__global__ void __launch_bounds__(CT_THREADS, 1)
    k_chunk_tc(const __grid_constant__ CUtensorMap kvmap, const __grid_constant__ CUtensorMap qmap,
               const __grid_constant__ ChunkArgs A, int kb) {
  using C = CtCfg<D>;
  constexpr int HALVES = D / 64, NBUF = C::NBUF;
  // a K or V tile lies as [8 keys][64-dim half][key][64 dims], as a box of whole pages brings it
  constexpr int GROUP = 1024 * HALVES;
  extern __shared__ unsigned char ct_raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(ct_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* qsm = base + NBUF * C::BUF;
  CtHeader& H = *reinterpret_cast<CtHeader*>(qsm + 2 * C::Q);
  static_assert(sizeof(CtHeader) + 1024 <= C::TAIL, "header and alignment slack");
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const uint32_t bufs = sm_addr(base), q_addr = sm_addr(qsm);
  if (t == 0) {
    for (int i = 0; i < CT_RING; ++i) {
      mbar_init(H.full + i, 1);
      mbar_init(H.done + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(H.s_full + i, 1);
      mbar_init(H.p_full + i, 4);
      mbar_init(H.o_done + i, 1);
      mbar_init(H.seg_full + i, 1);
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
    for (int s = t; s < A.ix.n_seq; s += CT_THREADS)
      if (ChunkSeq(A.ix, s).bad) atomicOr(A.err, DERR_POS);
  ChunkWalk walk;
  tc_fence_before();
  walk.init<CT_THREADS>(A);                      // (a block barrier at least)
  tc_fence_after();
  const uint32_t tmem = H.tmem;
  // A wait that runs out raises the block's abort flag, which ends its other waits
  // at once: every role leaves its loops, a softmax warp in the middle of a segment too, which
  // may have millions of tiles left. The segment has no result.
  auto wait = [&](const uint64_t* bar, uint32_t parity) {
    return mbar_try(sm_addr(bar), parity & 1) || wait_long(sm_addr(bar), parity & 1, &H.abort, A.err, A.deadlines());
  };
  auto waitw = [&](const uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
  const int P = A.kv.page_size;

  if (warp == 8) {
    // ---- producer: for each of the issuer's iterations V of a tile and K of the next, a box for each kb keys
    // of a page. An iteration has one barrier that says its loads are there and one that says it is over, and
    // with it the buffers that it read: a buffer's load waits for the iteration of the one before (lane b
    // knows buffer b's). Every iteration has a load, so none is passed over, and CT_RING of them are more than
    // there are buffers. ----
    static_assert(NBUF < CT_RING, "iterations on their way");
    const int nbox = CT_KEYS / kb, j = lane;
    const int planes = A.kv.n_layers * A.kv.n_kv_heads * 2;
    int b = 0;
    uint32_t it = 0, last = 0, loads = 0;
    bool ok = true;
    ChunkSeg g;
    while (ok && walk.next(g)) {
      const int32_t* bt = A.kv.block_table_dev + (size_t)g.s * A.kv.max_pages;
      const int plane = (A.layer * A.kv.n_kv_heads + g.hk) * 2;
      auto page_of = [&](int tile) {             // of this lane's box; -1 reads zeros
        const int key = tile * CT_KEYS + kb * j;
        int page = -1;
        if (lane < nbox && tile < g.t1 && key < g.n + g.m) {
          page = bt[key / P];
          if (page < 0 || page >= A.kv.n_pages) {
            page = -1;
            atomicOr(A.err, DERR_PAGE);
          }
        }
        return page;
      };
      int page = -1, next = page_of(g.t0);
      for (int i = 0, n = g.t1 - g.t0; ok && i <= n; ++i, ++it) {
        const uint32_t full = sm_addr(H.full + it % CT_RING);
        if (lane == 0)
          asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;"
                       ::"r"(full), "r"((uint32_t)((i > 0 && i < n ? 2 : 1) * C::BUF)) : "memory");
        __syncwarp();
#pragma unroll
        for (int v = 1; v >= 0; --v) {           // V of tile i - 1, K of tile i
          if (v ? i == 0 : i == n) continue;
          const int tile = g.t0 + i - v, key = tile * CT_KEYS + kb * j;
          if (!v) {
            page = next;
            next = page_of(tile + 1);
          }
          const uint32_t before = __shfl_sync(0xffffffffu, last, b);
          if (ok && loads >= NBUF) ok = waitw(H.done + before % CT_RING, before / CT_RING);
          if (!ok) break;
          if (lane < nbox)
            asm volatile(
                "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3, %4}], [%5];"
                ::"r"(bufs + b * C::BUF + j * kb * D * 2), "l"(reinterpret_cast<uint64_t>(&kvmap)), "r"(0), "r"(key % P / 8),
                  "r"(page < 0 ? -1 : page * planes + plane + v), "r"(full)
                : "memory");
          if (lane == b) last = it;
          ++loads;
          if (++b == NBUF) b = 0;
        }
      }
    }
    // shared memory outlives the copies (over, unless a wait was given up): those of the last iterations
    for (uint32_t k = it > CT_RING ? it - CT_RING : 0; k < it; ++k)
      mbar_wait_deadline(sm_addr(H.full + k % CT_RING), k / CT_RING & 1, nullptr);
  } else if (warp == 9) {
    // ---- MMA issuer. The whole warp runs the loop on values that are the same in
    // every lane, so that the descriptors stay in uniform registers; one lane issues.
    // instruction descriptors: bf16 x bf16 -> f32, M = 128; V is MN-major
    const uint32_t id_s = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(CT_KEYS >> 3) << 17) | (8u << 24);
    const uint32_t id_o = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | (8u << 24);
    const uint32_t one = elect_one(), tm = __shfl_sync(0xffffffffu, tmem, 0);
    auto same = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    uint32_t jobs[2] = {0, 0};                   // P V's of the groups so far
    int rbuf = 0;                                // ring position of the next load
    uint32_t it = 0;                             // iterations so far
    auto step = [&]() {
      const int b = rbuf;
      if (++rbuf == NBUF) rbuf = 0;
      return b;
    };
    bool ok = true;
    for (uint32_t seg = 0; ok; ++seg) {
      const int sb = seg & 1;
      if (!(ok = waitw(H.seg_full + sb, seg >> 1))) break;
      ChunkSeg g = H.seg[sb];
      g.nt = same(g.nt); g.t0 = same(g.t0); g.t1 = same(g.t1); g.n = same(g.n); g.m = same(g.m); g.rt = same(g.rt);
      if (g.nt == 0) break;
      const CtGroup G0(A, g, 0), G1(A, g, 1);
      const int nt = g.t1 - g.t0, n0 = same(G0.tiles), n1 = same(G1.tiles), e0 = same(G0.end), e1 = same(G1.end);
      if (!(ok = waitw(&H.q_full, seg))) break;
      // iteration i: P V of tile i - 1 (its V is the ring's next), S of tile i (its K behind)
      for (int i = 0; ok && i <= nt; ++i, ++it) {
        if (!(ok = waitw(H.full + it % CT_RING, it / CT_RING))) break;
        const int vbuf = i > 0 ? step() : 0, kbuf = i < nt ? step() : 0;
        if (i > 0) {
          // slots past the sequence's last may hold anything: those that the last MMA reads become zeros
          const int nk = g.n + g.m - (g.t0 + i - 1) * CT_KEYS;
          if (nk < CT_KEYS && nk % 16) {
            unsigned char* vb = base + vbuf * C::BUF;
            const int rows = 16 - nk % 16;
            for (int x = lane; x < rows * HALVES * 8; x += 32) {
              const int key = nk + x / (HALVES * 8), hf = x / 8 % HALVES;
              *reinterpret_cast<uint4*>(vb + key / 8 * GROUP + hf * 1024 + key % 8 * 128 + (x % 8) * 16) = make_uint4(0, 0, 0, 0);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
          }
        }
#pragma unroll
        for (int gr = 0; gr < 2; ++gr) {
          const int ng = gr ? n1 : n0, end = gr ? e1 : e0;
          if (ok && i > 0 && i <= ng) {
            if (!(ok = waitw(H.p_full + gr, jobs[gr]++))) break;
            tc_fence_after();
            const uint32_t d = tm + CT_OCOL + gr * D, a = tm + gr * 128;
            const uint64_t bd = tt_desc(bufs + vbuf * C::BUF, 1024, GROUP);
            const int steps = (min(CT_KEYS, end - (g.t0 + i - 1) * CT_KEYS) + 15) / 16;
            // 16 keys a step: their weights lie in columns 8 k ..
            auto part = [&](int k, bool acc) { mma_ts(d, a + 8 * k, bd + (uint64_t)(k * 2 * GROUP >> 4), id_o, acc, one); };
            part(0, i > 1);
            if (steps == CT_KEYS / 16) {
#pragma unroll
              for (int k = 1; k < CT_KEYS / 16; ++k) part(k, true);
            } else {
#pragma unroll 1
              for (int k = 1; k < steps; ++k) part(k, true);
            }
            if (i == ng) tc_commit(sm_addr(H.o_done + gr), one);
          }
          if (ok && i < ng) {
            const uint64_t ad = tt_desc(q_addr + gr * C::Q, 16, 1024), bd = tt_desc(bufs + kbuf * C::BUF, 16, GROUP);
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_ss(tm + gr * 128, ad + (uint64_t)(((k & 3) * 32 + (k >> 2) * CT_HALF) >> 4),
                     bd + (uint64_t)(((k & 3) * 32 + (k >> 2) * 1024) >> 4), id_s, k > 0, one);
            tc_commit(sm_addr(H.s_full + gr), one);
          }
        }
        if (!ok) break;
        tc_commit(sm_addr(H.done + it % CT_RING), one);
        if (i == nt - 1) tc_commit(sm_addr(&H.q_free), one);
      }
    }
    // everything issued is done before TMEM is freed (also after an abort)
    tc_commit(sm_addr(&H.fin), one);
    mbar_wait_deadline(sm_addr(&H.fin), 0, nullptr);
  } else if (warp == 10) {
    // ---- loader: the segments and their queries ----
    ChunkSeg g;
    const int tpg = A.tok / 2;                   // tokens of a group
    uint32_t asked = 0;                          // segments whose queries were asked for
    for (uint32_t seg = 0;; ++seg) {
      const int sb = seg & 1;
      const bool have = walk.next(g);
      if (seg >= 2 && !waitw(H.seg_free + sb, (seg >> 1) - 1)) break;
      if (!have) g.nt = 0;
      if (lane == 0) {
        H.seg[sb] = g;
        mbar_arrive(sm_addr(H.seg_full + sb));
        if (have && part_of(g) == 1) A.joint[blockIdx.x] = joint_of(walk, g, min(A.tok, g.m - g.rt * A.tok) * A.G);
      }
      if (!have) break;
      if (seg > 0 && !waitw(&H.q_free, seg - 1)) break;
      const int groups = CtGroup(A, g, 1).rows > 0 ? 2 : 1, copies = groups * HALVES;
      if (lane == 0)
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;"
                     ::"r"(sm_addr(&H.q_full)), "r"((uint32_t)(copies * tpg * A.G * 128)) : "memory");
      __syncwarp();
      ++asked;
      if (lane < copies) {
        const int half = lane % HALVES, gr = lane / HALVES;
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
            ::"r"(q_addr + gr * C::Q + half * CT_HALF), "l"(reinterpret_cast<uint64_t>(&qmap)), "r"(0), "r"(half),
              "r"(g.hk * A.G), "r"(g.r0 + (g.rt * 2 + gr) * tpg), "r"(sm_addr(&H.q_full))
            : "memory");
      }
    }
    if (asked > 0) mbar_wait_deadline(sm_addr(&H.q_full), (asked - 1) & 1, nullptr);   // (over, unless aborted)
  } else {
    // ---- softmax groups; their warps go on apart ----
    const int gr = warp >> 2, r = t & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t sT = tmem + lanes + gr * 128, oT = tmem + lanes + CT_OCOL + gr * D;
    const float sc = A.scale_l2e;
    const unsigned long long sc2 = pair(sc, sc);
    uint32_t jobs = 0, ends = 0;                 // tiles; segments with tiles
    for (uint32_t seg = 0;; ++seg) {
      const int sb = seg & 1;
      if (!waitw(H.seg_full + sb, seg >> 1)) break;
      const ChunkSeg g = H.seg[sb];
      if (g.nt == 0) break;
      const CtGroup R(A, g, gr);
      const bool live = r < R.rows, any_live = __any_sync(0xffffffffu, live);
      CtLane st{-INFINITY, 0.f, 0.f};
      bool far = false;                          // a lane of the warp goes by its largest score
      // keys that the lane sees, from the segment's first on; the warp's fewest
      int seen = live ? g.n + g.rt * A.tok + (R.row0 + r) / A.G + 1 - g.t0 * CT_KEYS : 0;
      const int least = __reduce_min_sync(0xffffffffu, live ? seen : 0x7fffffff);
      bool ok = true;
      for (int ti = 0; ti < R.tiles; ++ti, seen -= CT_KEYS) {
        if (!(ok = waitw(H.s_full + gr, jobs++))) break;
        tc_fence_after();
        if (any_live) {
          const CtTile T{sT, oT, sc, seen, ti == 0, live};
          const bool cut = least - ti * CT_KEYS < CT_KEYS;
          bool again = far;
          if (ti == 0) {                         // m: from the first keys
            uint32_t v[32];
            tmem_ld32(sT, v);
            if (cut) ct_mask(v, seen);
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < 32; i += 2) mx = max3(mx, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
            mx *= sc;
            if (fabsf(mx) <= CT_FAR) st.m = ceilf(mx) + CT_AHEAD;
            again = __any_sync(0xffffffffu, live && seen > 0 && !(fabsf(mx) <= CT_FAR));
          }
          if (!again) {
            // scores on their way beside the exponentials; nothing is written before all of them are known to do
            const float mb = st.m == -INFINITY ? 0.f : st.m;
            const unsigned long long nm2 = pair(-mb, -mb);
            uint32_t va[32], vb[32], w[64];
            unsigned long long sum[2] = {0, 0};
            tmem_ld32_start(sT, va);
            tmem_ld32_done(va);
            tmem_ld32_start(sT + 32, vb);
            if (cut) ct_mask(va, seen);
            ch_weights<0>(va, w, sc2, nm2, sum);
            tmem_ld32_done(vb);
            tmem_ld32_start(sT + 64, va);
            if (cut) ct_mask(vb, seen - 32);
            ch_weights<16>(vb, w, sc2, nm2, sum);
            tmem_ld32_done(va);
            tmem_ld32_start(sT + 96, vb);
            if (cut) ct_mask(va, seen - 64);
            ch_weights<32>(va, w, sc2, nm2, sum);
            tmem_ld32_done(vb);
            if (cut) ct_mask(vb, seen - 96);
            ch_weights<48>(vb, w, sc2, nm2, sum);
            const float2 s2 = halves(add2(sum[0], sum[1]));
            const float s1 = s2.x + s2.y;
            again = __any_sync(0xffffffffu, live && !(s1 <= CT_MUCH));
            if (!again) {
              tmem_st32_from<0>(sT, w);
              tmem_st32_from<32>(sT + 32, w);
              st.l += s1;
            }
          }
          if (again) {
#pragma unroll 1
            for (int c = 0; c < CT_KEYS / 32; ++c) st = ch_slow<D>(T, c, st);
            far = __any_sync(0xffffffffu, st.s0 != 0.f);
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sm_addr(H.p_full + gr));
      }
      if (!ok) break;                            // (aborted: no result)

      // ---- the segment's end ----
      const int part = part_of(g);
      const float ref = fminf(fmaxf(fmaf(st.s0, sc, st.m), -3e38f), 3e38f);   // (finite, whatever the scores)
      const bool some = st.m != -INFINITY;
      const size_t pr = (((size_t)blockIdx.x * 2 + part) * 2 + gr) * 128 + r;       // (part >= 0)
      if (part >= 0 && live) A.part_ml[pr] = make_float2(some ? ref : -INFINITY, some ? st.l : 0.f);
      if (R.tiles > 0) {
        if (!waitw(H.o_done + gr, ends++)) break;
        tc_fence_after();
        if (any_live) {
          const size_t row = row_at(A, g.r0, g.rt, g.hk, R.row0 + r);
          const float inv = 1.f / st.l;
          if (part < 0 && live && A.lse) A.lse[row] = (ref + log2f(st.l)) * LN2;
          // Results go out by four lanes together, 64 bytes of a row: lane q of them has the q-th 16 bytes of the four rows.
          const int q = lane & 3;
          uint4* og[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int rj = (r & ~3) + j;
            og[j] = part < 0 && rj < R.rows
                        ? reinterpret_cast<uint4*>(static_cast<uint16_t*>(A.out) + row_at(A, g.r0, g.rt, g.hk, R.row0 + rj) * D) + q
                        : nullptr;
          }
          // a part lies as [4 dims][row]
          float4* pg = reinterpret_cast<float4*>(A.part_o) + (((size_t)blockIdx.x * 2 + part) * 2 + gr) * 128 * (D / 4) + r;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t v[32];
            tmem_ld32(oT + 32 * c, v);
            if (part < 0) {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * inv);
              uint32_t y[4][4];
#pragma unroll
              for (int i = 0; i < 16; ++i) y[i / 4][i % 4] = pack_bf16(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
              // a transposition: by the lanes' first bit, then by their second
#pragma unroll
              for (int s = 1; s < 4; s <<= 1)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  if (i & s) continue;
#pragma unroll
                  for (int x = 0; x < 4; ++x) {
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, q & s ? y[i][x] : y[i + s][x], s);
                    if (q & s) y[i][x] = got;
                    else y[i + s][x] = got;
                  }
                }
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (og[j]) og[j][4 * c] = make_uint4(y[j][0], y[j][1], y[j][2], y[j][3]);
            } else if (live) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                pg[(8 * c + i) * 128] = make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                                    __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]));
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sm_addr(H.seg_free + sb));
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

// Joins the parts of a shared segment, as k_chunk_join does; the parts lie as [4 dims]
// [row of a group], so a warp takes 32 rows and 4 dims of each at a time, and rows go
// out through shared memory. grid (blocks, groups of 32 rows).
constexpr int CX_WARPS = 8;

template <int D>
__global__ void __launch_bounds__(CX_WARPS * 32) k_chunk_tc_join(const __grid_constant__ ChunkArgs A) {
  __shared__ __align__(16) uint2 y[32][D / 4 + 1];
  pdl_wait();
  pdl_trigger();
  const int4 jt = __ldcg(A.joint + blockIdx.x);
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = blockIdx.y / 4, r = blockIdx.y % 4 * 32 + lane;
  const int parts = jt.w >> 16, rpg = A.rows / 2, rows = min(rpg, (jt.w & 0xFFFF) - gr * rpg);   // of the group
  if (parts == 0 || (int)(blockIdx.y % 4) * 32 >= rows) return;
  const bool live = r < rows;
  // part 0 of the join is this block's part 1, then part 0 of the blocks after it
  auto at = [&](int c) { return ((size_t)(blockIdx.x + c) * 2 + (c == 0 ? 1 : 0)) * 2 + gr; };
  constexpr int PER = D / 4 / CX_WARPS, FLY = 2;  // pieces of 4 dims a warp; parts on their way at once
  float4 v[FLY][PER];
  float2 ml[FLY];
  auto fetch = [&](int c0) {
#pragma unroll
    for (int f = 0; f < FLY; ++f) {
      const bool on = live && c0 + f < parts;
      ml[f] = on ? __ldcg(A.part_ml + at(c0 + f) * 128 + r) : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (on) v[f][i] = __ldcg(reinterpret_cast<const float4*>(A.part_o) + at(c0 + f) * 128 * (D / 4) + (w * PER + i) * 128 + r);
    }
  };
  float M = -INFINITY, L = 0.f;
  float4 o[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c0 = 0; c0 < parts; c0 += FLY) {
    fetch(c0);
#pragma unroll
    for (int f = 0; f < FLY; ++f) {
      if (!(ml[f].y > 0.f)) continue;            // (a part that saw nothing of the row may hold anything)
      const float mn = fmaxf(M, ml[f].x), a = exp2f(M - mn), b = exp2f(ml[f].x - mn);
      M = mn;
      L = L * a + ml[f].y * b;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        o[i].x = fmaf(v[f][i].x, b, o[i].x * a);
        o[i].y = fmaf(v[f][i].y, b, o[i].y * a);
        o[i].z = fmaf(v[f][i].z, b, o[i].z * a);
        o[i].w = fmaf(v[f][i].w, b, o[i].w * a);
      }
    }
  }
  const float inv = 1.f / L;
  if (A.lse && w == 0 && live) A.lse[row_at(A, jt.x, jt.y, jt.z, gr * rpg + r)] = (M + log2f(L)) * LN2;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    o[i].x *= inv;
    o[i].y *= inv;
    o[i].z *= inv;
    o[i].w *= inv;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) y[lane][w * PER + i] = make_uint2(pack_bf16(o[i].x, o[i].y), pack_bf16(o[i].z, o[i].w));
  __syncthreads();
  for (int x = threadIdx.x; x < 32 * (D / 4); x += CX_WARPS * 32) {
    const int row = x / (D / 4), c = x % (D / 4), q = blockIdx.y % 4 * 32 + row;
    if (q >= rows) continue;
    reinterpret_cast<uint2*>(static_cast<uint16_t*>(A.out) + row_at(A, jt.x, jt.y, jt.z, gr * rpg + q) * D)[c] = y[row][c];
  }
}

// Shape of a launch, from sizes and types alone. A batch of few bf16 tokens goes by the tree
// attention's kernel, whose weights have 16 bits: tokens decoded without a prompt in the batch
// meet the arithmetic of those verified in a tree, 0.0017 off a 64-bit result for 0.0023. (With a
// prompt among them all go by the form here.) Its time and that of
// the tensor-core form here, one token each: one sequence of 5,236 on 10 heads 21.7 and
// 24.0 us, 64 of 336 to 5,236 168 and 162, 16 of them 62 and 55; one of 65,521 on 8 heads
// 59 and 64; 32 tokens on that 67 and 66, eight of 1,288 to 5,288 43 and 38. (With 256 rows
// in place of 128, 64 tokens of the eight take 63 and 43.)
struct ChunkPlan {
  int G, parts, tok, key_bits, extra;
  int max_blocks;           // of any grid (the workspace is sized without a device)
  size_t ml, joint, total;  // workspace: outputs at 0, statistics, joints
  bool chain;               // few tokens: the tree attention's kernel, each node the next one's parent
  ChunkPlan(const spec_kv_view& kv, int max_new, int hq) {
    chain = kv.dtype == SPEC_BF16 && max_new <= SPEC_TREE_MAX_NODES && max_new * (hq / kv.n_kv_heads) <= 128;
    if (chain) {
      total = chain_ws_bytes(kv, max_new, hq);
      return;
    }
    const bool tc = kv.dtype == SPEC_BF16;
    const int heads = hq / kv.n_kv_heads;
    parts = 1;
    while (!tc && (heads % parts || heads / parts > CF_ROWS)) ++parts;
    G = heads / parts;
    tok = tc ? 2 * (128 / G) : CF_ROWS / G;
    key_bits = tc ? 7 : 6;
    extra = tc ? CT_EXTRA : 0;
    max_blocks = tc ? 160 : 320;                 // one block per SM, or two
    const int lie = tc ? 256 : CF_ROWS;          // rows of a part
    ml = (size_t)max_blocks * 2 * lie * kv.head_dim * sizeof(float);
    joint = (ml + (size_t)max_blocks * 2 * lie * sizeof(float2) + 15) / 16 * 16;
    total = joint + (size_t)max_blocks * sizeof(int4);
  }
};

int check_attention(const spec_kv_view* kv, int n_seq, int max_new, int hq) {
  const int rc = check_chunks(kv, n_seq, hq);
  if (rc) return rc;
  if (max_new < 1) return set_last_error(SPEC_ERR_ARG, "max_new >= 1 required");
  if (hq / kv->n_kv_heads > CH_MAX_G) return set_last_error(SPEC_ERR_UNSUPPORTED, "more than 128 query heads per kv head");
  // a row tile's units, and a sequence's rows of a kv head, are counted in 32 bits
  if ((double)kv->max_pages * kv->page_size / CF_KEYS * hq > 2e9 ||
      (double)std::min<int64_t>(max_new, (int64_t)kv->max_pages * kv->page_size) * (hq / kv->n_kv_heads) > 2e9)
    return set_last_error(SPEC_ERR_UNSUPPORTED, "block table too long for this many heads");
  return SPEC_OK;
}

template <int D>
cudaError_t launch_tc(const ChunkArgs& A, const CUtensorMap& map, const CUtensorMap& qmap, int kb, int blocks, cudaStream_t st) {
  cudaError_t e = allow_dyn_smem_once<k_chunk_tc<D>>();
  if (e == cudaSuccess) e = launch_k(k_chunk_tc<D>, dim3(blocks), dim3(CT_THREADS), CtCfg<D>::SMEM, st, map, qmap, A, kb);
  return e == cudaSuccess ? launch_k(k_chunk_tc_join<D>, dim3(blocks, 8), dim3(CX_WARPS * 32), 0, st, A) : e;
}

template <int D>
cudaError_t launch_fma(const ChunkArgs& A, int blocks, cudaStream_t st) {
  cudaError_t e = allow_dyn_smem_once<k_chunk_fma<D>>();
  if (e == cudaSuccess) e = launch_k(k_chunk_fma<D>, dim3(blocks), dim3(CF_THREADS), sizeof(CfSmem<D>), st, A);
  if (e != cudaSuccess) return e;
  return launch_k(k_chunk_join<D>, dim3(blocks, CF_ROWS / CJ_WARPS), dim3(CJ_WARPS * 32), 0, st, A);
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
  const int64_t lse_bytes = (int64_t)n_rows * n_q_heads * 4;
  if (spans_meet(out_lse_dev, lse_bytes, q_dev, bytes) || spans_meet(out_lse_dev, lse_bytes, out_dev, bytes))
    return set_last_error(SPEC_ERR_ARG, "lse overlaps q or out");
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
                    reinterpret_cast<int4*>(w + plan.joint), layer, n_q_heads, plan.G, plan.parts, kv->n_kv_heads * plan.parts,
                    plan.tok, plan.tok * plan.G, plan.key_bits, plan.extra, scale * LOG2E};
  cudaError_t e;
  if (kv->dtype == SPEC_F32) {
    const int blocks = std::min(2 * sms, plan.max_blocks);
    e = d == 128 ? launch_fma<128>(A, blocks, st) : launch_fma<64>(A, blocks, st);
  } else {
    const int kb = key_box(kv->page_size, CT_KEYS);
    CUtensorMap map, qmap;
    if (q_make_map(&qmap, q_dev, d, n_q_heads, (uint64_t)n_rows, A.G, plan.tok / 2) ||
        kv_make_group_map(&map, kv->kv_dev, d, kv->page_size, (uint64_t)kv->n_pages * kv->n_layers * kv->n_kv_heads * 2, kb))
      return set_last_error(SPEC_ERR_UNSUPPORTED, "tensor map encoding failed");
    const int blocks = std::min(sms, plan.max_blocks);
    e = d == 128 ? launch_tc<128>(A, map, qmap, kb, blocks, st) : launch_tc<64>(A, map, qmap, kb, blocks, st);
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? SPEC_OK : set_last_error(SPEC_ERR_CUDA, cudaGetErrorString(e));
}
