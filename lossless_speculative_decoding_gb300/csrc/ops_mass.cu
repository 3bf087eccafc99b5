// Kernel-level entry point: the attention weight that each cached position draws
// from a chunk of new tokens.
//
// With lse the log of a row's sum of exponentials, a position's share of the row is
// exp(scale q.K_j - lse): no second pass over the row is needed, and the sum over
// rows stays with the position. A unit is (sequence, tile of keys, kv head): it
// brings its keys once, goes over the counted rows that see them, and writes its
// positions alone, so nothing is summed by atomics. Units of a sequence are
// numbered from its first keys on, which the most rows see; of each B units worker b
// (a block, or a pair of blocks) takes the b-th, and of the next B the b-th from their
// end, so that the sums of what the workers do stay close.
#include <cuda_runtime.h>

#include <algorithm>

#include "chunk.cuh"
#include "tc_attn.cuh"

namespace spec {
namespace {

constexpr int MS_MAX_G = 128;                    // query heads per kv head
constexpr float LN2_LO = -1.9046543e-9f;         // log 2 = LN2 (as a float) + LN2_LO

struct MassArgs {
  spec_kv_view kv;
  ChunkIndex ix;
  const void* q;
  const float* lse;
  const float* mass;
  float* out;
  int32_t* err;
  long long ld;
  int layer, hq, G, last;
  int tok;             // tokens of a tile of rows (tensor-core form)
  int nk, nq, q_half;  // its rings: tiles of keys (two rings) and of queries in shared memory, bytes of 64 dims of a tile of queries
  int pair;            // blocks that share a unit's rows: 1 or 2
  float scale_l2e;     // scale * log2 e
  float inv_scale;
};

// Unit: key tile `tile` of (sequence s, kv head hk), its rows from token i0 on.
struct MassUnit {
  int s, tile, hk;
  int n, m, r0, i0;
};

// A warp's walk over the units of worker `me` of `workers`.
template <int KEYS>
struct MassWalk {
  long long round, before;                       // `workers` units each; units before sequence s
  int s, me, workers;
  const MassArgs* A;
  __device__ MassWalk(const MassArgs& args, int me, int workers) : round(0), before(0), s(0), me(me), workers(workers), A(&args) {}
  __device__ static int tiles(int n, int m) { return (n + m + KEYS - 1) / KEYS; }
  __device__ bool next(MassUnit& g) {
    const int lane = threadIdx.x & 31, hkv = A->kv.n_kv_heads;
    const long long u = round * workers + (round & 1 ? workers - 1 - me : me);
    for (;;) {                                   // sequences 32 at a time
      if (s >= A->ix.n_seq) return false;
      const bool on = s + lane < A->ix.n_seq;
      const ChunkSeq z(A->ix, on ? s + lane : s);
      const long long mine = on && z.m > 0 ? (long long)tiles(z.n, z.m) * hkv : 0;
      long long end = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, end, o);
        if (lane >= o) end += v;
      }
      end += before;
      const uint32_t past = __ballot_sync(0xffffffffu, end > u);
      if (past) {
        const int l = __ffs(past) - 1;
        before = __shfl_sync(0xffffffffu, end - mine, l);
        s += l;
        g.n = __shfl_sync(0xffffffffu, z.n, l);
        g.m = __shfl_sync(0xffffffffu, z.m, l);
        g.r0 = __shfl_sync(0xffffffffu, z.r0, l);
        break;
      }
      before = __shfl_sync(0xffffffffu, end, 31);
      s += 32;
    }
    const int in = (int)(u - before);
    g.s = s;
    g.tile = in / hkv;
    g.hk = in % hkv;
    g.i0 = max(g.m - min(A->last, g.m), g.tile * KEYS - g.n);   // (the counted ones; of them, those that see the first key)
    ++round;
    return true;
  }
};

// A sum with the rounding error that it has not taken in.
struct Comp {
  float s, e;
  __device__ __forceinline__ void add(float x) {
    const float t = s + x, b = t - s;
    e += (s - (t - b)) + (x - b);
    s = t;
  }
};

// ---------------------------------------------------------------------------
// FMA form. 128 threads, 64 keys, 32 rows at a time, fp32. Thread (ty, tx) = (t / 16,
// t % 16) has rows 4 ty .. 4 ty + 3 and keys tx + 16 j of the score product. Its four
// weights of a key are added, and the steps of 32 rows by a compensated sum: 65,536
// equal rows were 7.6e-5 off in a plain one.
constexpr int MF_THREADS = 128;
constexpr int MF_ROWS = 32;
constexpr int MF_KEYS = 64;

template <int D>
struct MfSmem {
  static constexpr int KST = D + 4;
  float q[MF_ROWS][D];
  float k[MF_KEYS][KST];
  float sum[8][MF_KEYS];
  float lse[MF_ROWS];
  int page[MF_KEYS];
};

template <int D>
__global__ void __launch_bounds__(MF_THREADS) k_mass_fma(const __grid_constant__ MassArgs A) {
  using L = MfSmem<D>;
  extern __shared__ __align__(16) unsigned char sm_raw[];
  L& sm = *reinterpret_cast<L*>(sm_raw);
  const int t = threadIdx.x, tx = t & 15, ty = t >> 4;
  const int P = A.kv.page_size;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0)
    for (int s = t; s < A.ix.n_seq; s += MF_THREADS)
      if (ChunkSeq(A.ix, s).bad) atomicOr(A.err, DERR_POS);
  const size_t page_elems = (size_t)A.kv.n_layers * A.kv.n_kv_heads * 2 * P * D;
  MassWalk<MF_KEYS> walk(A, blockIdx.x, gridDim.x);
  MassUnit g;
  while (walk.next(g)) {
    const int k0 = g.tile * MF_KEYS, nk = min(MF_KEYS, g.n + g.m - k0);
    const int32_t* bt = A.kv.block_table_dev + (size_t)g.s * A.kv.max_pages;
    const size_t plane = (((size_t)A.layer * A.kv.n_kv_heads + g.hk) * 2) * P * D;
    __syncthreads();                             // the last unit's reads are done
    if (t < MF_KEYS) {
      int page = -1;
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
    for (int i = t; i < MF_KEYS * (D / 4); i += MF_THREADS) {
      const int key = i / (D / 4), c = 4 * (i % (D / 4)), page = sm.page[key];
      float4 kk = make_float4(0.f, 0.f, 0.f, 0.f);
      if (page >= 0)
        kk = *reinterpret_cast<const float4*>(static_cast<const float*>(A.kv.kv_dev) + page * page_elems + plane +
                                              (size_t)((k0 + key) % P) * D + c);
      *reinterpret_cast<float4*>(&sm.k[key][c]) = kk;
    }
    Comp sum[4] = {};
    const int end = g.m * A.G;
    for (int r0 = max(g.i0, 0) * A.G; r0 < end; r0 += MF_ROWS) {
      __syncthreads();
      for (int i = t; i < MF_ROWS * (D / 4); i += MF_THREADS) {
        const int r = i / (D / 4), c = 4 * (i % (D / 4)), rr = r0 + r;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (rr < end) {
          const size_t row = ((size_t)g.r0 + rr / A.G) * A.hq + g.hk * A.G + rr % A.G;
          v = *reinterpret_cast<const float4*>(static_cast<const float*>(A.q) + row * D + c);
          if (c == 0) sm.lse[r] = A.lse[row] * LOG2E;
        }
        *reinterpret_cast<float4*>(&sm.q[r][c]) = v;
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
      float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rr = r0 + 4 * ty + i;
        if (rr >= end) continue;
        const float lse = sm.lse[4 * ty + i];
        const int seen = g.n + rr / A.G + 1 - k0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (tx + 16 * j < seen) part[j] += exp2f(fmaf(x[i][j], A.scale_l2e, -lse));   // (scale * q may overflow)
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j].add(part[j]);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) sm.sum[ty][tx + 16 * j] = sum[j].s + sum[j].e;
    __syncthreads();
    if (t < nk) {
      float y = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) y += sm.sum[i][t];
      const size_t e = ((size_t)g.s * A.kv.n_kv_heads + g.hk) * A.ld + k0 + t;
      if (A.mass && k0 + t < g.n) y += A.mass[e];
      A.out[e] = y;
    }
  }
}

// ---------------------------------------------------------------------------
// Tensor-core form (bf16 cache). One block per SM, twenty warps: a TMA producer, a
// loader of the rows' lse, four groups of four warps that sum and an MMA issuer for
// each tile of keys (an issue waits until the MMAs before it are nearly over, so that
// one issuer's waits leave the tensor cores idle: 113 us for 105). A unit has two tiles
// of 128 keys; against each tile of up to 128 rows (whole tokens), S = K Q^T goes to
// tensor memory with the keys on the lanes, so that a thread sums its key's columns in
// registers and no sum crosses threads. Groups 0 and 1 take the even tiles of rows, 2
// and 3 the odd ones, each group one tile of keys; each has a quarter of tensor memory,
// which it gives back as soon as its scores are in registers.
//
// One more MMA adds (c - lse) / scale to every column: as three bf16 parts (24 bits) in
// three more dims of a row, against ones in those of a key. c, a whole number of log 2,
// is near the unit's first lse, so that what the tensor cores add stays small: their
// sums are cut, not rounded. (Read from shared memory by every thread, lse took the
// bandwidth that the MMAs need: 218 us for 113.)
//
// Where units have many tiles of rows and are few, two blocks (a cluster) share a unit,
// each every other tile of rows, so that the few units of a single prompt's first keys
// do not outlast the others; the second block's sums go to the first one's shared memory.
//
// The loader walks over the units and hands them to the other roles, with their pages,
// through a small ring: twenty warps that each looked for themselves took a third of the
// issue slots where a unit has one row (129 us for 87).
//
// Measured, L2 cold. Every token of a prompt of 5,288, 32 on 8 heads: 104 us, 0.56 of
// the MMA rate for 115 GFLOP (the added MMA is an eighth more, tiles on the diagonal are
// whole, and beside the MMAs every score is read from tensor memory and takes its
// exponential: 48 us of the special function units). One token of each of 64
// sequences of 336 .. 5,236 positions, 10 heads: 87 us, 0.81 of the copy rate.
//
// Sums: 128 weights in fp32, the tiles of rows by a compensated sum (its rounding error
// is carried along), so that thousands of rows lose no bits.
constexpr int MT_KEYS = 128;
constexpr int MT_UNIT = 2 * MT_KEYS;
constexpr int MT_SUM = 16;                       // warps that sum
constexpr int MT_THREADS = 32 * (MT_SUM + 4);
constexpr int MT_MAX_NK = 8, MT_MAX_NQ = 4;
constexpr int MT_PAIR_TILES = 8;                 // blocks work in pairs from so many tiles of rows a unit on,
constexpr int MT_PAIR_PLANES = 16;               // on up to so many (sequence, kv head)
constexpr int MT_EXT = 128 * 16;                 // bytes of 8 more dims of 128 rows
constexpr int MT_RING = 4;                       // units handed over at once

template <int D>
struct MtCfg {
  static constexpr int BUF = MT_KEYS * D * 2;    // a tile of keys
  static constexpr int TAIL = 6144;              // alignment slack and the header
  static constexpr int EXT = MT_EXT * (MT_MAX_NQ + 2);       // of each tile of rows; of keys: ones; zeros
  static constexpr int ROOM = (232448 - 512 - TAIL - EXT) / 1024 * 1024;
  static constexpr int SMEM = ROOM + EXT + TAIL;
};

struct MtHeader {
  uint64_t k_full[MT_MAX_NK], k_empty[MT_MAX_NK], q_full[MT_MAX_NQ], q_empty[MT_MAX_NQ], s_full[4], s_empty[4];
  uint64_t sum_full[2][2], sum_empty[2][2], pair_full[2][2], pair_empty[2][2], fin[2];  // [owner][tile of keys]
  uint64_t unit_full[MT_RING], unit_empty[MT_RING];
  uint32_t tmem;
  int abort;
  MassUnit unit[MT_RING];                        // s < 0: no more
  float near[MT_RING];                           // mt_near of the unit's first lse
  int page[MT_RING][2][MT_KEYS / 16];            // of each box of keys; -1 reads zeros
  float sum[2][MT_UNIT], pair[2][MT_UNIT];       // sums of a unit: of the odd or even tiles, of the other block
};

// The whole number of log 2 near x.
__device__ __forceinline__ float mt_near(float x) { return rintf(x * LOG2E); }

template <int D>
__global__ void __launch_bounds__(MT_THREADS, 1)
    k_mass_tc(const __grid_constant__ CUtensorMap kvmap, const __grid_constant__ CUtensorMap qmap,
              const __grid_constant__ MassArgs A, int kb) {
  using C = MtCfg<D>;
  constexpr int HALVES = D / 64;
  // a tile of keys lies as [8 keys][64-dim half][key][64 dims], as a box of whole pages brings it
  constexpr int GROUP = 1024 * HALVES;
  extern __shared__ unsigned char mt_raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(mt_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* ext = base + C::ROOM;           // [tile of rows][row][8 dims], ones, zeros
  MtHeader& H = *reinterpret_cast<MtHeader*>(ext + C::EXT);
  static_assert(sizeof(MtHeader) + 1024 <= C::TAIL, "header and alignment slack");
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int NH = A.nk / 2, NQ = A.nq, q_bytes = HALVES * A.q_half;
  const uint32_t kbufs = sm_addr(base), qbufs = kbufs + A.nk * C::BUF;
  const int rank = A.pair > 1 ? (int)cluster_rank() : 0;
  if (t == 0) {
    for (int i = 0; i < MT_MAX_NK; ++i) {
      mbar_init(H.k_full + i, 1);
      mbar_init(H.k_empty + i, 1);
    }
    for (int i = 0; i < MT_MAX_NQ; ++i) {
      mbar_init(H.q_full + i, 2);                // queries, lse
      mbar_init(H.q_empty + i, 2);               // the issuers
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(H.s_full + i, 1);
      mbar_init(H.s_empty + i, 4);
      mbar_init(&H.sum_full[0][0] + i, 4);
      mbar_init(&H.sum_empty[0][0] + i, 4);
      mbar_init(&H.pair_full[0][0] + i, 4);
      mbar_init(&H.pair_empty[0][0] + i, 4);
    }
    for (int i = 0; i < MT_RING; ++i) {
      mbar_init(H.unit_full + i, 1);
      mbar_init(H.unit_empty + i, MT_SUM + 3);   // every other warp
    }
    mbar_init(H.fin, 1);
    mbar_init(H.fin + 1, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    H.abort = 0;
  }
  // ones in the first three dims behind a key's; zeros behind all
  for (int i = t; i < 2 * 128; i += MT_THREADS)
    *reinterpret_cast<uint4*>(ext + (MT_MAX_NQ * 128 + i) * 16) = i < 128 ? make_uint4(0x3f803f80u, 0x3f80u, 0u, 0u) : make_uint4(0u, 0u, 0u, 0u);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  if (warp == MT_SUM) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sm_addr(&H.tmem)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0)
    for (int s = t; s < A.ix.n_seq; s += MT_THREADS)
      if (ChunkSeq(A.ix, s).bad) atomicOr(A.err, DERR_POS);
  tc_fence_before();
  __syncthreads();
  if (A.pair > 1) cluster_sync();                // the other block's barriers are there
  tc_fence_after();
  const uint32_t tmem = H.tmem;
  // A wait that runs out raises the block's abort flag, which ends its other waits at
  // once: every role leaves its loops (the sums of a unit that is not over are not
  // written), and so does the other block of a pair when its own wait runs out. (One
  // deadline: no wait is for a whole unit.)
  auto waitw = [&](const uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_try(sm_addr(bar), parity & 1) || wait_long(sm_addr(bar), parity & 1, &H.abort, A.err, 1)) != 0;
  };
  // the same for a barrier that the other block arrives at
  auto waitw_pair = [&](const uint64_t* bar, uint32_t parity) {
    const bool ok = mbar_try_cluster(sm_addr(bar), parity & 1) ||
                    (wait_long(sm_addr(bar), parity & 1, &H.abort, A.err, 1) && mbar_try_cluster(sm_addr(bar), parity & 1));
    return __all_sync(0xffffffffu, ok) != 0;
  };
  const int P = A.kv.page_size;
  MassUnit g;
  // the next unit of the ring; what else is of it is read before `taken`
  uint32_t units = 0;
  auto take = [&]() {
    if (!waitw(H.unit_full + units % MT_RING, units / MT_RING)) return false;
    g = H.unit[units % MT_RING];
    return g.s >= 0;
  };
  auto taken = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(sm_addr(H.unit_empty + units % MT_RING));
    ++units;
  };
  const int first = rank * A.tok, stride = A.pair * A.tok;   // this block's tiles of rows

  if (warp == MT_SUM) {
    // ---- producer: a unit's keys (a box for each kb keys of a page), then its tiles of queries ----
    const int nbox = MT_KEYS / kb;
    const int planes = A.kv.n_layers * A.kv.n_kv_heads * 2;
    int kn[2] = {0, 0}, qn = 0;                  // ring positions
    uint32_t kturn[2] = {0, 0}, qturn = 0;       // passes over the rings
    bool ok = true;
    while (ok && take()) {
      const MassUnit n = g;
      int page[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) page[h] = lane < nbox ? H.page[units % MT_RING][h][lane] : -1;
      taken();
      const int plane = (A.layer * A.kv.n_kv_heads + n.hk) * 2;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k0 = n.tile * MT_UNIT + h * MT_KEYS, key = k0 + kb * lane;
        if (!ok || k0 >= n.n + n.m) break;
        const int kbuf = h * NH + kn[h];
        if (kturn[h] > 0 && !waitw(H.k_empty + kbuf, kturn[h] - 1)) { ok = false; break; }
        const uint32_t full = sm_addr(H.k_full + kbuf);
        if (lane == 0)
          asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full), "r"((uint32_t)C::BUF) : "memory");
        __syncwarp();
        if (lane < nbox)
          asm volatile(
              "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3, %4}], [%5];"
              ::"r"(kbufs + kbuf * C::BUF + lane * kb * D * 2), "l"(reinterpret_cast<uint64_t>(&kvmap)), "r"(0), "r"(key % P / 8),
                "r"(page[h] < 0 ? -1 : page[h] * planes + plane), "r"(full)
              : "memory");
        if (++kn[h] == NH) { kn[h] = 0; ++kturn[h]; }
      }
      for (int i = n.i0 + first; ok && i < n.m; i += stride) {
        if (qturn > 0 && !waitw(H.q_empty + qn, qturn - 1)) { ok = false; break; }
        const uint32_t full = sm_addr(H.q_full + qn);
        if (lane == 0)
          asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;"
                       ::"r"(full), "r"((uint32_t)(HALVES * A.tok * A.G * 128)) : "memory");
        __syncwarp();
        if (lane < HALVES)
          asm volatile(
              "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
              ::"r"(qbufs + qn * q_bytes + lane * A.q_half), "l"(reinterpret_cast<uint64_t>(&qmap)), "r"(0), "r"(lane),
                "r"(n.hk * A.G), "r"(n.r0 + i), "r"(full)
              : "memory");
        if (++qn == NQ) { qn = 0; ++qturn; }
      }
    }
    // shared memory outlives the copies (over, unless a wait was given up): each buffer's last one
#pragma unroll
    for (int h = 0; h < 2; ++h)
      for (int i = 0; i < NH; ++i) mbar_wait_deadline(sm_addr(H.k_full + h * NH + i), (i < kn[h] ? kturn[h] : kturn[h] - 1) & 1, nullptr);
    for (int i = 0; i < NQ; ++i) mbar_wait_deadline(sm_addr(H.q_full + i), (i < qn ? qturn : qturn - 1) & 1, nullptr);
  } else if (warp == MT_SUM + 1 || warp == MT_SUM + 3) {
    // ---- MMA issuer of a unit's tile h of keys (the whole warp, on values that are the same in every lane) ----
    auto same = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    const int h = same(warp) == MT_SUM + 3;
    const uint32_t one = elect_one(), tm = __shfl_sync(0xffffffffu, tmem, 0), exts = sm_addr(ext);
    const uint32_t ones = exts + MT_MAX_NQ * MT_EXT, zeros = ones + MT_EXT;
    int kn = 0, qn = 0;
    uint32_t kturn = 0, qturn = 0, tiles = 0;
    uint32_t used[2] = {0, 0};
    bool ok = true;
    while (ok && take()) {
      taken();
      const int nh = same(g.n + g.m - g.tile * MT_UNIT > MT_KEYS ? 2 : 1), i0 = same(g.i0) + first, m = same(g.m);
      const int kbuf = h * NH + kn;
      if (h < nh && !(ok = waitw(H.k_full + kbuf, kturn))) break;
      const uint64_t ad = tt_desc(kbufs + kbuf * C::BUF, 16, GROUP);
      for (int i = i0; i < m; i += stride, ++tiles) {
        const int rows = min(A.tok, m - i) * A.G, gr = tiles & 1;
        if (!(ok = waitw(H.q_full + qn, qturn))) break;          // (also where there is no tile h: one arrival a turn)
        if (h < nh) {
          // bf16 x bf16 -> f32, M = 128, N the rows in whole 16s
          const uint32_t id = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)((rows + 15) / 16 * 2) << 17) | (8u << 24);
          const uint32_t k = gr ? used[1]++ : used[0]++;
          if (k > 0 && !(ok = waitw(H.s_empty + 2 * gr + h, k - 1))) break;
          tc_fence_after();
          const uint64_t bd = tt_desc(qbufs + qn * q_bytes, 16, 1024);
          const uint32_t d = tm + (2 * gr + h) * 128, qx = exts + qn * MT_EXT;
#pragma unroll
          for (int x = 0; x < D / 16; ++x)
            mma_ss(d, ad + (uint64_t)(((x & 3) * 32 + (x >> 2) * 1024) >> 4),
                   bd + (uint64_t)(((x & 3) * 32 + (x >> 2) * A.q_half) >> 4), id, x > 0, one);
          mma_ss(d, plain_desc(ones, zeros - ones, 128), plain_desc(qx, zeros - qx, 128), id, true, one);
          tc_commit(sm_addr(H.s_full + 2 * gr + h), one);
        }
        tc_commit(sm_addr(H.q_empty + qn), one);
        if (++qn == NQ) { qn = 0; ++qturn; }
      }
      if (!ok) break;
      if (h < nh) {
        tc_commit(sm_addr(H.k_empty + kbuf), one);
        if (++kn == NH) { kn = 0; ++kturn; }
      }
    }
    // everything issued is done before TMEM is freed (also after an abort)
    tc_commit(sm_addr(H.fin + h), one);
    mbar_wait_deadline(sm_addr(H.fin + h), 0, nullptr);
  } else if (warp == MT_SUM + 2) {
    // ---- loader: the units, and (c - lse) / scale of their rows as three bf16 parts, each the rounding of
    // what the ones before leave. It reads for the next tile of rows before it waits for a place for this one.
    MassWalk<MT_UNIT> walk(A, blockIdx.x / A.pair, gridDim.x / A.pair);
    const int nbox = MT_KEYS / kb;
    int at[4];                                   // of row lane + 32 k of a tile
#pragma unroll
    for (int k = 0; k < 4; ++k) at[k] = (lane + 32 * k) / A.G * A.hq + (lane + 32 * k) % A.G;
    int qn = 0, i = 0;
    uint32_t qturn = 0;
    float lse[4], near0 = 0.f;                   // of the next tile of rows; the unit's first lse
    int rows = 0, page[2];                       // (of the unit's boxes)
    bool fresh = true, have = false, ok = true;  // the tile is its unit's first
    auto look = [&]() {                          // the next tile of rows
      if (have) i += stride;
      fresh = !have || i >= g.m;
      if (fresh) {
        do {
          if (!walk.next(g)) return false;
          i = g.i0 + first;
        } while (i >= g.m);                      // (none of this block's)
        near0 = A.lse[(size_t)(g.r0 + g.i0) * A.hq + g.hk * A.G];
        const int32_t* bt = A.kv.block_table_dev + (size_t)g.s * A.kv.max_pages;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = g.tile * MT_UNIT + h * MT_KEYS + kb * lane;
          page[h] = lane < nbox && key < g.n + g.m ? bt[key / P] : -1;
        }
      }
      const float* src = A.lse + (size_t)(g.r0 + i) * A.hq + g.hk * A.G;
      rows = min(A.tok, g.m - i) * A.G;
#pragma unroll
      for (int k = 0; k < 4; ++k) lse[k] = lane + 32 * k < rows ? src[at[k]] : 0.f;
      return true;
    };
    have = look();
    while (have) {
      const float c = mt_near(near0);
      if (fresh) {
        const int u = units % MT_RING;
        if (units >= MT_RING && !(ok = waitw(H.unit_empty + u, units / MT_RING - 1))) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (lane < nbox) {
            const bool bad = page[h] < 0 || page[h] >= A.kv.n_pages;
            if (bad && g.tile * MT_UNIT + h * MT_KEYS + kb * lane < g.n + g.m) atomicOr(A.err, DERR_PAGE);
            H.page[u][h][lane] = bad ? -1 : page[h];
          }
        }
        if (lane == 0) {
          H.unit[u] = g;
          H.near[u] = c;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sm_addr(H.unit_full + u));
        ++units;
      }
      uint16_t p[4][3];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        split_parts(lane + 32 * k < rows ? fmaf(c, LN2_LO, fmaf(c, LN2, -lse[k])) * A.inv_scale : 0.f, 0, 3, p[k]);
      have = look();
      if (qturn > 0 && !(ok = waitw(H.q_empty + qn, qturn - 1))) break;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<uint4*>(ext + qn * MT_EXT + (lane + 32 * k) * 16) = make_uint4(p[k][0] | (uint32_t)p[k][1] << 16, p[k][2], 0u, 0u);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(sm_addr(H.q_full + qn));
      if (++qn == NQ) { qn = 0; ++qturn; }
    }
    // no more units (after an abort every wait ends by itself)
    const int u = units % MT_RING;
    if (ok && (units < MT_RING || waitw(H.unit_empty + u, units / MT_RING - 1)) && lane == 0) {
      H.unit[u].s = -1;
      mbar_arrive(sm_addr(H.unit_full + u));
    }
  } else {
    // ---- the groups that sum: tiles of rows gr, gr + 2, .. against tile h of the unit's keys ----
    const int h = warp >> 2 & 1, gr = warp >> 3, r = t & 127;
    const uint32_t sT = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (2 * gr + h) * 128;
    const unsigned long long sc2 = pair(A.scale_l2e, A.scale_l2e);
    uint32_t tiles = 0, used = 0;
    // Units whose sum is joined take turns: group p finishes every other one, alike in both blocks. So each of
    // the barriers has one group that waits on it, and that one sees its every phase.
    uint32_t joined = 0, got = 0, gave = 0;
    bool ok = true;
    while (ok && take()) {
      const float c = H.near[units % MT_RING];
      taken();
      const unsigned long long nc2 = pair(-c, -c);
      const int k0 = g.tile * MT_UNIT + h * MT_KEYS + r;
      const int all = (g.m - g.i0 + A.tok - 1) / A.tok, nt = (all - rank + A.pair - 1) / A.pair;   // tiles of rows; this block's
      const int other = A.pair > 1 ? all / 2 : 0;          // the second block's
      const uint32_t t0 = tiles;
      tiles += nt;
      if (k0 - r >= g.n + g.m) continue;         // (the unit has no second tile)
      const bool join = nt > 1 || other > 0;
      const uint32_t p = join ? joined & 1 : t0 & 1, turn = joined >> 1;
      joined += join;
      const bool owner = p == (uint32_t)gr;
      const bool give = nt > 1 || (t0 & 1) != p;           // (the other group has tiles too)
      const size_t e = ((size_t)g.s * A.kv.n_kv_heads + g.hk) * A.ld + k0;
      const float before = owner && rank == 0 && A.mass && k0 < g.n ? A.mass[e] : 0.f;
      Comp sum{0.f, 0.f};
      for (int j = (int)((t0 ^ gr) & 1); j < nt; j += 2) {
        const int i = g.i0 + first + j * stride, rows = min(A.tok, g.m - i) * A.G, chunks = (rows + 31) / 32;
        // the first row that sees the key
        const long long lo64 = (long long)(k0 - g.n - i) * A.G;
        const int lo = lo64 > 128 ? 128 : lo64 < 0 ? 0 : (int)lo64;
        const bool cut = rows < 32 * chunks || __any_sync(0xffffffffu, lo > 0);
        if (!(ok = waitw(H.s_full + 2 * gr + h, used++))) break;
        tc_fence_after();
        unsigned long long part[2] = {0, 0};
#pragma unroll 1
        for (int ch = 0; ch < chunks; ++ch) {
          uint32_t v[32];
          tmem_ld32(sT + 32 * ch, v);
          if (ch == chunks - 1) {                 // the scores are read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(sm_addr(H.s_empty + 2 * gr + h));
          }
          if (cut) {
            asm volatile("" ::: "memory");       // (behind a branch, not predicated)
            const int a = lo - 32 * ch, b = rows - 32 * ch;
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (x < a || x >= b) v[x] = 0xff800000u;
          }
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            const float2 y = halves(fma2(pair(__uint_as_float(v[x]), __uint_as_float(v[x + 1])), sc2, nc2));
            part[x / 2 & 1] = add2(part[x / 2 & 1], pair(ex2(y.x), ex2(y.y)));
          }
        }
        const float2 p = halves(add2(part[0], part[1]));
        sum.add(p.x + p.y);
      }
      if (!ok) break;
      if (give) {                                // the other group's tiles
        if (!owner) {
          if (gave > 0 && !(ok = waitw(&H.sum_empty[p][h], gave - 1))) break;
          ++gave;
          H.sum[p][h * MT_KEYS + r] = sum.s + sum.e;
          __syncwarp();
          if (lane == 0) mbar_arrive(sm_addr(&H.sum_full[p][h]));
        } else {
          if (!(ok = waitw(&H.sum_full[p][h], got++))) break;
          sum.add(H.sum[p][h * MT_KEYS + r]);
          __syncwarp();
          if (lane == 0) mbar_arrive(sm_addr(&H.sum_empty[p][h]));
        }
      }
      if (other > 0 && owner) {                  // the other block's
        if (rank > 0) {
          if (turn > 0 && !(ok = waitw_pair(&H.pair_empty[p][h], turn - 1))) break;
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(map_to(sm_addr(&H.pair[p][h * MT_KEYS + r]), 0)), "f"(sum.s + sum.e) : "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive_at(map_to(sm_addr(&H.pair_full[p][h]), 0));
        } else {
          if (!(ok = waitw_pair(&H.pair_full[p][h], turn))) break;
          sum.add(H.pair[p][h * MT_KEYS + r]);
          __syncwarp();
          if (lane == 0) mbar_arrive_at(map_to(sm_addr(&H.pair_empty[p][h]), 1));
        }
      }
      if (owner && rank == 0 && k0 < g.n + g.m) A.out[e] = before + (sum.s + sum.e);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == MT_SUM) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  if (A.pair > 1) cluster_sync();                // nothing is on its way to this block any more
}

template <int D>
cudaError_t launch_mass_tc(MassArgs A, int blocks, cudaStream_t st) {
  const int kb = key_box(A.kv.page_size, MT_KEYS);
  // tiles of rows: whole tokens, no more than a chunk counts; where they are small, the room goes to keys
  A.tok = std::max(1, std::min(128 / A.G, std::min(A.last, A.ix.max_new)));
  A.q_half = (A.tok * A.G + 15) / 16 * 16 * 128;
  A.nq = A.q_half <= 4096 ? 4 : 2;
  A.nk = std::min(MT_MAX_NK, (MtCfg<D>::ROOM - A.nq * A.q_half * (D / 64)) / MtCfg<D>::BUF / 2 * 2);   // a ring for each issuer
  // Pairs of blocks where units are long and few, alone and paired: every token of a prompt of 5,288 on 8 kv heads
  // 150 and 104 us, two of them 217 and 201, four 448 and 435, four of 2,000 93 and 98, the last 512 tokens of eight
  // prompts 101 and 113; the last 32 (one tile of rows) 22 and 30. (Four of 5,288 would gain 3%, four of 2,000, as
  // many planes, lose 5%; the rule leaves both alone.)
  A.pair = (std::min({A.last, A.ix.max_new, A.ix.capacity}) + A.tok - 1) / A.tok >= MT_PAIR_TILES &&
                   (int64_t)A.ix.n_seq * A.kv.n_kv_heads <= MT_PAIR_PLANES
               ? 2
               : 1;
  CUtensorMap map, qmap;
  if (q_make_map(&qmap, A.q, D, A.hq, (uint64_t)A.ix.n_rows, A.G, A.tok) ||
      kv_make_group_map(&map, A.kv.kv_dev, D, A.kv.page_size, (uint64_t)A.kv.n_pages * A.kv.n_layers * A.kv.n_kv_heads * 2, kb))
    return cudaErrorInvalidValue;
  cudaError_t e = allow_dyn_smem_once<k_mass_tc<D>>();
  return e == cudaSuccess ? launch_clusters(k_mass_tc<D>, dim3(blocks / A.pair * A.pair), dim3(MT_THREADS), MtCfg<D>::SMEM, A.pair,
                                            st, map, qmap, A, kb)
                          : e;
}

template <int D>
cudaError_t launch_mass_fma(const MassArgs& A, int blocks, cudaStream_t st) {
  cudaError_t e = allow_dyn_smem_once<k_mass_fma<D>>();
  return e == cudaSuccess ? launch_k(k_mass_fma<D>, dim3(blocks), dim3(MF_THREADS), sizeof(MfSmem<D>), st, A) : e;
}

}  // namespace
}  // namespace spec

using namespace spec;

extern "C" int spec_attention_mass(const spec_kv_view* kv, int layer, const void* q_dev, const float* lse_dev, int n_rows,
                                   int n_seq, int max_new, int last, int n_q_heads, const int32_t* row_start_dev,
                                   const int32_t* n_new_dev, const int32_t* cache_len_dev, float scale, const float* mass_dev,
                                   float* out_mass_dev, int64_t ld, int32_t* err_dev, uintptr_t cuda_stream) {
  int rc = check_chunks(kv, n_seq, n_q_heads);
  if (rc == SPEC_OK) rc = check_layer_rows(kv, layer, n_rows, max_new);
  if (rc) return rc;
  if (!q_dev || !lse_dev || !row_start_dev || !n_new_dev || !cache_len_dev || !out_mass_dev || !err_dev)
    return set_last_error(SPEC_ERR_ARG, "null pointer argument");
  if (last < 1) return set_last_error(SPEC_ERR_ARG, "last >= 1 required");
  if (n_q_heads / kv->n_kv_heads > MS_MAX_G) return set_last_error(SPEC_ERR_UNSUPPORTED, "more than 128 query heads per kv head");
  if (!(scale > 0.f) || !(scale * LOG2E < INFINITY)) return set_last_error(SPEC_ERR_ARG, "scale must be positive, and finite times log2 e");
  if (!aligned16(q_dev)) return set_last_error(SPEC_ERR_ARG, "q must be 16-byte aligned");
  if (scale < 5.4e-20f || scale > 1.9e19f) return set_last_error(SPEC_ERR_UNSUPPORTED, "scale beyond 2^-64 .. 2^64");
  if (ld < 1 || ld > ((int64_t)1 << 31)) return set_last_error(SPEC_ERR_ARG, "1 <= ld <= 2^31 required");
  const int64_t capacity = std::min<int64_t>((int64_t)kv->max_pages * kv->page_size, ld);
  // a sequence's units, and its rows of a kv head, are counted in 32 bits
  if ((double)capacity / MF_KEYS * kv->n_kv_heads > 2e9 || (double)std::min<int64_t>(max_new, capacity) * (n_q_heads / kv->n_kv_heads) > 2e9)
    return set_last_error(SPEC_ERR_UNSUPPORTED, "block table too long for this many heads");
  const int64_t mbytes = (int64_t)n_seq * kv->n_kv_heads * ld * 4;
  if (out_mass_dev != mass_dev && spans_meet(out_mass_dev, mbytes, mass_dev, mbytes))
    return set_last_error(SPEC_ERR_ARG, "out_mass overlaps mass without being the same array");
  const int64_t rows = (int64_t)n_rows * n_q_heads;
  if (spans_meet(out_mass_dev, mbytes, lse_dev, rows * 4) ||
      spans_meet(out_mass_dev, mbytes, q_dev, rows * kv->head_dim * (kv->dtype == SPEC_F32 ? 4 : 2)))
    return set_last_error(SPEC_ERR_ARG, "out_mass overlaps lse or q");
  const int sms = sm_count_once();
  if (sms < 1) return set_last_error(SPEC_ERR_CUDA, "no device");
  const int d = kv->head_dim;
  const MassArgs A{*kv, ChunkIndex{row_start_dev, n_new_dev, cache_len_dev, n_seq, n_rows, max_new, (int)capacity}, q_dev, lse_dev,
                   mass_dev, out_mass_dev, err_dev, ld, layer, n_q_heads, n_q_heads / kv->n_kv_heads, last, 0, 0, 0, 0, 1, scale * LOG2E, 1.f / scale};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
  cudaError_t e;
  if (kv->dtype == SPEC_F32) e = d == 128 ? launch_mass_fma<128>(A, 3 * sms, st) : launch_mass_fma<64>(A, 3 * sms, st);
  else e = d == 128 ? launch_mass_tc<128>(A, sms, st) : launch_mass_tc<64>(A, sms, st);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? SPEC_OK : set_last_error(SPEC_ERR_CUDA, cudaGetErrorString(e));
}
