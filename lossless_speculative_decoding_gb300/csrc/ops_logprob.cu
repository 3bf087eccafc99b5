// Kernel-level entry point: log probabilities of given tokens, with entropy,
// rank and the likeliest alternatives, from materialised logits, in one pass
// over them.
//
// With c = log2(e) / T, m the largest logit and y = c (x - m): z = sum 2^y, log
// p(t) = ln 2 (y_t - log2 z), and entropy = ln 2 (log2 z - sum 2^y y / z), two
// terms of one sign, so that nothing cancels. The order of tokens is (logit
// descending, index ascending), NaN as -inf.
//
// A thread's sums take y' = c x - R in one instruction, R the rounded product c m,
// and are set right at the row's end by 2^-d, d = c m - R = y' - y (one more rounding
// gives it exactly). Where |R| is above 2^24, d may be above 1 and soon as large
// as an exponent's range (rows masked throughout by a finite value, tiny
// temperatures): there they take the differences x - m themselves. (Set right
// at each step: 256 rows with 20 alternatives 36.7 us.)
//
// The rows' steps of 32 KB, row after row, are cut into one even run for each
// block that the GPU holds at once, so that a few rows use all of it and many
// rows leave no tail. A warp takes 4 KB of a step, one ahead by a bulk copy into
// its own shared memory; warps wait for each other where a row ends (from the
// third on, for the place that they leave its statistics in) and, with more than
// four alternatives, at a row's steps 1, 4, 16, .. Within a row a thread keeps a
// running (m, z, sum) and a count of the logits that come before the token.
//
// A step whose sum comes out as NaN (masked tokens, NaN logits) is added again
// with care, value by value: 256 rows of 129,280 fp32 logits with 20 alternatives
// take 36 us, 44 with one token of a thousand masked, 92 with half of them; 1,100
// bf16 rows of 151,936 88, 166 and 350.
//
// Alternatives: a warp holds the best 32 of what it has seen as sorted 64-bit
// keys (ordered logit, inverted index), one per lane. A thread's step is searched
// only if its maximum is not below a bound of the block's n-th best logit, which
// comes from the threads' maxima (it only saves work: what is found does not
// depend on it). 32 found keys are sorted and merged at a time. A ninth warp ends
// the rows while the others go on; a row that several blocks share is joined, in
// the blocks' order, by the last of them to finish (which one that is changes
// nothing).
//
// Bound: fp32 logits by HBM (1,024 rows of 129,280 without alternatives: 83 us,
// 6.4 TB/s, 0.94 of the measured copy rate). 16-bit ones (1,100 rows of 151,936,
// one alternative: 86 us, 3.9 TB/s, 0.57) take 10.7 instructions a logit, of
// which a scheduler issues 0.60 a cycle: the largest stalls are the barrier at the
// rows' ends and the latency of a warp's own chain. A few rows by the chain of a
// step and a row's end, some 10 us (4 rows of 129,280, five alternatives: 12.3 us).
#include <cuda_runtime.h>

#include <algorithm>

#include "kv_view.cuh"

namespace spec {
namespace {

typedef unsigned long long u64;

constexpr int LP_THREADS = 256;                  // that take the logits; one more warp ends the rows
constexpr int LP_ALL = LP_THREADS + 32;
constexpr int LP_WARPS = LP_THREADS / 32;
constexpr int LP_UNROLL = 8;                     // 16-byte vectors a thread has in flight
constexpr int LP_TILE = LP_THREADS * LP_UNROLL;  // vectors of a block's step
constexpr int LP_STAGES = 2;                     // steps of a warp in shared memory: one being added, the others on their way
constexpr int LP_BLOCKS = 2;                     // blocks on an SM at once (three, with fewer registers each: no faster)
constexpr int LP_MAX_VOCAB = 1 << 20;
constexpr int LP_MAX_BLOCKS = 512;
constexpr int LP_TOP = SPEC_LOGPROB_MAX_TOP;
static_assert(LP_TOP == 32, "a warp's list has one key per lane");

// What a block leaves of a row it shares: statistics, and a sorted list apart.
struct LpStats {
  float m, z, zy;           // largest logit, sum 2^y, sum 2^y y
  int before, bad;          // logits before the token; a NaN or +inf logit
};

struct LpArgs {
  const void* logits;
  int64_t ld;
  int n_rows, vocab, top_n, tiles;               // tiles: steps of a row
  const int32_t* tokens;
  float it, c;              // 1 / temperature, log2(e) / temperature
  float* logprob;
  float* entropy;
  int32_t* rank;
  int32_t* top_ids;
  float* top_lp;
  int* arrived;             // [LP_MAX_BLOCKS], of the row that starts in a block and goes on; zero between calls
  LpStats* stats;           // [LP_MAX_BLOCKS][2]: of a row begun in an earlier block, of one that goes on in the next
  u64* lists;               // [LP_MAX_BLOCKS][2][32]
};

template <class T> __device__ __forceinline__ float logit(const T* row, int v);
template <> __device__ __forceinline__ float logit<float>(const float* row, int v) { return row[v]; }
template <> __device__ __forceinline__ float logit<bf16_t>(const bf16_t* row, int v) { return bf16_to_f(row[v].v); }

__device__ __forceinline__ float lp_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float above(float x, float lim) {
  float r;
  asm("set.gt.f32.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(lim));
  return r;
}

// Vector j of a lane's part of a step, at shared address a; volatile, so that it
// is read again and not kept in registers from one use to the next.
__device__ __forceinline__ uint4 reread(uint32_t a, int j) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a + j * 512) : "memory");
  return v;
}

// A 16-byte vector's values, two at a time, and the maximum of a step's vectors
// (NaN as -inf).
template <class T> struct LpVec;
template <> struct LpVec<float> {
  static __device__ __forceinline__ float2 at(const uint4& v, int j) {
    return j ? make_float2(__uint_as_float(v.z), __uint_as_float(v.w)) : make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
  }
  // the value below x in the order of the type; how many of a vector are above lim
  static __device__ __forceinline__ float below(float x) { return nextafterf(x, -INFINITY); }
  typedef float Lim;
  typedef float Count;
  static __device__ __forceinline__ Lim lim(float x) { return x; }
  static __device__ __forceinline__ void count(Count& n, const uint4& v, Lim l) {
    n += (above(__uint_as_float(v.x), l) + above(__uint_as_float(v.y), l)) + (above(__uint_as_float(v.z), l) + above(__uint_as_float(v.w), l));
  }
  static __device__ __forceinline__ float total(Count n) { return n; }
  // A running maximum (NaN left out).
  typedef float Max;
  static __device__ __forceinline__ Max none() { return -INFINITY; }
  static __device__ __forceinline__ void larger(Max& m, const uint4& v) {
    asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(__uint_as_float(v.x)), "f"(__uint_as_float(v.y)));
    asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(__uint_as_float(v.z)), "f"(__uint_as_float(v.w)));
  }
  static __device__ __forceinline__ float value(Max m) { return m; }
};
template <> struct LpVec<bf16_t> {
  static __device__ __forceinline__ float2 at(const uint4& v, int j) {
    const uint32_t w = j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  static __device__ __forceinline__ float below(float x) {
    const uint32_t b = __float_as_uint(x);
    return x == 0.f ? __uint_as_float(0x80010000u) : __uint_as_float(b & 0x80000000u ? b + 0x10000u : b - 0x10000u);
  }
  typedef __nv_bfloat162 Lim;
  typedef __nv_bfloat162 Count;                  // two counts of a step, exact up to 256
  static_assert(LP_UNROLL * 4 <= 256, "counts in bf16");
  static __device__ __forceinline__ Lim lim(float x) { return __float2bfloat162_rn(x); }
  static __device__ __forceinline__ void count(Count& n, const uint4& v, Lim l) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) n = __hadd2(n, __hgt2(*reinterpret_cast<const __nv_bfloat162*>(&w[j]), l));
  }
  static __device__ __forceinline__ float total(Count n) {
    const float2 f = __bfloat1622float2(n);
    return f.x + f.y;
  }
  typedef uint2 Max;
  static __device__ __forceinline__ Max none() { return make_uint2(0xff80ff80u, 0xff80ff80u); }   // -inf
  static __device__ __forceinline__ void larger(Max& m, const uint4& v) {
    asm("max.bf16x2 %0, %1, %2;" : "=r"(m.x) : "r"(m.x), "r"(v.x));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(m.y) : "r"(m.y), "r"(v.y));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(m.x) : "r"(m.x), "r"(v.z));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(m.y) : "r"(m.y), "r"(v.w));
  }
  static __device__ __forceinline__ float value(Max m) {
    uint32_t a;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(m.x), "r"(m.y));
    return fmaxf(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u));
  }
};

// Keys: larger logit first, then the lower index. 0 is below every real key.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(am_key(x) + 0.f);     // one zero
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ u64 key_of(float x, int v) { return ((u64)ordered(x) << 32) | (uint32_t)~v; }
__device__ __forceinline__ float key_value(u64 k) { return unordered((uint32_t)(k >> 32)); }
__device__ __forceinline__ int key_index(u64 k) { return (int)~(uint32_t)k; }

// Bitonic networks over a warp, one key per lane, lane 0 the largest.
template <class K>
__device__ __forceinline__ K exchange(K k, int j, bool larger) {
  const K o = __shfl_xor_sync(0xffffffffu, k, j);
  return larger == (k > o) ? k : o;
}
template <class K>
__device__ __forceinline__ K warp_sort(K k) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 2; n <= 32; n <<= 1)
#pragma unroll
    for (int j = n >> 1; j > 0; j >>= 1) k = exchange(k, j, ((lane & j) == 0) == ((lane & n) == 0 || n == 32));
  return k;
}
// The best 32 of two sorted lists, sorted.
template <class K>
__device__ __forceinline__ K warp_merge(K a, K b) {
  const int lane = threadIdx.x & 31;
  const K r = __shfl_sync(0xffffffffu, b, 31 - lane);
  K k = a > r ? a : r;
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) k = exchange(k, j, (lane & j) == 0);
  return k;
}

// The best 32 of eight of them, as a tree: three merges' latency.
__device__ __forceinline__ u64 warp_merge8(u64 (&k)[8]) {
#pragma unroll
  for (int d = 1; d < 8; d <<= 1)
#pragma unroll
    for (int i = 0; i < 8; i += 2 * d) k[i] = warp_merge(k[i], k[i + d]);
  return k[0];
}

constexpr float LP_FAR = 16777216.f;             // |c m| up to which a step's sums go by the product

// c (x - m) of logits at the types' ends too: halves, whose difference stays in range.
__device__ __forceinline__ float lp_diff(float x, float m, float c) { return fmaf(0.5f, x, -0.5f * m) * c * 2.f; }
// The same with a floor below any power, for sums of 2^y y (x = -inf: masked, nothing seen).
__device__ __forceinline__ float lp_shift(float x, float m, float c) { return fmaxf(lp_diff(x, m, c), -1e30f); }

// (m, z, zy) += (m2, z2, zy2), either of which may hold nothing (m = -inf).
__device__ __forceinline__ void stats_merge(float& m, float& z, float& zy, float m2, float z2, float zy2, float c) {
  const bool keep = m >= m2;                     // the one with the larger logit stays as it is
  const float mm = keep ? m : m2, by = lp_shift(keep ? m2 : m, mm == -INFINITY ? 0.f : mm, c), f = lp_ex2(by);
  const float zl = keep ? z2 : z, zyl = keep ? zy2 : zy;
  zy = fmaf(fmaf(zl, by, zyl), f, keep ? zy : zy2);
  z = fmaf(zl, f, keep ? z : z2);
  m = mm;
}

struct LpShared {
  LpStats stats[2][LP_WARPS];                    // the warps' parts of a row, for the warp that ends it
  u64 list[2][LP_WARPS][32];
  u64 pend[LP_WARPS][64];                        // found keys
  uint64_t full[LP_WARPS][LP_STAGES];            // a warp's step is there
  int abort;
  u64 top[32];                                   // each warp's four largest thread maxima, with their row
};

template <class T>
__global__ void __launch_bounds__(LP_ALL, LP_BLOCKS) k_logprob(const __grid_constant__ LpArgs A) {
  constexpr int PER = Elt<T>::per16, U = LP_UNROLL, STEP = U * PER;
  static_assert(STEP % 32 == 0, "whole warps search a thread's step");
  __shared__ LpShared sh;
  const int t = threadIdx.x, lane = t & 31, w = t >> 5, V = A.vocab, n = A.top_n;
  const int64_t units = (int64_t)A.n_rows * A.tiles, end = units * (blockIdx.x + 1) / gridDim.x;
  int64_t pos = units * blockIdx.x / gridDim.x;  // (the grid has no more blocks than there are units)
  const float nan = __int_as_float(0x7fc00000), LN2 = 0.6931471805599453f;
  int r = (int)(pos / A.tiles), s0 = (int)(pos % A.tiles), rows = 0;
  // Rows are handed over through the two halves of `stats` and `list`: barrier
  // 1 + half when one is written, 3 + half when it is read.
  auto bar_sync = [](int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); };
  auto bar_arrive = [](int id, int n) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory"); };
  if (w < LP_WARPS) {
  // A warp's part of a step is 4 KB of the row in one piece. It goes through the
  // warp's own stages of shared memory, by a bulk copy; no other warp waits for it.
  extern __shared__ __align__(16) uint4 stage_mem[];       // [LP_WARPS][LP_STAGES][U * 32]
  uint4* stage = stage_mem + w * LP_STAGES * U * 32;
  if (lane == 0) {
    for (int i = 0; i < LP_STAGES; ++i)
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"((uint32_t)__cvta_generic_to_shared(&sh.full[w][i])));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    sh.abort = 0;
  }
  if (lane < 32 / LP_WARPS) sh.top[32 / LP_WARPS * w + lane] = 0;
  bar_sync(5, LP_THREADS);
  int in = 0, out = 0, filled = 0, phase = 0;              // stages to fill and to read next; their phases
  auto row_of = [&](int i) { return static_cast<const T*>(A.logits) + (int64_t)i * A.ld; };
  auto skip_of = [&](const T* row) { return (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T)); };
  auto fetch = [&](const T* row, int skip, int st) {       // (every lane has read what the stage held)
    uint4* dst = stage + in * U * 32;
    const uint32_t bar = (uint32_t)__cvta_generic_to_shared(&sh.full[w][in]);
    if (++in == LP_STAGES) {
      in = 0;
      filled ^= 1;
    }
    const int e0 = (st * LP_TILE + w * 32 * U) * PER - skip;
    int v0 = 0, v1 = U * 32;                               // vectors that lie whole in the row
    if (e0 < 0 || e0 + U * 32 * PER > V) {                 // an end of the row: -inf outside it
      v0 = e0 < 0 ? 1 : 0;
      v1 = max(v0, min(v1, (V - e0) / PER));
      if (e0 >= V) v1 = v0;                                // (nothing of it is looked at)
      else for (int i = lane; i < U * 32; i += 32) {
        if (i >= v0 && i < v1) continue;
        const int e = e0 + i * PER;
        T* x = reinterpret_cast<T*>(dst + i);
#pragma unroll 1
        for (int q = 0; q < PER; ++q) {
          if constexpr (sizeof(T) == 4) x[q] = e + q >= 0 && e + q < V ? row[e + q] : -INFINITY;
          else x[q].v = e + q >= 0 && e + q < V ? row[e + q].v : 0xff80;
        }
      }
      // before a later bulk copy into the same bytes (its issue follows a __syncwarp)
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (lane == 0) {
      const uint32_t bytes = (uint32_t)(v1 - v0) * 16;
      asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
      if (bytes)
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                     ::"r"((uint32_t)__cvta_generic_to_shared(dst + v0)), "l"(row + (e0 + v0 * PER)), "r"(bytes), "r"(bar) : "memory");
    }
  };
  // the fetches run LP_STAGES - 1 steps ahead of (r, st), over the block's rows
  int left = (int)(end - pos), f_step = s0, f_skip = skip_of(row_of(r));   // (a block has far fewer than 2^31 steps)
  const T* f_row = row_of(r);
  bool lost = false;                                       // a copy was given up (by the whole warp)
  auto fetch_next = [&]() {
    if (left == 0) return;
    fetch(f_row, f_skip, f_step);
    --left;
    if (++f_step == A.tiles) {
      f_step = 0;
      f_row += A.ld;
      f_skip = skip_of(f_row);
    }
  };
  for (int i = 0; i < LP_STAGES - 1; ++i) fetch_next();
#pragma unroll 1
  for (; pos < end; ++r, s0 = 0, ++rows) {
    const int s1 = (int)min((int64_t)A.tiles, s0 + (end - pos));
    pos += s1 - s0;
    // the row as aligned vectors, a warp's of a step next to each other: vector i holds elements i PER - skip ..
    const T* row = row_of(r);
    const int skip = skip_of(row);
    const int tok = A.tokens ? A.tokens[r] : -1;
    const bool have = tok >= 0 && tok < V;
    const float raw_t = have ? logit<T>(row, tok) : 0.f, key_t = am_key(raw_t);
    // a logit comes before the token if it is larger, or equal at a lower
    // index: x > up in vectors behind the token's (and, but for its ties, in
    // it), x > down, the next value below, in vectors ahead of it
    const int tvec = have ? (tok + skip) / PER : -1;
    const bool low = have && key_t == -INFINITY;           // ties with NaN and -inf: compared one by one
    const float up = have && !low ? key_t : INFINITY, down = have && !low ? LpVec<T>::below(key_t) : INFINITY;
    float m = -INFINITY;                                   // the largest logit
    float R = 0.f;                                         // c m rounded
    bool far = false;                                      // |R| above LP_FAR: sums by differences
    auto rest_of = [&]() { return far ? 0.f : fmaf(A.c, m, -R); };           // d: the sums are against c m - d
    auto start_at = [&](float to) {
      m = to;
      R = A.c * to;
      far = !(fabsf(R) <= LP_FAR);
    };
    float z = 0.f, zy = 0.f, ahead = 0.f;
    int before = 0, pending = 0;
    bool bad = lost;
    u64 list = 0;
    uint32_t bound = 0;                                    // no key below it can be among the block's best n
#pragma unroll 1
    for (int st = s0; st < s1; ++st) {
      const int first = st * LP_TILE + w * 32 * U + lane;
      fetch_next();
      if (!__all_sync(0xffffffffu, mbar_wait_deadline((uint32_t)__cvta_generic_to_shared(&sh.full[w][out]), phase, &sh.abort))) {
        // (not expected: the values of this row and the block's later ones become NaN; no more copies)
        *reinterpret_cast<volatile int*>(&sh.abort) = DERR_TIMEOUT;
        bad = lost = true;
        left = 0;
      }
      __syncwarp();
      const uint4* mine = stage + out * U * 32 + lane;
      const uint32_t at = (uint32_t)__cvta_generic_to_shared(mine);
      if (++out == LP_STAGES) {
        out = 0;
        phase ^= 1;
      }
      float bm = -INFINITY;
      if ((st * LP_TILE + w * 32 * U) * PER - skip < V) {  // (the last step may end before the warp's part of it)
        auto move_to = [&](float to) {                       // a larger m
          const float was = m, d = rest_of();
          float by = R;
          const bool apart = far;
          start_at(to);
          by -= R;
          if (apart || far) by = fmaxf(lp_diff(was, to, A.c) - d + rest_of(), -1e30f);
          const float f = lp_ex2(by);
          zy = fmaf(z, by, zy) * f;
          z *= f;
        };
        typename LpVec<T>::Max run = LpVec<T>::none();
        if (m == -INFINITY) {                                // nothing seen yet: the step's own maximum first
#pragma unroll
          for (int j = 0; j < U; ++j) LpVec<T>::larger(run, reread(at, j));
          bm = LpVec<T>::value(run);
          if (bm > -INFINITY) start_at(bm);
        }
        float z0 = 0.f, z1 = 0.f, zy0 = 0.f, zy1 = 0.f;      // (the step's own sums: two chains each)
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const uint4 v = reread(at, j);
          LpVec<T>::larger(run, v);
#pragma unroll
          for (int q = 0; q < PER / 2; ++q) {
            const float2 x = LpVec<T>::at(v, q);
            const float ya = fmaf(x.x, A.c, -R), yb = fmaf(x.y, A.c, -R), pa = lp_ex2(ya), pb = lp_ex2(yb);
            z0 += pa;
            z1 += pb;
            zy0 = fmaf(pa, ya, zy0);
            zy1 = fmaf(pb, yb, zy1);
          }
        }
        bm = LpVec<T>::value(run);
        zy0 += zy1;
        z0 += z1;
        // masked tokens (0 times -inf), NaN, values at the type's ends, or a
        // logit so far above all before that its power is infinite
        if (!(fabsf(zy0) < INFINITY) || far) {
          if (bm > m) move_to(bm);
          const float mb = m == -INFINITY ? 0.f : m;
          z0 = zy0 = 0.f;
#pragma unroll 4
          for (int e = 0; e < STEP; ++e) {
            const float x = logit<T>(reinterpret_cast<const T*>(mine + e / PER * 32), e % PER);
            // (a difference that passes fp32's range is as far below zero in c (x - m), m being far)
            const float y = fmaxf(far ? (x - mb) * A.c : fmaf(x, A.c, -R), -1e30f), p = lp_ex2(y);
            bad = bad || !(x < INFINITY);
            z0 += p;
            zy0 = fmaf(p, y, zy0);
          }
        }
        z += z0;
        zy += zy0;
        if (bm > m) move_to(bm);                             // m follows the maximum, so that the entropy's terms keep one sign
        if (bm > down) {                                     // some may come before the token
          typename LpVec<T>::Count some = LpVec<T>::lim(0.f);
          const typename LpVec<T>::Lim lu = LpVec<T>::lim(up), ld = LpVec<T>::lim(down);
#pragma unroll
          for (int j = 0; j < U; ++j) LpVec<T>::count(some, reread(at, j), first + 32 * j < tvec ? ld : lu);
          ahead += LpVec<T>::total(some);
        }
        if (low) {
#pragma unroll 1
          for (int e = 0; e < STEP; ++e) {
            const int i = (first + 32 * (e / PER)) * PER - skip + e % PER;
            if (i >= 0 && i < V) before += logit<T>(row, i) > -INFINITY || i < tok;
          }
        }
      }
      if (n == 0) {
        __syncwarp();                                      // before the stage is filled again
        continue;
      }
      // After 1, 4, 16, .. steps a warp makes its four largest thread maxima
      // known, marked with the row. The n-th largest of those that are there
      // bounds the n-th best logit seen, and so does the warp's own n-th largest.
      // A few alternatives take what is there; more wait for the other warps,
      // whose maxima they need (with the barrier / without: 256 fp32 rows, top 1
      // 30.9 / 31.0 us, 4 33.0 / 32.8, 5 33.0 / 33.8, 20 36.6 / 48.2; 1,100 bf16
      // rows, top 1 89.0 / 88.0, 4 95.8 / 95.8, 5 97.4 / 99.0, 20 123 / 171).
      const int done = st - s0 + 1;
      if ((done & (done - 1)) == 0 && (done & 0x55555555)) {
        uint32_t k = ordered(m);
#pragma unroll
        for (int i = 0; i < 32 / LP_WARPS; ++i) {
          const uint32_t mx = __reduce_max_sync(0xffffffffu, k);
          if (lane == 0) *reinterpret_cast<volatile u64*>(&sh.top[32 / LP_WARPS * w + i]) = ((u64)(rows + 1) << 32) | mx;
          if (lane == __ffs(__ballot_sync(0xffffffffu, k == mx)) - 1) k = 0;
        }
        if (n > 4) bar_sync(5, LP_THREADS);
        else __syncwarp();
        const u64 known = *reinterpret_cast<volatile u64*>(&sh.top[lane]);
        const uint32_t mine_or_none = (uint32_t)(known >> 32) == (uint32_t)(rows + 1) ? (uint32_t)known : 0u;
        uint32_t b = n == 1 ? __reduce_max_sync(0xffffffffu, mine_or_none) : __shfl_sync(0xffffffffu, warp_sort(mine_or_none), n - 1);
        if (b == 0) b = __shfl_sync(0xffffffffu, warp_sort(ordered(m)), n - 1);
        bound = bound > b ? bound : b;
      }
      const bool cand = ordered(bm) >= bound;
      uint32_t rest = __ballot_sync(0xffffffffu, cand);
      __syncwarp();
      if (!rest) continue;
      do {                                                 // a thread's step, a logit per lane at a time
        const int src = __ffs(rest) - 1;
        rest &= rest - 1;
        const uint4* its = mine - lane + src;
#pragma unroll 1
        for (int e = lane; e < STEP; e += 32) {
          const int i = (st * LP_TILE + (w * U + e / PER) * 32 + src) * PER - skip + e % PER;
          const u64 k = i >= 0 && i < V ? key_of(logit<T>(reinterpret_cast<const T*>(its + e / PER * 32), e % PER), i) : 0;
          const u64 least = __shfl_sync(0xffffffffu, list, n - 1);
          const bool in = k > least && (uint32_t)(k >> 32) >= bound;
          const uint32_t who = __ballot_sync(0xffffffffu, in);
          if (in) sh.pend[w][pending + __popc(who & ((1u << lane) - 1))] = k;
          pending += __popc(who);
          if (pending >= 32) {                             // 32 of them into the list
            __syncwarp();
            const u64 p = sh.pend[w][lane], more = sh.pend[w][32 + lane];
            __syncwarp();
            sh.pend[w][lane] = more;
            pending -= 32;
            list = warp_merge(list, warp_sort(p));
            const uint32_t nth = (uint32_t)(__shfl_sync(0xffffffffu, list, n - 1) >> 32);
            bound = bound > nth ? bound : nth;
            __syncwarp();
          }
        }
      } while (rest);
      __syncwarp();                                        // before the stage is filled again
    }

    // ---- the block's part of the row: the warps' statistics and lists to one of them ----
    if (n > 0 && pending > 0) {
      __syncwarp();
      list = warp_merge(list, warp_sort(lane < pending ? sh.pend[w][lane] : 0));
      __syncwarp();
    }
    if (m > -INFINITY) {
      const float d = rest_of(), f = lp_ex2(-d);
      zy = fmaf(-d, z, zy) * f;
      z *= f;
    }
    before = __reduce_add_sync(0xffffffffu, before + (int)ahead);
    bad = __any_sync(0xffffffffu, bad);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float mo = __shfl_xor_sync(0xffffffffu, m, o), zo = __shfl_xor_sync(0xffffffffu, z, o),
                  zyo = __shfl_xor_sync(0xffffffffu, zy, o);
      stats_merge(m, z, zy, mo, zo, zyo, A.c);
    }
    const int half = rows & 1;                             // the next row takes the other one
    if (rows >= 2) bar_sync(3 + half, LP_ALL);
    if (lane == 0) sh.stats[half][w] = LpStats{m, z, zy, before, bad};
    if (n > 0) sh.list[half][w][lane] = list;
    bar_arrive(1 + half, LP_ALL);
  }
  // shared memory outlives the copies (over, unless one was given up): each stage's last one
  if (lost)
    for (int i = 0; i < LP_STAGES; ++i)
      mbar_wait_deadline((uint32_t)__cvta_generic_to_shared(&sh.full[w][i]), i < in ? filled : filled ^ 1, nullptr);
  return;
  }

  // ---- the ninth warp: a row's end ----
#pragma unroll 1
  for (; pos < end; ++r, s0 = 0, ++rows) {
    const int s1 = (int)min((int64_t)A.tiles, s0 + (end - pos)), half = rows & 1;
    pos += s1 - s0;
    const T* row = static_cast<const T*>(A.logits) + (int64_t)r * A.ld;
    const int skip = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    const int tok = A.tokens ? A.tokens[r] : -1;
    const bool have = tok >= 0 && tok < V;
    const float raw_t = have ? logit<T>(row, tok) : 0.f, key_t = am_key(raw_t);
    const bool low = have && key_t == -INFINITY;
    // ties of the token ahead of it in its vector, which the others left out
    int before = 0, ties = 0;
    if (have && !low && A.rank) {
      const int v0 = max(0, (tok + skip) / PER * PER - skip);
      ties = __popc(__ballot_sync(0xffffffffu, v0 + lane < tok && am_key(logit<T>(row, v0 + lane)) == key_t));
    }
    float m, z, zy;
    bool bad;
    u64 list = 0;
    // `parts` statistics, in lanes 0 .. (at most 32 at a time), in a fixed tree
    auto gather = [&](auto&& of, int parts) {
      m = -INFINITY;
      z = zy = 0.f;
      before = 0;
      bad = false;
      for (int p0 = 0; p0 < parts; p0 += 32) {
        LpStats q{-INFINITY, 0.f, 0.f, 0, 0};
        if (p0 + lane < parts) q = of(p0 + lane);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const float mo = __shfl_xor_sync(0xffffffffu, q.m, o), zo = __shfl_xor_sync(0xffffffffu, q.z, o),
                      zyo = __shfl_xor_sync(0xffffffffu, q.zy, o);
          stats_merge(q.m, q.z, q.zy, mo, zo, zyo, A.c);
        }
        stats_merge(m, z, zy, q.m, q.z, q.zy, A.c);
        before += __reduce_add_sync(0xffffffffu, q.before);
        bad = bad || __any_sync(0xffffffffu, q.bad != 0);
      }
    };
    bar_sync(1 + half, LP_ALL);
    gather([&](int i) { return sh.stats[half][i]; }, LP_WARPS);
    u64 k[LP_WARPS];
    if (n > 0) {
#pragma unroll
      for (int i = 0; i < LP_WARPS; ++i) k[i] = sh.list[half][i][lane];
      list = warp_merge8(k);
    }
    __syncwarp();
    bar_arrive(3 + half, LP_ALL);
    if (s0 > 0 || s1 < A.tiles) {
      // ---- a shared row: leave the part; the last of its blocks, b0 .. b1, joins them ----
      const int64_t u0 = (int64_t)r * A.tiles;
      auto block_of = [&](int64_t unit) { return (int)(((unit + 1) * gridDim.x - 1) / units); };
      const int b0 = block_of(u0), b1 = block_of(u0 + A.tiles - 1);
      auto slot = [&](int b) { return (size_t)b * 2 + (b == b0 ? 1 : 0); };
      const size_t mine = slot(blockIdx.x);
      if (n > 0) A.lists[mine * 32 + lane] = list;
      if (lane == 0) A.stats[mine] = LpStats{m, z, zy, before, bad};
      __threadfence();
      __syncwarp();
      int last = 0;
      if (lane == 0) last = atomicAdd(A.arrived + b0, 1) == b1 - b0;
      if (!__shfl_sync(0xffffffffu, last, 0)) continue;
      __threadfence();
      if (lane == 0) A.arrived[b0] = 0;
      auto fetch = [&](int b) {                            // eight lists' loads in flight
#pragma unroll
        for (int i = 0; i < LP_WARPS; ++i) k[i] = b + i <= b1 ? __ldcg(A.lists + slot(b + i) * 32 + lane) : 0;
      };
      if (n > 0) fetch(b0);
      gather([&](int i) {
        const LpStats* q = A.stats + slot(b0 + i);
        return LpStats{__ldcg(&q->m), __ldcg(&q->z), __ldcg(&q->zy), __ldcg(&q->before), __ldcg(&q->bad)};
      }, b1 - b0 + 1);
      if (n > 0) {
        list = warp_merge8(k);
        for (int b = b0 + LP_WARPS; b <= b1; b += LP_WARPS) {
          fetch(b);
          list = warp_merge(list, warp_merge8(k));
        }
      }
    }
    const bool none = bad || m == -INFINITY;
    const float lz = none ? nan : log2f(z);
    auto logp = [&](float x) {                             // (in natural units where those of base 2 may pass fp32's range)
      const float y = lp_diff(x, m, A.c);
      return y > -1e30f ? (y - lz) * LN2 : fmaf(-LN2, lz, lp_diff(x, m, A.it));
    };
    if (lane == 0) {
      if (A.logprob) A.logprob[r] = have ? logp(raw_t) : nan;
      if (A.entropy) A.entropy[r] = none ? nan : (lz - zy / z) * LN2;
      if (A.rank) A.rank[r] = have ? before + ties + 1 : 0;
    }
    if (lane < n) {
      A.top_ids[(size_t)r * n + lane] = key_index(list);
      A.top_lp[(size_t)r * n + lane] = logp(key_value(list));
    }
  }
}

// Counters first, then statistics and lists; the same for every shape, so that
// any calls may follow each other on a workspace.
struct LpWs {
  static constexpr size_t stats = LP_MAX_BLOCKS * sizeof(int);
  static constexpr size_t lists = (stats + 2 * LP_MAX_BLOCKS * sizeof(LpStats) + 15) / 16 * 16;
  static constexpr size_t total = lists + 2 * LP_MAX_BLOCKS * 32 * sizeof(u64);
};

template <class T>
cudaError_t launch_logprob(LpArgs A, cudaStream_t st) {
  // vectors of a row at the least alignment, steps of those, blocks for the steps
  constexpr int per = 16 / (int)sizeof(T), tile = LP_TILE;
  A.tiles = ((A.vocab + per - 1 + per - 1) / per + tile - 1) / tile;
  const int sms = sm_count_once();
  if (sms < 1) return cudaErrorInvalidDevice;
  const int blocks = (int)std::min<int64_t>((int64_t)A.n_rows * A.tiles, std::min(LP_BLOCKS * sms, LP_MAX_BLOCKS));
  constexpr size_t smem = LP_STAGES * LP_TILE * 16;
  const cudaError_t e = allow_dyn_smem_once<k_logprob<T>>();
  if (e != cudaSuccess) return e;
  k_logprob<T><<<blocks, LP_ALL, smem, st>>>(A);
  return cudaGetLastError();
}

}  // namespace
}  // namespace spec

using namespace spec;

extern "C" int64_t spec_token_logprobs_ws_bytes(int n_rows, int vocab, int top_n) {
  if (n_rows < 1 || n_rows > 65535 || vocab < 1 || top_n < 0 || top_n > LP_TOP || top_n > vocab)
    return set_last_error(SPEC_ERR_ARG, "1 <= n_rows <= 65535, vocab >= 1 and 0 <= top_n <= min(32, vocab) required");
  if (vocab > LP_MAX_VOCAB) return set_last_error(SPEC_ERR_UNSUPPORTED, "vocab above 1048576");
  return (int64_t)LpWs::total;
}

extern "C" int spec_token_logprobs(const void* logits_dev, int dtype, int64_t ld, int n_rows, int vocab,
                                   const int32_t* tokens_dev, float temperature, int top_n, float* out_logprob_dev,
                                   float* out_entropy_dev, int32_t* out_rank_dev, int32_t* out_top_ids_dev,
                                   float* out_top_logprobs_dev, void* ws_dev, size_t ws_bytes,
                                   uintptr_t cuda_stream) {
  const int64_t need = spec_token_logprobs_ws_bytes(n_rows, vocab, top_n);
  if (need < 0) return (int)need;
  if (!logits_dev || !ws_dev || (!tokens_dev && (out_logprob_dev || out_rank_dev)) ||
      (top_n > 0 && (!out_top_ids_dev || !out_top_logprobs_dev)))
    return set_last_error(SPEC_ERR_ARG, "null pointer argument");
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return set_last_error(SPEC_ERR_UNSUPPORTED, "logits: F32 or BF16");
  if (ld < vocab) return set_last_error(SPEC_ERR_ARG, "ld below vocab");
  const float c = 1.4426950408889634f / temperature;
  if (!(temperature > 0.f) || !(c < INFINITY) || !(1.f / temperature > 0.f)) return set_last_error(SPEC_ERR_ARG, "temperature must be positive");
  const int esz = dtype == SPEC_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits_dev) % esz || !aligned16(ws_dev))
    return set_last_error(SPEC_ERR_ARG, "misaligned logits or workspace");
  if ((int64_t)ws_bytes < need) return set_last_error(SPEC_ERR_ARG, "workspace too small");
  char* w = static_cast<char*>(ws_dev);
  const LpArgs A{logits_dev, ld, n_rows, vocab, top_n, 0, tokens_dev, 1.f / temperature, c, out_logprob_dev,
                 out_entropy_dev, out_rank_dev, out_top_ids_dev, out_top_logprobs_dev, reinterpret_cast<int*>(w),
                 reinterpret_cast<LpStats*>(w + LpWs::stats), reinterpret_cast<u64*>(w + LpWs::lists)};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = dtype == SPEC_F32 ? launch_logprob<float>(A, st) : launch_logprob<bf16_t>(A, st);
  return e == cudaSuccess ? SPEC_OK : set_last_error(SPEC_ERR_CUDA, cudaGetErrorString(e));
}
