// Kernel-level entry point: log probabilities of given tokens, with entropy,
// rank and the likeliest alternatives, from materialised logits, in one pass
// over them.
//
// With m the largest logit x and y = (x - m) log2(e) / T (the difference first:
// a row of the type's lowest values stays a row of equal ones): z = sum 2^y, log
// p(t) = ln 2 (y_t - log2 z), and entropy = ln 2 (log2 z - sum 2^y y / z), two
// terms of one sign, so that nothing cancels. The order of tokens is (logit
// descending, index ascending), NaN as -inf.
//
// A row is cut into slices, one block each; a thread keeps a running (m, z,
// sum) and a count of the logits that come before the token, batch by batch,
// with the batch's maximum taken first. Alternatives: a warp holds the best 32
// of what it has seen as sorted 64-bit keys (ordered logit, inverted index),
// one per lane. An element joins the warp's pending buffer only if it is not
// below a bound of the block's n-th best logit, which the batch maximum decides
// for a whole batch at once; the bound is the n-th largest of the threads'
// maxima, renewed after 1, 2, 4, .. steps. 32 pending keys are sorted and merged
// at a time. The last block of a row to finish joins the
// slices in their order (which block that is changes nothing).
//
// Bound: HBM. The logits are read once; some eight instructions a logit, one
// of them an exponential, keep the SMs at about half to two thirds of their
// issue rate while the logits stream.
#include <cuda_runtime.h>

#include <algorithm>

#include "kv_view.cuh"

namespace spec {
namespace {

typedef unsigned long long u64;

constexpr int LP_THREADS = 256;
constexpr int LP_WARPS = LP_THREADS / 32;
constexpr int LP_UNROLL = 4;                     // 16-byte vectors a thread has in flight
constexpr int LP_TILE = LP_THREADS * LP_UNROLL;  // vectors of a block's step
constexpr int LP_MAX_VOCAB = 1 << 20;
constexpr int LP_MAX_SLICES = 64;
constexpr int LP_COUNTERS = 4096;                // rows of a call that may cut them into slices
constexpr int LP_TOP = SPEC_LOGPROB_MAX_TOP;
// Blocks on an SM at once: the bf16 form holds twice the values in registers.
__host__ __device__ constexpr int lp_blocks(int esz) { return esz == 4 ? 4 : 3; }
static_assert(LP_TOP == 32, "a warp's list has one key per lane");

// What a slice leaves: statistics, and (behind them) its sorted keys.
struct LpStats {
  float m, z, zy;           // max x, sum 2^y, sum 2^y y
  int before, bad;          // logits before the token; a NaN or +inf logit
};

struct LpArgs {
  const void* logits;
  int64_t ld;
  int n_rows, vocab, top_n, slices;
  const int32_t* tokens;
  float it, c;              // 1 / temperature, log2(e) / temperature
  float* logprob;
  float* entropy;
  int32_t* rank;
  int32_t* top_ids;
  float* top_lp;
  int* arrived;             // [LP_COUNTERS], zero between calls
  LpStats* stats;           // [n_rows][slices]
  u64* lists;               // [n_rows][slices][32]
};

template <class T> __device__ __forceinline__ float logit(const T* row, int v);
template <> __device__ __forceinline__ float logit<float>(const float* row, int v) { return row[v]; }
template <> __device__ __forceinline__ float logit<bf16_t>(const bf16_t* row, int v) { return bf16_to_f(row[v].v); }

__device__ __forceinline__ float lp_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two fp32 values in one 64-bit register pair, for the packed instructions.
__device__ __forceinline__ u64 pair(float a, float b) {
  u64 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 halves(u64 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
  u64 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
  u64 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
  u64 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// A 16-byte vector: its maximum (NaN if it holds one), its minimum, and its
// values, two at a time.
template <class T> struct LpVec;
template <> struct LpVec<float> {
  static __device__ __forceinline__ float2 at(const uint4& v, int j) {
    return j ? make_float2(__uint_as_float(v.z), __uint_as_float(v.w)) : make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
  }
  static __device__ __forceinline__ void range(const uint4& v, float& hi, float& lo) {
    float m;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(__uint_as_float(v.x)), "f"(__uint_as_float(v.y)), "f"(__uint_as_float(v.z)));
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(hi) : "f"(hi), "f"(m), "f"(__uint_as_float(v.w)));
    asm("min.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(__uint_as_float(v.x)), "f"(__uint_as_float(v.y)), "f"(__uint_as_float(v.z)));
    asm("min.f32 %0, %1, %2, %3;" : "=f"(lo) : "f"(lo), "f"(m), "f"(__uint_as_float(v.w)));
  }
};
template <> struct LpVec<bf16_t> {
  static __device__ __forceinline__ float2 at(const uint4& v, int j) {
    const uint32_t w = j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  static __device__ __forceinline__ void range(const uint4& v, float& hi, float& lo) {
    uint32_t a, b;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(v.x), "r"(v.y));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(v.z), "r"(v.w));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(hi) : "f"(hi), "f"(__uint_as_float(a << 16)), "f"(__uint_as_float(a & 0xFFFF0000u)));
    asm("min.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(v.x), "r"(v.y));
    asm("min.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(v.z), "r"(v.w));
    asm("min.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
    asm("min.f32 %0, %1, %2, %3;" : "=f"(lo) : "f"(lo), "f"(__uint_as_float(a << 16)), "f"(__uint_as_float(a & 0xFFFF0000u)));
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

// y of a difference of logits; -inf (a masked token, nothing seen yet) stays
// finite, so that 2^y = 0 and 0 y = 0.
__device__ __forceinline__ float lp_y(float diff, float c) { return fmaxf(diff * c, -1e30f); }

// (m, z, zy) += (m2, z2, zy2).
__device__ __forceinline__ void stats_merge(float& m, float& z, float& zy, float m2, float z2, float zy2, float c) {
  const float mm = fmaxf(m, m2), mb = mm == -INFINITY ? 0.f : mm;
  const float da = lp_y(m - mb, c), db = lp_y(m2 - mb, c), a = lp_ex2(da), b = lp_ex2(db);
  zy = fmaf(z, da, zy) * a + fmaf(z2, db, zy2) * b;
  z = z * a + z2 * b;
  m = mm;
}

struct LpShared {
  float m[LP_WARPS], z[LP_WARPS], zy[LP_WARPS];
  int before[LP_WARPS];
  int last;
  u64 pend[LP_WARPS][64];
  u64 list[LP_WARPS][32];
  uint32_t top[LP_WARPS][32];
  uint4 raw[LP_UNROLL][LP_THREADS];              // a step's vectors, for the search of one with candidates
};

// The warps' lists into one, in warp 0's lanes.
template <class K>
__device__ __forceinline__ K block_lists(K list, K (*sh)[32]) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll 1
  for (int h = LP_WARPS / 2; h > 0; h >>= 1) {
    if (w >= h && w < 2 * h) sh[w][lane] = list;
    __syncthreads();
    if (w < h) list = warp_merge(list, sh[w + h][lane]);
  }
  return list;
}

// grid (slices, rows).
template <class T>
__global__ void __launch_bounds__(LP_THREADS, lp_blocks(sizeof(T))) k_logprob(const __grid_constant__ LpArgs A) {
  constexpr int PER = Elt<T>::per16;
  __shared__ LpShared sh;
  const int t = threadIdx.x, lane = t & 31, w = t >> 5, V = A.vocab, n = A.top_n;
  const int r = blockIdx.y, slice = blockIdx.x;
  const T* row = static_cast<const T*>(A.logits) + (int64_t)r * A.ld;
  // the row as aligned vectors: vector i holds elements i PER - skip ..
  const int skip = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
  const int nv = (skip + V + PER - 1) / PER, tiles = (nv + LP_TILE - 1) / LP_TILE;
  const int i0 = (int)((int64_t)tiles * slice / A.slices) * LP_TILE, i1 = (int)((int64_t)tiles * (slice + 1) / A.slices) * LP_TILE;
  const int tok = A.tokens ? A.tokens[r] : -1;
  const bool have = tok >= 0 && tok < V;
  auto load = [&](int i) {
    uint4 v;
    const int e = i * PER - skip;
    if (e >= 0 && e + PER <= V) {
      v = ld_stream(row + e);
    } else {                                     // the row's ends: element by element, -inf outside
      uint32_t x[4];
      for (int u = 0; u < 4; ++u) {
        if (sizeof(T) == 4) {
          x[u] = e + u >= 0 && e + u < V ? reinterpret_cast<const uint32_t*>(row)[e + u] : 0xff800000u;
        } else {
          const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
          const int q = e + 2 * u;
          x[u] = (q >= 0 && q < V ? p[q] : 0xff80u) | ((q + 1 >= 0 && q + 1 < V ? p[q + 1] : 0xff80u) << 16);
        }
      }
      v = make_uint4(x[0], x[1], x[2], x[3]);
    }
    return v;
  };
  uint4 buf[LP_UNROLL];
#pragma unroll
  for (int u = 0; u < LP_UNROLL; ++u) buf[u] = load(i0 + (w * LP_UNROLL + u) * 32 + lane);   // a warp's vectors are consecutive
  const float raw_t = have ? logit<T>(row, tok) : 0.f, key_t = am_key(raw_t);
  // a logit comes before the token if it is larger, or equal at a lower index:
  // x > up in vectors behind the token's (and, but for its ties, in it), x >
  // down, the next value below, in vectors ahead of it
  const int tvec = have ? (tok + skip) / PER : -1;
  const bool low = have && key_t == -INFINITY;             // ties with NaN and -inf: compared one by one
  const float up = have && !low ? key_t : INFINITY, down = have && !low ? nextafterf(key_t, -INFINITY) : INFINITY;
  float m = -INFINITY, mk = -INFINITY;                     // of the statistics; the same with NaN as -inf
  u64 z2 = 0, zy2 = 0;                                     // two zeros
  int before = 0, pending = 0, step = 0;
  bool bad = false;
  u64 list = 0;
  uint32_t bound = 0;                                      // no key below it can be among the block's best n
  const u64 c2 = pair(A.c, A.c);
#pragma unroll 1
  for (int at = i0; at < i1; at += LP_TILE, ++step) {
    const int base = at + w * 32 * LP_UNROLL + lane;
    uint4 cur[LP_UNROLL];
    float bm = -INFINITY, lo = INFINITY;
#pragma unroll
    for (int u = 0; u < LP_UNROLL; ++u) {
      cur[u] = buf[u];
      LpVec<T>::range(cur[u], bm, lo);
    }
    if (at + LP_TILE < i1) {
#pragma unroll
      for (int u = 0; u < LP_UNROLL; ++u) buf[u] = load(base + LP_TILE + 32 * u);
    }
    if (!(bm < INFINITY)) {                                // NaN or +inf: the row's statistics are NaN, its order is not
      bad = true;
      bm = -INFINITY;
#pragma unroll
      for (int u = 0; u < LP_UNROLL; ++u)
#pragma unroll
        for (int j = 0; j < PER / 2; ++j) {
          const float2 x = LpVec<T>::at(cur[u], j);
          bm = fmaxf(bm, fmaxf(am_key(x.x), am_key(x.y)));
        }
    }
    if (bm > m) {
      const float d = lp_y(m - bm, A.c), f = lp_ex2(d);
      const u64 f2 = pair(f, f);
      zy2 = mul2(fma2(z2, pair(d, d), zy2), f2);
      z2 = mul2(z2, f2);
      m = bm;
    }
    const float mb = m == -INFINITY ? 0.f : m;
    const u64 nm2 = pair(-mb, -mb);
    if ((lo - mb) * A.c > -1e30f) {
#pragma unroll
      for (int u = 0; u < LP_UNROLL; ++u)
#pragma unroll
        for (int j = 0; j < PER / 2; ++j) {
          const float2 x = LpVec<T>::at(cur[u], j);
          const u64 y2 = mul2(add2(pair(x.x, x.y), nm2), c2);
          const float2 y = halves(y2);
          const u64 p2 = pair(lp_ex2(y.x), lp_ex2(y.y));
          z2 = add2(z2, p2);
          zy2 = fma2(p2, y2, zy2);
        }
    } else {                                               // masked tokens, or values as far down: y stays finite
#pragma unroll
      for (int u = 0; u < LP_UNROLL; ++u)
#pragma unroll
        for (int j = 0; j < PER / 2; ++j) {
          const float2 x = LpVec<T>::at(cur[u], j);
          const u64 y2 = pair(lp_y(x.x - mb, A.c), lp_y(x.y - mb, A.c));
          const float2 y = halves(y2);
          const u64 p2 = pair(lp_ex2(y.x), lp_ex2(y.y));
          z2 = add2(z2, p2);
          zy2 = fma2(p2, y2, zy2);
        }
    }
    if (bm > down) {                                       // some may come before the token
#pragma unroll
      for (int u = 0; u < LP_UNROLL; ++u) {
        const float lim = base + 32 * u < tvec ? down : up;
#pragma unroll
        for (int j = 0; j < PER / 2; ++j) {
          const float2 x = LpVec<T>::at(cur[u], j);
          before += (x.x > lim) + (x.y > lim);
        }
      }
    }
    if (low) {
#pragma unroll 1
      for (int e = 0; e < LP_UNROLL * PER; ++e) {
        const int v = (base + 32 * (e / PER)) * PER - skip + e % PER;
        if (v >= 0 && v < V) before += logit<T>(row, v) > -INFINITY || v < tok;
      }
    }
    if (n > 0) {
      mk = fmaxf(mk, bm);
      // at steps 1, 2, 4, ..: the n-th largest thread maximum of the block is a
      // bound of its n-th best logit, and a near one
      if ((step & (step + 1)) == 0) {
        const uint32_t k = block_lists(warp_sort(ordered(mk)), sh.top);
        if (w == 0) sh.top[0][lane] = k;
        __syncthreads();
        const uint32_t b = sh.top[0][n - 1];
        bound = bound > b ? bound : b;
        __syncthreads();
      }
      if (__any_sync(0xffffffffu, ordered(bm) >= bound)) {
#pragma unroll
        for (int u = 0; u < LP_UNROLL; ++u) sh.raw[u][t] = cur[u];
#pragma unroll 1
        for (int u = 0; u < LP_UNROLL; ++u) {
          const uint4 v4 = sh.raw[u][t];
          float vm = -INFINITY;
#pragma unroll
          for (int j = 0; j < PER / 2; ++j) {
            const float2 x = LpVec<T>::at(v4, j);
            vm = fmaxf(vm, fmaxf(x.x, x.y));               // NaN as -inf
          }
          if (!__any_sync(0xffffffffu, ordered(vm) >= bound)) continue;
#pragma unroll 1
          for (int e = 0; e < PER; ++e) {
            const int v = (base + 32 * u) * PER - skip + e;
            const u64 k = v >= 0 && v < V ? key_of(logit<T>(reinterpret_cast<const T*>(&sh.raw[u][t]), e), v) : 0;
            const u64 least = __shfl_sync(0xffffffffu, list, n - 1);
            const bool in = k > least && (uint32_t)(k >> 32) >= bound;
            const uint32_t who = __ballot_sync(0xffffffffu, in);
            if (in) sh.pend[w][pending + __popc(who & ((1u << lane) - 1))] = k;
            pending += __popc(who);
            if (pending >= 32) {                           // 32 of them into the list
              __syncwarp();
              const u64 p = sh.pend[w][lane], rest = sh.pend[w][32 + lane];
              __syncwarp();
              sh.pend[w][lane] = rest;
              pending -= 32;
              list = warp_merge(list, warp_sort(p));
              const uint32_t nth = (uint32_t)(__shfl_sync(0xffffffffu, list, n - 1) >> 32);
              bound = bound > nth ? bound : nth;
              __syncwarp();
            }
          }
        }
      }
    }
  }
  if (n > 0 && pending > 0) {
    __syncwarp();
    list = warp_merge(list, warp_sort(lane < pending ? sh.pend[w][lane] : 0));
  }
  const float2 zh = halves(z2), yh = halves(zy2);
  float z = zh.x + zh.y, zy = yh.x + yh.y;
  // ---- the block's statistics and list ----
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), z2 = __shfl_xor_sync(0xffffffffu, z, o),
                zy2 = __shfl_xor_sync(0xffffffffu, zy, o);
    stats_merge(m, z, zy, m2, z2, zy2, A.c);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  if (lane == 0) {
    sh.m[w] = m;
    sh.z[w] = z;
    sh.zy[w] = zy;
    sh.before[w] = before;
  }
  bad = __syncthreads_or(bad) != 0;
  if (n > 0) list = block_lists(list, sh.list);
  if (t == 0) {
    for (int i = 1; i < LP_WARPS; ++i) {
      stats_merge(m, z, zy, sh.m[i], sh.z[i], sh.zy[i], A.c);
      before += sh.before[i];
    }
  }
  if (A.slices > 1) {
    // ---- leave the slice; the row's last block joins them in order ----
    const size_t at = (size_t)r * A.slices;
    if (w == 0) {
      if (n > 0) A.lists[(at + slice) * 32 + lane] = list;
      if (lane == 0) A.stats[at + slice] = LpStats{m, z, zy, before, bad};
    }
    __threadfence();
    __syncthreads();
    if (t == 0) sh.last = atomicAdd(A.arrived + r, 1) == A.slices - 1;
    __syncthreads();
    if (!sh.last) return;
    __threadfence();
    list = 0;
    if (n > 0) {
      for (int i = w; i < A.slices; i += LP_WARPS) list = warp_merge(list, __ldcg(A.lists + (at + i) * 32 + lane));
      list = block_lists(list, sh.list);
    }
    if (t == 0) {
      A.arrived[r] = 0;
      m = -INFINITY;
      z = zy = 0.f;
      before = 0;
      bad = false;
      for (int i = 0; i < A.slices; ++i) {
        const LpStats* s = A.stats + at + i;
        stats_merge(m, z, zy, __ldcg(&s->m), __ldcg(&s->z), __ldcg(&s->zy), A.c);
        before += __ldcg(&s->before);
        bad = bad || __ldcg(&s->bad) != 0;
      }
    }
  }
  if (w != 0) return;
  const float nan = __int_as_float(0x7fc00000), LN2 = 0.6931471805599453f;
  const bool none = bad || m == -INFINITY;
  const float lz = __shfl_sync(0xffffffffu, none ? nan : log2f(z), 0), mm = __shfl_sync(0xffffffffu, m, 0);
  if (lane == 0) {
    if (A.logprob) A.logprob[r] = have ? (raw_t - mm) * A.it - lz * LN2 : nan;
    if (A.entropy) A.entropy[r] = none ? nan : (lz - zy / z) * LN2;
    if (A.rank) {
      if (!low)                                            // ties inside the token's vector
        for (int v = max(0, tvec * PER - skip); v < tok; ++v) before += am_key(logit<T>(row, v)) == key_t;
      A.rank[r] = have ? before + 1 : 0;
    }
  }
  if (lane < n) {
    A.top_ids[(size_t)r * n + lane] = key_index(list);
    A.top_lp[(size_t)r * n + lane] = (key_value(list) - mm) * A.it - lz * LN2;
  }
}

// Slices of a row: as many steps of LP_TILE vectors as a row has at most; the
// count that gives the least (waves of blocks) x (steps of a slice + 2), two
// steps being about what a block spends on its end (measured: one row block's
// end takes some 1.5 us, a step of 16 KB at a quarter of an SM's share 0.8 us).
int lp_slices(int n_rows, int vocab, int esz) {
  const int resident = lp_blocks(esz) * 152;
  const int64_t tiles = ((int64_t)vocab * esz + 15 + LP_TILE * 16 - 1) / (LP_TILE * 16);
  int best = 1;
  int64_t cost = INT64_MAX;
  const int most = n_rows > LP_COUNTERS ? 1 : (int)std::min<int64_t>(tiles, LP_MAX_SLICES);
  for (int s = 1; s <= most; ++s) {
    const int64_t waves = ((int64_t)n_rows * s + resident - 1) / resident, c = waves * ((tiles + s - 1) / s + 2);
    if (c < cost) { cost = c; best = s; }
  }
  return best;
}

// The counters come first and keep their place, so that calls of other shapes
// on the same workspace find them at zero.
struct LpWs {
  static constexpr size_t stats = LP_COUNTERS * sizeof(int);
  size_t lists, total;
  LpWs(int n_rows, int slices) {
    const size_t parts = slices > 1 ? (size_t)n_rows * slices : 0;
    lists = (stats + parts * sizeof(LpStats) + 15) / 16 * 16;
    total = lists + parts * 32 * sizeof(u64);
  }
};

}  // namespace
}  // namespace spec

using namespace spec;

extern "C" int64_t spec_token_logprobs_ws_bytes(int n_rows, int vocab, int top_n) {
  if (n_rows < 1 || n_rows > 65535 || vocab < 1 || top_n < 0 || top_n > LP_TOP || top_n > vocab)
    return set_last_error(SPEC_ERR_ARG, "1 <= n_rows <= 65535, vocab >= 1 and 0 <= top_n <= min(32, vocab) required");
  if (vocab > LP_MAX_VOCAB) return set_last_error(SPEC_ERR_UNSUPPORTED, "vocab above 1048576");
  return (int64_t)std::max(LpWs(n_rows, lp_slices(n_rows, vocab, 4)).total, LpWs(n_rows, lp_slices(n_rows, vocab, 2)).total);
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
  const int slices = lp_slices(n_rows, vocab, esz);
  const LpWs ws(n_rows, slices);
  char* w = static_cast<char*>(ws_dev);
  const LpArgs A{logits_dev, ld, n_rows, vocab, top_n, slices, tokens_dev, 1.f / temperature, c, out_logprob_dev, out_entropy_dev,
                 out_rank_dev, out_top_ids_dev, out_top_logprobs_dev, reinterpret_cast<int*>(w),
                 reinterpret_cast<LpStats*>(w + ws.stats), reinterpret_cast<u64*>(w + ws.lists)};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
  if (dtype == SPEC_F32) k_logprob<float><<<dim3(slices, n_rows), LP_THREADS, 0, st>>>(A);
  else k_logprob<bf16_t><<<dim3(slices, n_rows), LP_THREADS, 0, st>>>(A);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SPEC_OK : set_last_error(SPEC_ERR_CUDA, cudaGetErrorString(e));
}
