// Kernel-level entry point: the attention weight that each cached position draws
// from a chunk of new tokens.
//
// With lse the log of a row's sum of exponentials, a position's share of the row is
// exp(scale q.K_j - lse): no second pass over the row is needed, and the sum over
// rows stays with the position. A unit is (sequence, tile of keys, kv head): it
// brings its keys once, goes over the counted rows that see them, and writes its
// positions alone, so nothing is summed by atomics. Units of a sequence are
// numbered from its first keys on, which the most rows see; block b takes units b,
// b + B, ..
#include <cuda_runtime.h>

#include <algorithm>

#include "chunk.cuh"
#include "tc_attn.cuh"

namespace spec {
namespace {

constexpr int MS_MAX_G = 128;                    // query heads per kv head

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
  float scale_l2e;     // scale * log2 e
};

// Unit: key tile `tile` of (sequence s, kv head hk), its rows from token i0 on.
struct MassUnit {
  int s, tile, hk;
  int n, m, r0, i0;
};

// A warp's walk over the units first, first + step, .. .
template <int KEYS>
struct MassWalk {
  long long u, before;                           // next unit; units before sequence s
  int s;
  const MassArgs* A;
  __device__ MassWalk(const MassArgs& args, long long first) : u(first), before(0), s(0), A(&args) {}
  __device__ static int tiles(int n, int m) { return (n + m + KEYS - 1) / KEYS; }
  __device__ bool next(MassUnit& g, int step) {
    const int lane = threadIdx.x & 31, hkv = A->kv.n_kv_heads;
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
    u += step;
    return true;
  }
};

// ---------------------------------------------------------------------------
// FMA form. 128 threads, 64 keys, 32 rows at a time, fp32. Thread (ty, tx) = (t / 16,
// t % 16) has rows 4 ty .. 4 ty + 3 and keys tx + 16 j of the score product.
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
  MassWalk<MF_KEYS> walk(A, blockIdx.x);
  MassUnit g;
  while (walk.next(g, gridDim.x)) {
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
      if (page >= 0) kk = load4<KT>(A.kv.kv_dev, page * page_elems + plane + (size_t)((k0 + key) % P) * D + c);
      *reinterpret_cast<float4*>(&sm.k[key][c]) = kk;
    }
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    const int end = g.m * A.G;
    for (int r0 = max(g.i0, 0) * A.G; r0 < end; r0 += MF_ROWS) {
      __syncthreads();
      for (int i = t; i < MF_ROWS * (D / 4); i += MF_THREADS) {
        const int r = i / (D / 4), c = 4 * (i % (D / 4)), rr = r0 + r;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (rr < end) {
          const size_t row = ((size_t)g.r0 + rr / A.G) * A.hq + g.hk * A.G + rr % A.G;
          v = load4<KT>(A.q, row * D + c);
          v = make_float4(v.x * A.scale_l2e, v.y * A.scale_l2e, v.z * A.scale_l2e, v.w * A.scale_l2e);
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
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rr = r0 + 4 * ty + i;
        if (rr >= end) continue;
        const float lse = sm.lse[4 * ty + i];
        const int seen = g.n + rr / A.G + 1 - k0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (tx + 16 * j < seen) sum[j] += exp2f(x[i][j] - lse);
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) sm.sum[ty][tx + 16 * j] = sum[j];
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

template <int D, class KT>
cudaError_t launch_mass_fma(const MassArgs& A, int blocks, cudaStream_t st) {
  cudaError_t e = allow_dyn_smem_once<k_mass_fma<KT, D>>();
  return e == cudaSuccess ? launch_k(k_mass_fma<KT, D>, dim3(blocks), dim3(MF_THREADS), sizeof(MfSmem<D>), st, A) : e;
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
  if (ld < 1 || ld > ((int64_t)1 << 31)) return set_last_error(SPEC_ERR_ARG, "1 <= ld <= 2^31 required");
  const int64_t capacity = std::min<int64_t>((int64_t)kv->max_pages * kv->page_size, ld);
  // a sequence's units, and its rows of a kv head, are counted in 32 bits
  if ((double)capacity / MF_KEYS * kv->n_kv_heads > 2e9 || (double)std::min<int64_t>(max_new, capacity) * (n_q_heads / kv->n_kv_heads) > 2e9)
    return set_last_error(SPEC_ERR_UNSUPPORTED, "block table too long for this many heads");
  const int64_t mbytes = (int64_t)n_seq * kv->n_kv_heads * ld * 4;
  if (out_mass_dev != mass_dev && spans_meet(out_mass_dev, mbytes, mass_dev, mbytes))
    return set_last_error(SPEC_ERR_ARG, "out_mass overlaps mass without being the same array");
  const int sms = sm_count_once();
  if (sms < 1) return set_last_error(SPEC_ERR_CUDA, "no device");
  const int d = kv->head_dim;
  const MassArgs A{*kv, ChunkIndex{row_start_dev, n_new_dev, cache_len_dev, n_seq, n_rows, max_new, (int)capacity}, q_dev, lse_dev,
                   mass_dev, out_mass_dev, err_dev, ld, layer, n_q_heads, n_q_heads / kv->n_kv_heads, last, scale * LOG2E};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
  const int blocks = 3 * sms;
  cudaError_t e;
  if (kv->dtype == SPEC_F32) e = d == 128 ? launch_mass_fma<128, float>(A, blocks, st) : launch_mass_fma<64, float>(A, blocks, st);
  else e = d == 128 ? launch_mass_fma<128, bf16_t>(A, blocks, st) : launch_mass_fma<64, bf16_t>(A, blocks, st);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? SPEC_OK : set_last_error(SPEC_ERR_CUDA, cudaGetErrorString(e));
}
