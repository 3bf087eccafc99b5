// Kernel-level entry point: log probabilities of given tokens, with entropy,
// rank and the likeliest alternatives, from materialised logits.
//
// With x = logits / T and m = max x: z = sum e^(x - m), log p(t) = x_t - m -
// log z, entropy = log z - sum e^(x - m) (x - m) / z (two terms of one sign:
// no cancellation). The order of tokens is (logit descending, index
// ascending), NaN as -inf.
#include <cuda_runtime.h>

#include <algorithm>

#include "kv_view.cuh"

namespace spec {
namespace {

constexpr int LP_THREADS = 512;
constexpr int LP_MAX_VOCAB = 1 << 20;

struct LpArgs {
  const void* logits;
  int64_t ld;
  int n_rows, vocab, top_n;
  const int32_t* tokens;
  float it;                 // 1 / temperature
  float* logprob;
  float* entropy;
  int32_t* rank;
  int32_t* top_ids;
  float* top_lp;
};

template <class T> __device__ __forceinline__ float logit(const T* row, int v);
template <> __device__ __forceinline__ float logit<float>(const float* row, int v) { return row[v]; }
template <> __device__ __forceinline__ float logit<bf16_t>(const bf16_t* row, int v) { return bf16_to_f(row[v].v); }

// (value, index) order: larger first, then the lower index.
__device__ __forceinline__ bool before(float a, int ia, float b, int ib) { return a > b || (a == b && ia < ib); }

// One block per row: a pass for the maximum, one for the sums, one per
// alternative.
template <class T>
__global__ void __launch_bounds__(LP_THREADS) k_logprob(LpArgs A) {
  __shared__ float red[32];
  __shared__ float bv[LP_THREADS / 32];
  __shared__ int bi[LP_THREADS / 32];
  const int t = threadIdx.x, lane = t & 31, w = t >> 5, V = A.vocab;
  for (int r = blockIdx.x; r < A.n_rows; r += gridDim.x) {
    const T* row = static_cast<const T*>(A.logits) + (int64_t)r * A.ld;
    float pv = INFINITY, m = 0.f, lse = 0.f;
    int pi = -1;
    const int tok = A.tokens ? A.tokens[r] : -1;
    const bool have = tok >= 0 && tok < V;
    const float raw_t = have ? logit<T>(row, tok) : 0.f, key_t = am_key(raw_t);
    auto best_after = [&](float v0, int i0) {    // the first (value, index) after (v0, i0) in the order
      float v = -INFINITY;
      int i = V;
      for (int c = t; c < V; c += LP_THREADS) {
        const float x = am_key(logit<T>(row, c));
        if (before(v0, i0, x, c) && before(x, c, v, i)) { v = x; i = c; }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float v2 = __shfl_xor_sync(0xffffffffu, v, o);
        const int i2 = __shfl_xor_sync(0xffffffffu, i, o);
        if (before(v2, i2, v, i)) { v = v2; i = i2; }
      }
      __syncthreads();
      if (lane == 0) { bv[w] = v; bi[w] = i; }
      __syncthreads();
      pv = bv[0];
      pi = bi[0];
      for (int j = 1; j < LP_THREADS / 32; ++j)
        if (before(bv[j], bi[j], pv, pi)) { pv = bv[j]; pi = bi[j]; }
    };
    best_after(INFINITY, -1);
    m = pv * A.it;
    float z = 0.f, zx = 0.f;
    bool odd = false;                            // a NaN or +inf logit
    int n_before = 0;
    for (int c = t; c < V; c += LP_THREADS) {
      const float x = logit<T>(row, c), y = x * A.it - m, e = expf(y);
      odd = odd || !(x < INFINITY);
      z += e;
      if (e > 0.f) zx += e * y;
      if (have && before(am_key(x), c, key_t, tok)) ++n_before;
    }
    z = block_sum(z, red);
    zx = block_sum(zx, red);
    int nb = n_before;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) nb += __shfl_xor_sync(0xffffffffu, nb, o);
    if (lane == 0) bi[w] = nb;
    const bool bad = __syncthreads_or(odd) != 0 || pv == -INFINITY;
    nb = 0;
    for (int j = 0; j < LP_THREADS / 32; ++j) nb += bi[j];
    const float nan = __int_as_float(0x7fc00000);
    const float lz = logf(z);
    lse = bad ? nan : lz;
    __syncthreads();
    if (t == 0) {
      if (A.logprob) A.logprob[r] = have ? (raw_t * A.it - m) - lse : nan;
      if (A.rank) A.rank[r] = have ? nb + 1 : 0;
      if (A.entropy) A.entropy[r] = bad ? nan : lz - zx / z;
    }
    for (int j = 0; j < A.top_n; ++j) {
      if (t == 0) {
        A.top_ids[(size_t)r * A.top_n + j] = pi;
        A.top_lp[(size_t)r * A.top_n + j] = (pv * A.it - m) - lse;
      }
      if (j + 1 < A.top_n) best_after(pv, pi);
    }
  }
}

}  // namespace
}  // namespace spec

using namespace spec;

extern "C" int64_t spec_token_logprobs_ws_bytes(int n_rows, int vocab, int top_n) {
  if (n_rows < 1 || vocab < 1 || top_n < 0 || top_n > SPEC_LOGPROB_MAX_TOP || top_n > vocab)
    return set_last_error(SPEC_ERR_ARG, "n_rows >= 1, vocab >= 1 and 0 <= top_n <= min(32, vocab) required");
  return 16;
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
  if (vocab > LP_MAX_VOCAB) return set_last_error(SPEC_ERR_UNSUPPORTED, "vocab above 1048576");
  if (ld < vocab) return set_last_error(SPEC_ERR_ARG, "ld below vocab");
  if (!(temperature > 0.f) || !(1.f / temperature < INFINITY) || !(1.f / temperature > 0.f))
    return set_last_error(SPEC_ERR_ARG, "temperature must be positive");
  if (reinterpret_cast<uintptr_t>(logits_dev) % (dtype == SPEC_F32 ? 4 : 2) || !aligned16(ws_dev))
    return set_last_error(SPEC_ERR_ARG, "misaligned logits or workspace");
  if ((int64_t)ws_bytes < need) return set_last_error(SPEC_ERR_ARG, "workspace too small");
  const LpArgs A{logits_dev, ld, n_rows, vocab, top_n, tokens_dev, 1.f / temperature, out_logprob_dev,
                 out_entropy_dev, out_rank_dev, out_top_ids_dev, out_top_logprobs_dev};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
  const int blocks = std::min(n_rows, 65535);
  if (dtype == SPEC_F32) k_logprob<float><<<blocks, LP_THREADS, 0, st>>>(A);
  else k_logprob<bf16_t><<<blocks, LP_THREADS, 0, st>>>(A);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SPEC_OK : set_last_error(SPEC_ERR_CUDA, cudaGetErrorString(e));
}
