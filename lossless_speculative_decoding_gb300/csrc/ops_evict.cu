// Kernel-level entry point: eviction of cache positions by accumulated attention
// weight, each (layer, kv head) for itself.
//
// k_evict_select, one block per (layer, sequence, head): the budget - recent
// largest masses by radix selection. A mass becomes a key that orders as it does
// (sign folded, NaN lowest); three passes of 11, 11 and 10 bits each count the keys
// that share the digits found so far and fix one more digit of the threshold, the
// smallest key that is kept. One more pass writes what is kept in order of
// position: every key above the threshold, the first ones equal to it, the
// `recent` last positions.
//
// k_evict_move, blocks per (plane, K | V, piece of a row): slot j <- slot kept[j] >=
// j. Rows come to shared memory in batches, a few batches ahead, and a batch is stored
// when all of it is there. Batches on their way read from kept[j'] >= j' past every
// slot that earlier ones are stored to, and rows that stay are not touched.
//
// Bound: HBM, by the rows moved. Measured, L2 cold: 36 layers x 2 x 8 heads of 3,288
// and 5,288 positions to 2,048, 1.2 GB read and written: 232 us, 0.79 of the copy rate
// (the selection 33, the rows 185: reads and writes of HBM in turn); 12 layers x 10 heads
// of 1,357 to 1,024 40 us (11, 26). Keys in registers, where two blocks fit an SM: the
// selection 42 and 13 us.
#include <cuda_runtime.h>

#include <algorithm>

#include "chunk.cuh"

namespace spec {
namespace {

constexpr int EV_THREADS = 512;
constexpr int EV_KEYS = 8192;                    // keys held in shared memory; of longer sequences they are read again
constexpr int EV_BLOCKS = 4;                     // on an SM
constexpr int EV_BINS = 2048;
constexpr int MV_THREADS = 256;
constexpr int MV_ROWS = 4;                       // pieces of a batch for each thread
// Batches in shared memory and blocks on an SM: 4 and 3, or 3 and 4 where there are
// blocks enough: 576 planes of 2,048 rows 245 us with 4 and 3, 233 with 3 and 4; 120 of
// 1,024 rows 42 and 46.5 (fewer columns a block, 46 and 264).
template <int STAGES>
struct MvShape {
  static constexpr int BLOCKS = STAGES == 3 ? 4 : 3, SMEM = STAGES * MV_ROWS * MV_THREADS * 16;
};

struct EvictArgs {
  spec_kv_view kv;
  const int32_t* cache_len;
  const float* mass;
  float* out_mass;
  int32_t* kept;
  int32_t* out_len;
  int32_t* err;
  long long ld;
  int n_seq, budget, recent, capacity;
};

__device__ __forceinline__ uint32_t mass_key(float x) {
  if (x != x) return 0;
  const uint32_t b = __float_as_uint(x + 0.f);   // (one zero)
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Sum of the last lanes' v of the warps before this one.
__device__ __forceinline__ int warps_before(int v, int* red) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  __syncthreads();
  if (lane == 31) red[w] = v;
  __syncthreads();
  int before = lane < w ? red[lane] : 0;         // (no more warps than lanes)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  return before;
}

__global__ void __launch_bounds__(EV_THREADS, EV_BLOCKS) k_evict_select(const __grid_constant__ EvictArgs A) {
  __shared__ int hist[EV_BINS];
  __shared__ uint32_t keys[EV_KEYS];             // (a thread's own)
  __shared__ int red[EV_THREADS / 32];
  __shared__ uint32_t s_digit;
  __shared__ int s_left;
  const int t = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  // planes [layer][sequence][head]
  const int plane = blockIdx.x, s = plane / A.kv.n_kv_heads % A.n_seq;
  const int n = A.cache_len[s];
  const int32_t* bt = A.kv.block_table_dev + (size_t)s * A.kv.max_pages;
  const float* mass = A.mass + (size_t)plane * A.ld;
  float* out_mass = A.out_mass + (size_t)plane * A.ld;
  int32_t* kept = A.kept + (size_t)plane * A.budget;
  const bool first = plane < A.kv.n_kv_heads * A.n_seq && plane % A.kv.n_kv_heads == 0;
  bool ok = n >= 0 && n <= A.capacity;
  if (!ok && first && t == 0) atomicOr(A.err, DERR_POS);
  if (ok && n > A.budget) {
    // every page up to n: the sequence moves in all planes or in none
    bool bad = false;
    for (int i = t; i < (n + A.kv.page_size - 1) / A.kv.page_size; i += EV_THREADS)
      bad |= bt[i] < 0 || bt[i] >= A.kv.n_pages;
    if (__syncthreads_or(bad)) {
      ok = false;
      if (first && t == 0) atomicOr(A.err, DERR_PAGE);
    }
  }
  if (first && t == 0) A.out_len[s] = ok ? min(n, A.budget) : n;
  if (!ok || n <= A.budget) {
    for (int j = t; j < A.budget; j += EV_THREADS) kept[j] = ok && j < n ? j : -1;
    if (ok)
      for (int j = t; j < n; j += EV_THREADS) out_mass[j] = mass[j];
    return;
  }
  const int old = n - A.recent;                  // positions that compete
  // warp w has positions w len .. , 32 at a time
  const int lane = t & 31, w = t >> 5, len = (n + EV_THREADS - 1) / EV_THREADS * 32, w0 = w * len;
  const bool hold = len * (EV_THREADS / 32) <= EV_KEYS;
  if (hold) {
#pragma unroll 4
    for (int i = w0 + lane; i < w0 + len; i += 32) keys[i] = i < old ? mass_key(mass[i]) : 0u;
  }
  // f(position, key) for this thread's positions, all of a warp's lanes together (i may be n or more)
  auto each = [&](auto&& f) {
    if (hold) {
#pragma unroll 4
      for (int i = w0 + lane; i < w0 + len; i += 32) f(i, keys[i]);
    } else {
      for (int i = w0 + lane; i < w0 + len; i += 32) f(i, i < old ? mass_key(mass[i]) : 0u);
    }
  };
  int left = A.budget - A.recent;                // of them to be kept; those equal to the threshold at last
  uint32_t key = 0, known = 0;                   // the threshold's digits so far, their bits
  if (left > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
      for (int i = t; i < EV_BINS; i += EV_THREADS) hist[i] = 0;
      __syncthreads();
      each([&](int i, uint32_t x) {
        if (i < old && (x & known) == key) atomicAdd(&hist[(x >> shift) & (bins - 1)], 1);
      });
      __syncthreads();
      // bins from the top: thread t has bins top - 4 t ..; the digit is where the count reaches `left`
      constexpr int PER = EV_BINS / EV_THREADS;
      int c[PER], sum = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        c[i] = hist[EV_BINS - 1 - (t * PER + i)];
        sum += c[i];
      }
      int inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      int above = warps_before(inc, red) + inc - sum;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (above < left && above + c[i] >= left) {
          s_digit = EV_BINS - 1 - (t * PER + i);
          s_left = left - above;
        }
        above += c[i];
      }
      __syncthreads();
      key |= s_digit << shift;
      known |= (uint32_t)(bins - 1) << shift;
      left = s_left;
    }
  }
  // kept positions in order: above the threshold, the first `left` equal to it, the last `recent`
  const bool any = A.budget > A.recent;
  auto is_above = [&](int i, uint32_t x) { return i < n && (i >= old || (any && x > key)); };
  auto is_equal = [&](int i, uint32_t x) { return i < old && any && x == key; };
  int up = 0, eq = 0;
  each([&](int i, uint32_t x) {
    up += __popc(__ballot_sync(0xffffffffu, is_above(i, x)));
    eq += __popc(__ballot_sync(0xffffffffu, is_equal(i, x)));
  });
  up = warps_before(up, red);
  eq = warps_before(eq, red);
  const uint32_t lower = (1u << lane) - 1;
  each([&](int i, uint32_t x) {
    const uint32_t a = __ballot_sync(0xffffffffu, is_above(i, x)), e = __ballot_sync(0xffffffffu, is_equal(i, x));
    const int me = eq + __popc(e & lower);       // equal ones before this position
    if ((a >> lane & 1) || ((e >> lane & 1) && me < left)) {
      const int j = up + __popc(a & lower) + min(me, left);
      kept[j] = i;
      out_mass[j] = mass[i];
    }
    up += __popc(a);
    eq += __popc(e);
  });
}

// n / d for 0 <= n < 2^31, 1 <= d <= 2^30: with 2^s >= d and f = ceil(2^(31 + s) / d), f d
// is above 2^(31 + s) by less than 2^s, so n f / 2^(31 + s) is above n / d by less than 1 / d.
struct FastDiv {
  uint32_t d, f, s;
  explicit FastDiv(uint32_t by) : d(by), s(0) {
    while ((1u << s) < by) ++s;
    f = (uint32_t)(((1ull << (31 + s)) + by - 1) / by);
  }
  __device__ int div(int n) const { return (int)((uint64_t)(uint32_t)n * f >> (31 + s)); }
};

__device__ __forceinline__ void cp_async16(uint32_t smem, const void* gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(gmem) : "memory");
}

// grid (planes x pieces of a row, K | V); SPAN 16-byte columns a block.
template <int SPAN, int STAGES>
__global__ void __launch_bounds__(MV_THREADS, MvShape<STAGES>::BLOCKS) k_evict_move(const __grid_constant__ EvictArgs A, int row16, FastDiv P) {
  constexpr int ROWS = MV_THREADS / SPAN, BATCH = ROWS * MV_ROWS;        // rows of the block at once, of a batch
  extern __shared__ uint4 mv_stage[];
  const int t = threadIdx.x, r = t / SPAN, cols = row16 / SPAN;
  pdl_wait();
  pdl_trigger();
  const int plane = blockIdx.x / cols, c = blockIdx.x % cols * SPAN + t % SPAN;
  const int h = plane % A.kv.n_kv_heads, s = plane / A.kv.n_kv_heads % A.n_seq, layer = plane / A.kv.n_kv_heads / A.n_seq;
  const int n = A.cache_len[s];
  if (n <= A.budget || n > A.capacity) return;
  const int32_t* kept = A.kept + (size_t)plane * A.budget;
  if (kept[A.budget - 1] < 0) return;            // (a bad page)
  const int32_t* bt = A.kv.block_table_dev + (size_t)s * A.kv.max_pages;
  const size_t page16 = (size_t)A.kv.n_layers * A.kv.n_kv_heads * 2 * P.d * row16;
  uint4* base = static_cast<uint4*>(A.kv.kv_dev) + (((size_t)layer * A.kv.n_kv_heads + h) * 2 + blockIdx.y) * P.d * row16 + c;
  auto at = [&](int pos) {
    const int page = P.div(pos);
    return base + bt[page] * page16 + (size_t)(pos - page * (int)P.d) * row16;
  };
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(mv_stage + t);
  const int batches = (A.budget + BATCH - 1) / BATCH;
  int from[MV_ROWS];                             // old slots of the next batch to be asked for (the slot itself: nothing to move)
  auto look = [&](int b) {
#pragma unroll
    for (int u = 0; u < MV_ROWS; ++u) {
      const int j = b * BATCH + u * ROWS + r;
      from[u] = j < A.budget ? kept[j] : j;
    }
  };
  uint32_t moves = 0;                            // MV_ROWS bits for each batch on its way, the newest lowest
  auto ask = [&](int b) {
    moves <<= MV_ROWS;
    if (b < batches) {
#pragma unroll
      for (int u = 0; u < MV_ROWS; ++u)
        if (from[u] > b * BATCH + u * ROWS + r) {
          moves |= 1u << u;
          cp_async16(mine + (b % STAGES * MV_ROWS + u) * MV_THREADS * 16, at(from[u]));
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    look(b + 1);
  };
  look(0);
#pragma unroll 1
  for (int b = 0; b < STAGES - 1; ++b) ask(b);
#pragma unroll 1
  for (int b = 0; b < batches; ++b) {
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
    __syncthreads();                             // the whole batch is there, and nobody asks for more of it
    const uint32_t bits = moves >> (MV_ROWS * (STAGES - 2));
#pragma unroll
    for (int u = 0; u < MV_ROWS; ++u)
      if (bits >> u & 1) *at(b * BATCH + u * ROWS + r) = mv_stage[(b % STAGES * MV_ROWS + u) * MV_THREADS + t];
    ask(b + STAGES - 1);
  }
}

template <int SPAN, int STAGES>
cudaError_t launch_move(const EvictArgs& A, int64_t blocks, int row16, cudaStream_t st) {
  cudaError_t e = allow_dyn_smem_once<k_evict_move<SPAN, STAGES>>();
  if (e != cudaSuccess) return e;
  return launch_k(k_evict_move<SPAN, STAGES>, dim3((unsigned)blocks, 2), dim3(MV_THREADS), MvShape<STAGES>::SMEM, st, A, row16,
                  FastDiv(A.kv.page_size));
}

}  // namespace
}  // namespace spec

using namespace spec;

extern "C" int spec_kv_evict(const spec_kv_view* kv, int n_seq, const int32_t* cache_len_dev, const float* mass_dev, int64_t ld,
                             int budget, int recent, float* out_mass_dev, int32_t* out_kept_dev, int32_t* out_len_dev,
                             int32_t* err_dev, uintptr_t cuda_stream) {
  const int rc = check_chunks(kv, n_seq, kv ? kv->n_kv_heads : 0);
  if (rc) return rc;
  if (!cache_len_dev || !mass_dev || !out_mass_dev || !out_kept_dev || !out_len_dev || !err_dev)
    return set_last_error(SPEC_ERR_ARG, "null pointer argument");
  if (budget < 1 || recent < 0 || recent > budget) return set_last_error(SPEC_ERR_ARG, "1 <= budget and 0 <= recent <= budget required");
  if (budget > (1 << 30)) return set_last_error(SPEC_ERR_UNSUPPORTED, "budget above 2^30");   // (nor is a sequence longer)
  if (ld < 1 || ld > ((int64_t)1 << 31)) return set_last_error(SPEC_ERR_ARG, "1 <= ld <= 2^31 required");
  const int64_t planes = (int64_t)kv->n_layers * n_seq * kv->n_kv_heads;
  const int row16 = kv->head_dim * (kv->dtype == SPEC_F32 ? 4 : 2) / 16;
  if (planes * row16 > 0x7fffffff) return set_last_error(SPEC_ERR_UNSUPPORTED, "too many (layer, sequence, head) planes");
  struct Span { const void* p; int64_t n; };
  const Span out[4] = {{out_mass_dev, planes * ld * 4}, {out_kept_dev, planes * budget * 4}, {out_len_dev, (int64_t)n_seq * 4},
                       {kv->kv_dev, cache_bytes(*kv)}};
  const Span in[3] = {{cache_len_dev, (int64_t)n_seq * 4}, {mass_dev, planes * ld * 4},
                      {kv->block_table_dev, (int64_t)n_seq * kv->max_pages * 4}};
  for (int i = 0; i < 4; ++i) {
    for (const Span& b : in)
      if (spans_meet(out[i].p, out[i].n, b.p, b.n)) return set_last_error(SPEC_ERR_ARG, "an output overlaps an input");
    for (int j = 0; j < i; ++j)
      if (spans_meet(out[i].p, out[i].n, out[j].p, out[j].n)) return set_last_error(SPEC_ERR_ARG, "two outputs overlap");
  }
  const int sms = sm_count_once();
  if (sms < 1) return set_last_error(SPEC_ERR_CUDA, "no device");
  const EvictArgs A{*kv, cache_len_dev, mass_dev, out_mass_dev, out_kept_dev, out_len_dev, err_dev, ld, n_seq, budget, recent,
                    (int)std::min<int64_t>(ld, (int64_t)kv->max_pages * kv->page_size)};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
  cudaError_t e = launch_k(k_evict_select, dim3((unsigned)planes), dim3(EV_THREADS), 0, st, A);
  const int span = row16 % 16 ? 8 : 16;
  const int64_t blocks = planes * (row16 / span);
  const bool many = 2 * blocks >= 4 * (int64_t)sms;
  if (e == cudaSuccess && span == 8) e = many ? launch_move<8, 3>(A, blocks, row16, st) : launch_move<8, 4>(A, blocks, row16, st);
  else if (e == cudaSuccess) e = many ? launch_move<16, 3>(A, blocks, row16, st) : launch_move<16, 4>(A, blocks, row16, st);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? SPEC_OK : set_last_error(SPEC_ERR_CUDA, cudaGetErrorString(e));
}
