// Kernel-level entry point: norm and rotation of new tokens' queries and keys, and
// the way of their keys and values into the paged cache.
//
// A head of d values lies on LPH = d / (16 bytes) lanes, one 16-byte piece each,
// so that a warp holds one to four heads of a row. A block takes 8 tokens at a time:
// their places, the cosines and sines of their angles into shared memory, then the
// heads, up to four of a lane's on their way at once. A lane's piece is the same in every
// head, so what it is multiplied by is made once for them: with gamma folded
// in, y[i] = r (x[i] C[i] + x'[i] S[i]), x' the partner's piece (a shuffle), r =
// 1 / sqrt(mean x^2 + eps), C = gamma cos, S = -+ gamma' sin. Pieces behind the rotated
// dims have C = gamma, S = 0.
//
// The angle of position p is p F of a 64-bit turn, F = freq / 2 pi in units of
// 2^-64 of a turn: the product wraps as the angle does, so it is as exact at
// position 2^31 as at 1. Its upper 32 bits, reduced to an eighth of a turn either
// way, go to sincospif.
//
// Bound: HBM, by the bytes of the rows.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "chunk.cuh"
#include "tc_attn.cuh"

namespace spec {
namespace {

constexpr int RP_THREADS = 256;
constexpr int RP_TOKENS = 8;                     // tokens of a block at a time
constexpr int RP_FLY = 4;                        // heads a lane has in flight
constexpr int RP_BLOCKS = 4;                     // on an SM

struct RopeArgs {
  spec_kv_view kv;
  ChunkIndex ix;
  const char* qkv;
  char* q_out;
  const int32_t* positions;
  const float* gamma[2];                         // of queries, of keys
  int32_t* err;
  long long ld;                                  // bytes of a row
  int layer, hq, half8;                          // half8: rotated pairs / values of a piece
  int chunks[2], heads[2];                       // of queries, of keys (and values): lane groups that share a token's, heads of each
  float eps;
  uint64_t turn[SPEC_ROPE_MAX_PAIRS];            // freq in 2^-64 turns
  uint8_t axis[SPEC_ROPE_MAX_PAIRS];
};

// cos and sin of a turn's 2^-32 parts.
__device__ __forceinline__ void turn_cos_sin(uint32_t a, float& c, float& s) {
  const uint32_t quarter = (a + 0x20000000u) >> 30;
  const int rest = (int)(a - (quarter << 30));   // [-1/8, 1/8) of a turn
  float s0, c0;
  sincospif((float)rest * 4.656612873077393e-10f, &s0, &c0);   // 2^-31: half turns
  const float x = quarter & 1 ? s0 : c0, y = quarter & 1 ? c0 : s0;
  c = (quarter == 1 || quarter == 2) ? -x : x;
  s = quarter >= 2 ? -y : y;
}

template <int NV>
__device__ __forceinline__ uint4 pack_piece(const float (&y)[NV]) {
  uint4 r;
  uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (NV == 4) w[i] = __float_as_uint(y[i]);
    else w[i] = pack_bf16(y[2 * i], y[2 * i + 1]);
  }
  return r;
}

// Pairs of a piece's values.
template <class KT>
__device__ __forceinline__ void unpack2(const uint4& v, unsigned long long (&f)[Elt<KT>::per16 / 2]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (Elt<KT>::per16 == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) f[i] = pair(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
}

template <class KT, int D>
__global__ void __launch_bounds__(RP_THREADS, RP_BLOCKS) k_qk_norm_rope(const __grid_constant__ RopeArgs A) {
  constexpr int NV = Elt<KT>::per16, N2 = NV / 2, LPH = D / NV, GROUPS = RP_THREADS / LPH;
  __shared__ long long w_sum[RP_THREADS / 32];
  __shared__ int t_seq[RP_TOKENS], t_row[RP_TOKENS], t_pos[RP_TOKENS], t_page[RP_TOKENS];
  __shared__ __align__(16) float t_cos[RP_TOKENS][D / 2], t_sin[RP_TOKENS][D / 2], gam[2][D];
  const int t = threadIdx.x, lane = t & 31, w = t >> 5;
  pdl_wait();
  pdl_trigger();

  for (int i = t; i < 2 * D; i += RP_THREADS) {
    const float* gm = A.gamma[i / D];
    gam[i / D][i % D] = gm ? gm[i % D] : 1.f;
  }
  // this thread's sequences, the tokens before them and of them
  const int per = (A.ix.n_seq + RP_THREADS - 1) / RP_THREADS;
  const int a = min(t * per, A.ix.n_seq), a1 = min(a + per, A.ix.n_seq);
  long long sum = 0;
  for (int i = a; i < a1; ++i) {
    const ChunkSeq z(A.ix, i);
    if (z.bad && blockIdx.x == 0) atomicOr(A.err, DERR_POS);
    sum += z.m;
  }
  long long inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) w_sum[w] = inc;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < RP_THREADS / 32; ++i) {
    if (i < w) before += w_sum[i];
    total += w_sum[i];
  }
  before += inc - sum;
  // this block's tokens: [c T / B, (c + 1) T / B) of all T
  const long long blocks = gridDim.x, blk = blockIdx.x;
  const long long k0 = total / blocks * blk + total % blocks * blk / blocks;
  const long long k1 = total / blocks * (blk + 1) + total % blocks * (blk + 1) / blocks;

  const int g = t / LPH, gl = t % LPH;
  const uint32_t gmask = LPH == 32 ? 0xffffffffu : ((1u << (LPH & 31)) - 1) << (lane / LPH * LPH);
  const int half = A.half8 * NV, rotated = 2 * A.half8;
  const bool low = gl < A.half8, turns = gl < rotated;
  const int partner = low ? gl + A.half8 : turns ? gl - A.half8 : gl, p0 = (low ? gl : gl - A.half8) * NV;
  const size_t plane16 = (size_t)A.kv.page_size * LPH;
  uint4* const cache = static_cast<uint4*>(A.kv.kv_dev);
  for (long long k = k0; k < k1; k += RP_TOKENS) {
    const int nt = (int)min((long long)RP_TOKENS, k1 - k);
    __syncthreads();                             // the last tokens' places are read
    if (before < k + nt && before + sum > k) {   // tokens k .. k + nt - 1: some are of this thread's sequences
      long long lo = before;
      for (int i = a; i < a1 && lo < k + nt; ++i) {
        const ChunkSeq z(A.ix, i);
        for (long long x = max(lo, k); x < min(lo + z.m, k + nt); ++x) {
          const int slot = (int)(x - k), c = (int)(x - lo);
          t_seq[slot] = i;
          t_row[slot] = z.r0 + c;
          t_pos[slot] = z.n + c;
        }
        lo += z.m;
      }
    }
    __syncthreads();
    if (t < nt) {
      const int pos = t_pos[t];
      int page = A.kv.block_table_dev[(size_t)t_seq[t] * A.kv.max_pages + pos / A.kv.page_size];
      if (page < 0 || page >= A.kv.n_pages) {
        page = -1;
        atomicOr(A.err, DERR_PAGE);
      }
      t_page[t] = page;
      t_pos[t] = pos % A.kv.page_size;
    }
    for (int x = t; x < nt * half; x += RP_THREADS) {
      const int tok = x / half, p = x - tok * half;
      const int64_t pos = A.positions[(size_t)A.axis[p] * A.ix.n_rows + t_row[tok]];
      turn_cos_sin((uint32_t)(((uint64_t)pos * A.turn[p]) >> 32), t_cos[tok][p], t_sin[tok][p]);
    }
    __syncthreads();
    // a lane group takes up to RP_FLY heads of a token
    const int items = A.chunks[0] + 2 * A.chunks[1];
    for (int x = g; x < nt * items; x += GROUPS) {
      const int tok = x / items, row = t_row[tok], page = t_page[tok];
      int c = x - tok * items, kind = 0;         // queries, keys, values
      if (c >= A.chunks[0]) {
        c -= A.chunks[0];
        kind = 1;
        if (c >= A.chunks[1]) {
          c -= A.chunks[1];
          kind = 2;
        }
      }
      const int k1 = kind > 0, hk = k1 ? A.kv.n_kv_heads : A.hq, h0 = c * A.heads[k1], nh = min(A.heads[k1], hk - h0);
      const int in0 = h0 + (kind == 0 ? 0 : kind == 1 ? A.hq : A.hq + A.kv.n_kv_heads);
      const uint4* src = reinterpret_cast<const uint4*>(A.qkv + row * A.ld) + (size_t)in0 * LPH + gl;
      uint4 v[RP_FLY];
#pragma unroll
      for (int u = 0; u < RP_FLY; ++u)
        if (u < nh) v[u] = ld_stream(src + u * LPH);
      uint4* dst = reinterpret_cast<uint4*>(A.q_out) + ((size_t)row * A.hq + h0) * LPH + gl;
      size_t step = LPH;
      if (k1) {
        step = 2 * plane16;
        dst = page < 0 ? nullptr
                       : cache + (((size_t)page * A.kv.n_layers + A.layer) * A.kv.n_kv_heads + h0) * step +
                             (kind - 1) * plane16 + (size_t)t_pos[tok] * LPH + gl;
      }
      if (kind < 2) {
        const bool norm = A.gamma[kind] != nullptr;
        unsigned long long C[N2], S[N2];
        {
          float cs[NV], s[NV];
#pragma unroll
          for (int i = 0; i < NV; i += 4) {
            float4 a4 = make_float4(1.f, 1.f, 1.f, 1.f), b4 = make_float4(0.f, 0.f, 0.f, 0.f);
            if (turns) {
              a4 = *reinterpret_cast<const float4*>(&t_cos[tok][p0 + i]);
              b4 = *reinterpret_cast<const float4*>(&t_sin[tok][p0 + i]);
            }
            const float4 ga = *reinterpret_cast<const float4*>(&gam[kind][gl * NV + i]);
            const float4 gb = *reinterpret_cast<const float4*>(&gam[kind][partner * NV + i]);
            cs[i] = a4.x * ga.x; cs[i + 1] = a4.y * ga.y; cs[i + 2] = a4.z * ga.z; cs[i + 3] = a4.w * ga.w;
            s[i] = b4.x * gb.x; s[i + 1] = b4.y * gb.y; s[i + 2] = b4.z * gb.z; s[i + 3] = b4.w * gb.w;
          }
#pragma unroll
          for (int i = 0; i < N2; ++i) {
            C[i] = pair(cs[2 * i], cs[2 * i + 1]);
            S[i] = low ? pair(-s[2 * i], -s[2 * i + 1]) : pair(s[2 * i], s[2 * i + 1]);
          }
        }
#pragma unroll
        for (int u = 0; u < RP_FLY; ++u) {
          if (u >= nh) break;
          unsigned long long f[N2], o[N2];
          unpack2<KT>(v[u], f);
          float r = 1.f;
          if (norm) {
            unsigned long long s2 = mul2(f[0], f[0]);
#pragma unroll
            for (int i = 1; i < N2; ++i) s2 = fma2(f[i], f[i], s2);
            const float2 sq = halves(s2);
            float ss = sq.x + sq.y;
#pragma unroll
            for (int d = 1; d < LPH; d <<= 1) ss += __shfl_xor_sync(gmask, ss, d, LPH);
            r = rsqrtf(ss * (1.f / D) + A.eps);
          }
          uint4 pv;
          pv.x = __shfl_sync(gmask, v[u].x, partner, LPH);
          pv.y = __shfl_sync(gmask, v[u].y, partner, LPH);
          pv.z = __shfl_sync(gmask, v[u].z, partner, LPH);
          pv.w = __shfl_sync(gmask, v[u].w, partner, LPH);
          if (!turns) pv = make_uint4(0u, 0u, 0u, 0u);         // (also where the piece is not finite)
          unpack2<KT>(pv, o);
          const unsigned long long r2 = pair(r, r);
          float y[NV];
#pragma unroll
          for (int i = 0; i < N2; ++i) {
            const float2 z = halves(mul2(r2, fma2(f[i], C[i], mul2(o[i], S[i]))));
            y[2 * i] = z.x;
            y[2 * i + 1] = z.y;
          }
          v[u] = pack_piece<NV>(y);
        }
      }
      if (dst) {
#pragma unroll
        for (int u = 0; u < RP_FLY; ++u)
          if (u < nh) dst[u * step] = v[u];
      }
    }
  }
}

template <class KT, int D>
cudaError_t launch_rope(const RopeArgs& A, int blocks, cudaStream_t st) {
  return launch_k(k_qk_norm_rope<KT, D>, dim3(blocks), dim3(RP_THREADS), 0, st, A);
}

}  // namespace
}  // namespace spec

using namespace spec;

extern "C" int spec_qk_norm_rope(const spec_kv_view* kv, int layer, const void* qkv_dev, int64_t ld, int n_rows, int n_seq,
                                 int n_q_heads, const int32_t* row_start_dev, const int32_t* n_new_dev,
                                 const int32_t* cache_len_dev, const spec_rope* rope, const int32_t* positions_dev,
                                 const float* q_gamma_dev, const float* k_gamma_dev, float eps, void* q_out_dev,
                                 int32_t* err_dev, uintptr_t cuda_stream) {
  int rc = check_chunks(kv, n_seq, n_q_heads);
  if (rc == SPEC_OK) rc = check_layer_rows(kv, layer, n_rows, 1);
  if (rc) return rc;
  if (!qkv_dev || !row_start_dev || !n_new_dev || !cache_len_dev || !rope || !q_out_dev || !err_dev)
    return set_last_error(SPEC_ERR_ARG, "null pointer argument");
  const int esz = kv->dtype == SPEC_F32 ? 4 : 2, d = kv->head_dim;
  const int64_t heads = (int64_t)n_q_heads + 2 * (int64_t)kv->n_kv_heads;
  if (heads > (1 << 20)) return set_last_error(SPEC_ERR_UNSUPPORTED, "more than 2^20 heads");
  if (ld < heads * d || ld % (16 / esz) || ld > ((int64_t)1 << 40))
    return set_last_error(SPEC_ERR_ARG, "ld: at least a row's heads, a multiple of 16 bytes");
  if (!aligned16(qkv_dev) || !aligned16(q_out_dev)) return set_last_error(SPEC_ERR_ARG, "qkv and q must be 16-byte aligned");
  if (!(eps >= 0.f) || !(eps < INFINITY)) return set_last_error(SPEC_ERR_ARG, "eps must be finite and not negative");
  if (rope->dim < 0 || rope->dim > d || rope->dim % 16) return set_last_error(SPEC_ERR_ARG, "rope dim: a multiple of 16 up to head_dim");
  if (rope->n_axes < 1 || rope->n_axes > SPEC_ROPE_MAX_AXES) return set_last_error(SPEC_ERR_ARG, "1 to 4 axes");
  if (rope->dim > 0 && !positions_dev) return set_last_error(SPEC_ERR_ARG, "null positions");
  RopeArgs A{*kv, ChunkIndex{row_start_dev, n_new_dev, cache_len_dev, n_seq, n_rows, n_rows, kv->max_pages * kv->page_size},
             static_cast<const char*>(qkv_dev), static_cast<char*>(q_out_dev), positions_dev, {q_gamma_dev, k_gamma_dev},
             err_dev, ld * esz, layer, n_q_heads, rope->dim / 2 / (16 / esz), {}, {}, eps, {}, {}};
  for (int p = 0; p < rope->dim / 2; ++p) {
    if (!std::isfinite(rope->freq[p])) return set_last_error(SPEC_ERR_ARG, "a frequency is not finite");
    if (rope->axis[p] >= rope->n_axes) return set_last_error(SPEC_ERR_ARG, "a pair's axis is out of range");
    double turn = rope->freq[p] / 6.283185307179586476925286766559;
    turn -= std::floor(turn);                    // [0, 1]: whole turns do not matter
    A.turn[p] = turn < 1.0 ? (uint64_t)std::ldexp(turn, 64) : 0;
    A.axis[p] = rope->axis[p];
  }
  const int64_t in_bytes = ((n_rows - 1) * ld + heads * d) * esz, q_bytes = (int64_t)n_rows * n_q_heads * d * esz;
  if (spans_meet(q_out_dev, q_bytes, qkv_dev, in_bytes) || spans_meet(q_out_dev, q_bytes, kv->kv_dev, cache_bytes(*kv)))
    return set_last_error(SPEC_ERR_ARG, "q_out overlaps qkv or the cache");
  if (spans_meet(qkv_dev, in_bytes, kv->kv_dev, cache_bytes(*kv))) return set_last_error(SPEC_ERR_ARG, "qkv overlaps the cache");
  const int sms = sm_count_once();
  if (sms < 1) return set_last_error(SPEC_ERR_CUDA, "no device");
  int items = 0;
  for (int i = 0; i < 2; ++i) {
    const int n = i ? kv->n_kv_heads : n_q_heads;
    A.chunks[i] = (n + RP_FLY - 1) / RP_FLY;
    A.heads[i] = (n + A.chunks[i] - 1) / A.chunks[i];
    A.chunks[i] = (n + A.heads[i] - 1) / A.heads[i];
    items += (i + 1) * A.chunks[i];
  }
  const int groups = RP_THREADS / (d * esz / 16);
  const int blocks = (int)std::min<int64_t>(((int64_t)n_rows * items + groups - 1) / groups, sms * RP_BLOCKS);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
  cudaError_t e;
  if (esz == 2) e = d == 128 ? launch_rope<bf16_t, 128>(A, blocks, st) : launch_rope<bf16_t, 64>(A, blocks, st);
  else e = d == 128 ? launch_rope<float, 128>(A, blocks, st) : launch_rope<float, 64>(A, blocks, st);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? SPEC_OK : set_last_error(SPEC_ERR_CUDA, cudaGetErrorString(e));
}
