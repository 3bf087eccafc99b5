// Kernel-level entry point: norm and rotation of new tokens' queries and keys, and
// the way of their keys and values into the paged cache.
//
// A head of d values lies on LPH = d / (16 bytes) lanes, so that a warp holds one to
// four heads of a row. A lane has 8 bytes of the lower half of the rotated dims and
// their partners of the upper half (behind the rotated dims any 16 bytes), so a turn
// crosses no lanes. A block takes 4 tokens at a time: their places, the cosines and sines
// of their angles into shared memory, then the heads, up to four of a lane's on their
// way at once, whose sums of squares cross the lanes together. A lane's dims are the
// same in every head, so what they are multiplied by is made once for them: with gamma
// folded in, y_lo = r (lo CL + hi SL), y_hi = r (hi CH + lo SH), r = 1 / sqrt(mean x^2 +
// eps), CL = gamma cos, SL = -gamma' sin ..; behind the rotated dims C = gamma, S = 0.
//
// The angle of position p is p F of a 64-bit turn, F = freq / 2 pi in units of
// 2^-64 of a turn: the product wraps as the angle does. F is off by one unit at most
// (frequencies up to 10^9, of either sign), so p F is by 2^-33 of a turn at position 2^31,
// and by as much again where its upper 32 bits are rounded. They go, reduced to an eighth
// of a turn either way and rounded to fp32 (2^-28 at most), to sincospif.
//
// Bound: HBM, by the bytes of the rows, and below some 10^4 tokens the way there: places,
// angles, rows and results follow one another, in one turn or two of a block. Measured, L2
// cold, bf16, 32 query and 8 kv heads of 128: 16,000 tokens 79 us, 0.75 of the copy rate;
// 4,677 tokens 29.7 us, 0.58. (Pieces of 16 bytes with their partners by shuffle: 31.5;
// the next heads' loads beside a head's arithmetic, which takes the registers of a
// block in four: 35.6, or 33.0 with three blocks; 8 tokens at a time 30.5.)
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "chunk.cuh"
#include "tc_attn.cuh"

namespace spec {
namespace {

constexpr int RP_THREADS = 256;
constexpr int RP_TOKENS = 4;                     // tokens of a block at a time
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
  int layer, hq, half8;                          // half8: rotated pairs / values of 8 bytes
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

// Pairs of the values of 8 bytes, and back.
template <class KT>
__device__ __forceinline__ void unpack2(uint2 v, unsigned long long (&f)[Elt<KT>::per16 / 4]) {
  if constexpr (Elt<KT>::per16 == 4) {
    f[0] = pair(__uint_as_float(v.x), __uint_as_float(v.y));
  } else {
    f[0] = pair(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u));
    f[1] = pair(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
  }
}
template <class KT>
__device__ __forceinline__ uint2 pack2(const unsigned long long (&f)[Elt<KT>::per16 / 4]) {
  const float2 x = halves(f[0]);
  if constexpr (Elt<KT>::per16 == 4) {
    return make_uint2(__float_as_uint(x.x), __float_as_uint(x.y));
  } else {
    const float2 y = halves(f[1]);
    return make_uint2(pack_bf16(x.x, x.y), pack_bf16(y.x, y.y));
  }
}
__device__ __forceinline__ uint2 ld_stream8(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// FULL: all dims turn (16,000 tokens 79 us, 81 without the choice of partners left out).
template <class KT, int D, bool FULL>
__global__ void __launch_bounds__(RP_THREADS, RP_BLOCKS) k_qk_norm_rope(const __grid_constant__ RopeArgs A) {
  constexpr int HV = Elt<KT>::per16 / 2, N2 = HV / 2, LPH = D / (2 * HV), GROUPS = RP_THREADS / LPH;
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
  const int half = A.half8 * HV;
  // the lane's dims: lo .. and their partners hi ..; behind the rotated ones, any two pieces
  const bool turns = FULL || gl < A.half8;
  const int lo = turns ? gl * HV : 2 * half + 2 * (gl - A.half8) * HV, hi = turns ? half + lo : lo + HV;
  const size_t plane = (size_t)A.kv.page_size * D;
  KT* const cache = static_cast<KT*>(A.kv.kv_dev);
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
      turn_cos_sin((uint32_t)(((uint64_t)pos * A.turn[p] + 0x80000000u) >> 32), t_cos[tok][p], t_sin[tok][p]);
    }
    __syncthreads();
    // a lane group takes up to RP_FLY heads of a token
    const int items = A.chunks[0] + 2 * A.chunks[1];
    for (int x = g; x < nt * items; x += GROUPS) {
      const int tok = x / items, row = t_row[tok], page = t_page[tok];
      int part = x - tok * items, kind = 0;      // queries, keys, values
      if (part >= A.chunks[0]) {
        part -= A.chunks[0];
        kind = 1;
        if (part >= A.chunks[1]) {
          part -= A.chunks[1];
          kind = 2;
        }
      }
      const int k1 = kind > 0, hk = k1 ? A.kv.n_kv_heads : A.hq, h0 = part * A.heads[k1], nh = min(A.heads[k1], hk - h0);
      const int in0 = h0 + (kind == 0 ? 0 : kind == 1 ? A.hq : A.hq + A.kv.n_kv_heads);
      const KT* src = reinterpret_cast<const KT*>(A.qkv + row * A.ld) + (size_t)in0 * D;
      uint2 vl[RP_FLY], vh[RP_FLY];
#pragma unroll
      for (int u = 0; u < RP_FLY; ++u) {
        vl[u] = vh[u] = make_uint2(0u, 0u);
        if (u < nh) {
          vl[u] = ld_stream8(src + u * D + lo);
          vh[u] = ld_stream8(src + u * D + hi);
        }
      }
      KT* dst = reinterpret_cast<KT*>(A.q_out) + ((size_t)row * A.hq + h0) * D;
      size_t step = D;
      if (k1) {
        step = 2 * plane;
        dst = page < 0 ? nullptr
                       : cache + (((size_t)page * A.kv.n_layers + A.layer) * A.kv.n_kv_heads + h0) * step + (kind - 1) * plane +
                             (size_t)t_pos[tok] * D;
      }
      if (kind < 2) {
        float r = 1.f;                           // lane u < RP_FLY: of head u
        if (A.gamma[kind]) {
          float ss[RP_FLY];
#pragma unroll
          for (int u = 0; u < RP_FLY; ++u) {
            unsigned long long fl[N2], fh[N2];
            unpack2<KT>(vl[u], fl);
            unpack2<KT>(vh[u], fh);
            unsigned long long s2 = mul2(fl[0], fl[0]);
#pragma unroll
            for (int i = 1; i < N2; ++i) s2 = fma2(fl[i], fl[i], s2);
#pragma unroll
            for (int i = 0; i < N2; ++i) s2 = fma2(fh[i], fh[i], s2);
            const float2 sq = halves(s2);
            ss[u] = sq.x + sq.y;
          }
          // four sums over the group's lanes at once: a lane keeps the heads of its two lowest bits
          const bool b0 = gl & 1, b1 = gl & 2;
          const float s0 = (b0 ? ss[1] : ss[0]) + __shfl_xor_sync(gmask, b0 ? ss[0] : ss[1], 1, LPH);
          const float s1 = (b0 ? ss[3] : ss[2]) + __shfl_xor_sync(gmask, b0 ? ss[2] : ss[3], 1, LPH);
          float sum4 = (b1 ? s1 : s0) + __shfl_xor_sync(gmask, b1 ? s0 : s1, 2, LPH);
#pragma unroll
          for (int d = 4; d < LPH; d <<= 1) sum4 += __shfl_xor_sync(gmask, sum4, d, LPH);
          r = rsqrtf(sum4 * (1.f / D) + A.eps);
        }
        // y_lo = r (lo CL + hi SL), y_hi = r (hi CH + lo SH)
        unsigned long long CL[N2], SL[N2], CH[N2], SH[N2];
        using F = std::conditional_t<HV == 4, float4, float2>;
        union Row { F f; float2 p[N2]; };
        Row c, s, gl2, gh2;
        if (turns) {
          c.f = *reinterpret_cast<const F*>(&t_cos[tok][lo]);
          s.f = *reinterpret_cast<const F*>(&t_sin[tok][lo]);
        }
        gl2.f = *reinterpret_cast<const F*>(&gam[kind][lo]);
        gh2.f = *reinterpret_cast<const F*>(&gam[kind][hi]);
#pragma unroll
        for (int i = 0; i < N2; ++i) {
          const float2 c2 = turns ? c.p[i] : make_float2(1.f, 1.f), s2 = turns ? s.p[i] : make_float2(0.f, 0.f), ga = gl2.p[i], gb = gh2.p[i];
          CL[i] = pair(c2.x * ga.x, c2.y * ga.y);
          SL[i] = pair(-s2.x * gb.x, -s2.y * gb.y);
          CH[i] = pair(c2.x * gb.x, c2.y * gb.y);
          SH[i] = pair(s2.x * ga.x, s2.y * ga.y);
        }
#pragma unroll
        for (int u = 0; u < RP_FLY; ++u) {
          if (u >= nh) break;
          const float ru = __shfl_sync(gmask, r, u, LPH);
          const unsigned long long r2 = pair(ru, ru);
          unsigned long long fl[N2], fh[N2];
          unpack2<KT>(vl[u], fl);
          unpack2<KT>(vh[u], fh);
#pragma unroll
          for (int i = 0; i < N2; ++i) {
            // (where nothing turns, whatever the partner is)
            const unsigned long long a2 = mul2(turns ? fh[i] : 0ull, SL[i]), b2 = mul2(turns ? fl[i] : 0ull, SH[i]);
            fl[i] = mul2(r2, fma2(fl[i], CL[i], a2));
            fh[i] = mul2(r2, fma2(fh[i], CH[i], b2));
          }
          vl[u] = pack2<KT>(fl);
          vh[u] = pack2<KT>(fh);
        }
      }
      if (dst) {
#pragma unroll
        for (int u = 0; u < RP_FLY; ++u) {
          if (u < nh) {
            *reinterpret_cast<uint2*>(dst + u * step + lo) = vl[u];
            *reinterpret_cast<uint2*>(dst + u * step + hi) = vh[u];
          }
        }
      }
    }
  }
}

// freq / 2 pi modulo 1 in units of 2^-64: the product with 1 / 2 pi as two doubles, each of
// its two parts rounded to a unit. (The quotient in double would be off by 2^-53 of itself, which
// far positions multiply, and a negative one by 2^-53 of a turn where it is brought to [0, 1).)
uint64_t turn_of(double freq) {
  constexpr double INV = 0.15915494309189535, INV_LO = -9.839338337591243e-18;
  auto units = [](double x) { return (uint64_t)std::rint((x - std::floor(x)) * 0x1p64); };   // x >= 0
  const double a = std::fabs(freq), hi = a * INV, lo = std::fma(a, INV, -hi) + a * INV_LO;
  const uint64_t u = units(hi) + (lo < 0 ? 0 - units(-lo) : units(lo));
  return freq < 0 ? 0 - u : u;
}

template <class KT, int D>
cudaError_t launch_rope(const RopeArgs& A, int blocks, cudaStream_t st) {
  return A.half8 * 8 * 2 == D * (int)sizeof(KT) ? launch_k(k_qk_norm_rope<KT, D, true>, dim3(blocks), dim3(RP_THREADS), 0, st, A)
                                                : launch_k(k_qk_norm_rope<KT, D, false>, dim3(blocks), dim3(RP_THREADS), 0, st, A);
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
  if (ld < heads * d || ld % (16 / esz)) return set_last_error(SPEC_ERR_ARG, "ld: at least a row's heads, a multiple of 16 bytes");
  if ((double)ld * n_rows > 1e18) return set_last_error(SPEC_ERR_UNSUPPORTED, "rows of more than 10^18 elements");
  if (!aligned16(qkv_dev) || !aligned16(q_out_dev)) return set_last_error(SPEC_ERR_ARG, "qkv and q must be 16-byte aligned");
  if (!(eps >= 0.f) || !(eps < INFINITY)) return set_last_error(SPEC_ERR_ARG, "eps must be finite and not negative");
  if (rope->dim < 0 || rope->dim > d || rope->dim % 16) return set_last_error(SPEC_ERR_ARG, "rope dim: a multiple of 16 up to head_dim");
  if (rope->n_axes < 1 || rope->n_axes > SPEC_ROPE_MAX_AXES) return set_last_error(SPEC_ERR_ARG, "1 to 4 axes");
  if (rope->dim > 0 && !positions_dev) return set_last_error(SPEC_ERR_ARG, "null positions");
  RopeArgs A{*kv, ChunkIndex{row_start_dev, n_new_dev, cache_len_dev, n_seq, n_rows, n_rows, kv->max_pages * kv->page_size},
             static_cast<const char*>(qkv_dev), static_cast<char*>(q_out_dev), positions_dev, {q_gamma_dev, k_gamma_dev},
             err_dev, ld * esz, layer, n_q_heads, rope->dim / 2 / (8 / esz), {}, {}, eps, {}, {}};
  for (int p = 0; p < rope->dim / 2; ++p) {
    if (!std::isfinite(rope->freq[p])) return set_last_error(SPEC_ERR_ARG, "a frequency is not finite");
    if (rope->axis[p] >= rope->n_axes) return set_last_error(SPEC_ERR_ARG, "a pair's axis is out of range");
    A.turn[p] = turn_of(rope->freq[p]);
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
