// iq_run.hip -- tokens through encoded weights: iq_linear (a projection with the
// low-rank adapters of many requests) and iq_moe (a mixture-of-experts layer),
// declared in include/iq_run.h.
//
// A weight is d * m * v: d the block's fp16 scale, m the group's odd multiplier,
// v its signed codebook value.  The products run on the fp16 matrix cores:
// m * v is formed in packed fp16 (exact for the layouts' codebooks: at most 11
// bits), d and the tokens' power-of-two block scales are applied in fp32 to
// each 256-column block's sum.
//
// Operand layout (v_mfma_f32_16x16x32_f16): the weights are B, lane l holding
// eight consecutive k of row n = l % 16; the tokens are A, lane l holding the
// same k of token m = l % 16; D has lane l hold row n = l % 16 and tokens
// 4 (l / 16) + 0..3.  The order of k is free as long as both operands use it:
// lane quarter q = l / 16 takes the block's 64 columns from 64 q on, eight at a
// step, so that a lane's share of the payload is contiguous (two to three wide
// loads a block) and one group of eight values is one codebook entry.

#include "iq_run.h"
#include "iq_common.hpp"
#include "iq_internal.hpp"

namespace iq {
namespace {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8v __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int ST_ROUNDED = 32;
constexpr int kGridN[5] = {256, 512, 1024, 2048, 2048};

bool launched_ok() { return hipGetLastError() == hipSuccess; }

// ---------------------------------------------------------------------------
// Payload fields
// ---------------------------------------------------------------------------
template <class T> __device__ __forceinline__ T ldu(const uint8_t *p) {  // any alignment
  T v;
  __builtin_memcpy(&v, p, sizeof(T));
  return v;
}

// One lane's share of a block: the fields of groups 8q .. 8q + 7.
struct Raw {
  uint32_t a[4];
  uint32_t s;
  uint32_t d16;
};

template <int F> __device__ __forceinline__ Raw load_raw(const uint8_t *blk, int q) {
  Raw r;
  if (F == IQ2_XXS || F == IQ2_XS) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.a[i] = ldu<uint32_t>(blk + 2 + 16 * q + 4 * i);
    r.s = F == IQ2_XS ? ldu<uint16_t>(blk + 66 + 2 * q) : 0;
    r.d16 = ldu<uint16_t>(blk);
  } else if (F == IQ2_S) {
    r.a[0] = ldu<uint32_t>(blk + 2 + 8 * q);
    r.a[1] = ldu<uint32_t>(blk + 6 + 8 * q);
    r.a[2] = ldu<uint32_t>(blk + 34 + 8 * q);
    r.a[3] = ldu<uint32_t>(blk + 38 + 8 * q);
    r.s = ldu<uint16_t>(blk + 66 + 2 * q) | (static_cast<uint32_t>(ldu<uint16_t>(blk + 74 + 2 * q)) << 16);
    r.d16 = ldu<uint16_t>(blk);
  } else if (F == IQ1_S) {
    r.a[0] = ldu<uint32_t>(blk + 2 + 8 * q);
    r.a[1] = ldu<uint32_t>(blk + 6 + 8 * q);
    r.a[2] = ldu<uint32_t>(blk + 34 + 4 * q);
    r.a[3] = r.s = 0;
    r.d16 = ldu<uint16_t>(blk);
  } else {
    r.a[0] = ldu<uint32_t>(blk + 8 * q);
    r.a[1] = ldu<uint32_t>(blk + 8 * q + 4);
    r.a[2] = ldu<uint32_t>(blk + 32 + 4 * q);
    r.a[3] = 0;
    r.s = ldu<uint16_t>(blk + 48 + 2 * q);
    const uint32_t w0 = ldu<uint32_t>(blk + 48), w1 = ldu<uint32_t>(blk + 52);
    r.d16 = ((w0 >> 12) & 15u) | ((w0 >> 28) << 4) | (((w1 >> 12) & 15u) << 8) | ((w1 >> 28) << 12);
  }
  return r;
}

template <int F> __device__ __forceinline__ float block_scale(const Raw &r) {
  const float d = f16_bits_to_f32(static_cast<uint16_t>(r.d16));
  return Geo<F>::IQ1 ? d : d * 0.125f;  // exact: a power of two
}

// m * v of group 8q + i as eight fp16 values (tab: the codebook in fp16).
template <int F> __device__ __forceinline__ half8v group_half8(const Raw &r, int i, const uint4 *tab) {
  uint32_t k, ls, mask = 0, h = 0;
  if (F == IQ2_XXS) {
    const uint32_t word = r.a[2 * (i >> 2) + 1];
    k = (r.a[2 * (i >> 2)] >> (8 * (i & 3))) & 255u;
    mask = (word >> (7 * (i & 3))) & 127u;
    ls = word >> 28;
  } else if (F == IQ2_XS) {
    const uint32_t v = (r.a[i >> 1] >> (16 * (i & 1))) & 0xffffu;
    k = v & 511u;
    mask = v >> 9;
    ls = (r.s >> (4 * (i >> 1))) & 15u;
  } else if (F == IQ2_S) {
    k = ((r.a[i >> 2] >> (8 * (i & 3))) & 255u) | (((r.s >> (2 * i)) & 3u) << 8);
    mask = (r.a[2 + (i >> 2)] >> (8 * (i & 3))) & 255u;
    ls = (r.s >> (16 + 4 * (i >> 1))) & 15u;
  } else if (F == IQ1_S) {
    const uint32_t w = (r.a[2] >> (16 * (i >> 2))) & 0xffffu;
    k = ((r.a[i >> 2] >> (8 * (i & 3))) & 255u) | (((w >> (3 * (i & 3))) & 7u) << 8);
    ls = (w >> 12) & 7u;
    h = w >> 15;
  } else {
    const uint32_t nib = (r.a[2] >> (4 * i)) & 15u;
    k = ((r.a[i >> 2] >> (8 * (i & 3))) & 255u) | ((nib & 7u) << 8);
    h = nib >> 3;
    ls = (r.s >> (3 * (i >> 1))) & 7u;
  }
  const uint4 e = tab[k];
  const _Float16 m = static_cast<_Float16>(static_cast<uint16_t>(2 * ls + 1));
  const half2v m2 = {m, m};
  uint32_t o[4] = {e.x, e.y, e.z, e.w};
  if (Geo<F>::IQ1) {
    const half2v c2 = m2 * (h ? static_cast<_Float16>(-0.125f) : static_cast<_Float16>(0.125f));
#pragma unroll
    for (int p = 0; p < 4; ++p)  // m g + m delta, rounded once
      o[p] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(half2v, o[p]), m2, c2));
  } else {
    // the eighth sign is the parity of the seven (IQ2_S holds it); then bit 2p
    // to 2p and bit 2p + 1 to 2p + 16, so one shift brings a pair's signs home
    if (Geo<F>::PARITY) mask |= __builtin_popcount(mask) << 7;
    const uint32_t sp = (mask & 0x55u) | ((mask & 0xaau) << 15);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const half2v v = __builtin_bit_cast(half2v, o[p]) * m2;
      o[p] = __builtin_bit_cast(uint32_t, v) ^ ((sp << (15 - 2 * p)) & 0x80008000u);
    }
  }
  return __builtin_bit_cast(half8v, make_uint4(o[0], o[1], o[2], o[3]));
}

// ---------------------------------------------------------------------------
// Tokens in fp16: x16 [block][tile of 16 tokens][part][step 0..7][lane][8], the
// A operand of step i as 1 KiB of consecutive memory; ex [block][tokens]: the
// power of two that undoes the block's scaling.  Tokens past T are left
// unwritten: they only reach outputs that are not stored.
// ---------------------------------------------------------------------------
struct Tokens {
  _Float16 *x16;
  int32_t *ex;
  int64_t ntile;  // tiles of 16 tokens
  int parts;
};

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v = max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), o, 64)));
  return v;
}

// One wave: token t's block b (lane: columns 4 lane .. + 3, given in v).
__device__ __forceinline__ void store_block(const Tokens &X, int64_t t, int64_t b, int lane, const float v[4]) {
  uint32_t e = 1;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t u = (__float_as_uint(v[j]) >> 23) & 255u;
    e = max(e, u == 255u ? 1u : u);
  }
  const int n = 141 - static_cast<int>(wave_max(e));  // 14 - (e - 127): |x 2^n| < 2^15
  _Float16 hi[4], lo[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float f = ldexpf(v[j], n);
    hi[j] = static_cast<_Float16>(f);
    lo[j] = finite_f(f) ? static_cast<_Float16>(f - static_cast<float>(hi[j])) : static_cast<_Float16>(0.0f);
  }
  const int q = lane >> 4, i = (lane & 15) >> 1;
  const int64_t tile = b * X.ntile + (t >> 4);
  const int64_t at = (static_cast<int64_t>(i) * 64 + q * 16 + (t & 15)) * 8 + (lane & 1) * 4;
  _Float16 *p = X.x16 + tile * X.parts * 4096 + at;
  *reinterpret_cast<uint2 *>(p) = __builtin_bit_cast(uint2, hi);
  if (X.parts == 2) *reinterpret_cast<uint2 *>(p + 4096) = __builtin_bit_cast(uint2, lo);
  if (lane == 0) X.ex[b * X.ntile * 16 + t] = -n;
}

__device__ __forceinline__ float load1(const void *x, int dtype, int64_t i) {
  return dtype == 1 ? bf16_to_f32(static_cast<const uint16_t *>(x)[i]) : static_cast<const float *>(x)[i];
}

__device__ __forceinline__ void store1(void *y, int dtype, int64_t i, float v) {
  if (dtype == 1)
    static_cast<uint16_t *>(y)[i] = f32_to_bf16(v);
  else
    static_cast<float *>(y)[i] = v;
}

// Workgroups 0 .. nconv - 1 convert tokens (four blocks each), the one after
// them the codebook, and one more a second codebook if there is one.
struct PrepArgs {
  const void *x;
  int dtype;
  int64_t T, cols, nconv;
  Tokens X;
  const float *grid[2];
  _Float16 *tab[2];
  int n[2], iq1[2];
  int32_t *status;
};

__device__ void convert_codebook(const float *grid, _Float16 *tab, int n, bool iq1, int32_t *status) {
  bool inexact = false;
  for (int i = threadIdx.x; i < n * 8; i += blockDim.x) {
    const float g = grid[i];
    tab[i] = static_cast<_Float16>(g);
    for (int m = 1; m < (iq1 ? 16 : 32); m += 2) {
      const float f = static_cast<float>(m);
      if (iq1) {
        inexact |= static_cast<float>(static_cast<_Float16>(f * (g + 0.125f))) != f * (g + 0.125f);
        inexact |= static_cast<float>(static_cast<_Float16>(f * (g - 0.125f))) != f * (g - 0.125f);
      } else {
        inexact |= static_cast<float>(static_cast<_Float16>(f * g)) != f * g;
      }
    }
    inexact |= static_cast<float>(tab[i]) != g;
  }
  if (inexact) raise_status(status, ST_ROUNDED);
}

__global__ void __launch_bounds__(256) run_prep_kernel(PrepArgs P) {
  if (blockIdx.x >= P.nconv) {
    const int w = static_cast<int>(blockIdx.x - P.nconv);
    convert_codebook(P.grid[w], P.tab[w], P.n[w], P.iq1[w], P.status);
    return;
  }
  const int64_t nb = P.cols >> 8, i = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (i >= P.T * nb) return;
  const int lane = threadIdx.x & 63;
  const int64_t t = i / nb, b = i - t * nb;
  float v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = load1(P.x, P.dtype, t * P.cols + b * 256 + lane * 4 + j);
  store_block(P.X, t, b, lane, v);
}

template <int F> __device__ __forceinline__ void load_table(uint4 *s_tab, const _Float16 *tab) {
  for (int i = threadIdx.x; i < Geo<F>::N; i += blockDim.x) s_tab[i] = reinterpret_cast<const uint4 *>(tab)[i];
}

// acc += one block of a 16-row by 16-token product.  rowp: the lane's row in
// the payload; xlane: which of the tile's tokens the lane feeds.
template <int F>
__device__ __forceinline__ void block_product(const uint8_t *blk, const uint4 *s_tab, const Tokens &X, int64_t b,
                                              int64_t tile, int xlane, int q, f32x4 &acc, const int ex[4]) {
  const Raw r = load_raw<F>(blk, q);
  f32x4 part = {0.0f, 0.0f, 0.0f, 0.0f};
  const _Float16 *xp = X.x16 + (b * X.ntile + tile) * X.parts * 4096 + (q * 16 + xlane) * 8;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const half8v w = group_half8<F>(r, i, s_tab);
    part = __builtin_amdgcn_mfma_f32_16x16x32_f16(*reinterpret_cast<const half8v *>(xp + i * 512), w, part, 0, 0, 0);
    if (X.parts == 2)
      part = __builtin_amdgcn_mfma_f32_16x16x32_f16(*reinterpret_cast<const half8v *>(xp + 4096 + i * 512), w, part,
                                                    0, 0, 0);
  }
  const float d = block_scale<F>(r);
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] += ldexpf(d * part[k], ex[k]);
}

// ---------------------------------------------------------------------------
// Mixture of experts
// ---------------------------------------------------------------------------
// logits[t][e] in fp64, one wave each
__global__ void __launch_bounds__(256) router_kernel(const void *x, int dtype, const void *router, int rdtype,
                                                      int64_t T, int64_t K, int E, double *logits) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (i >= T * E) return;
  const int lane = threadIdx.x & 63;
  const int64_t t = i / E, e = i - t * E;
  double s = 0.0;
  for (int64_t k = lane; k < K; k += 64)
    s = fma(static_cast<double>(load1(router, rdtype, e * K + k)), static_cast<double>(load1(x, dtype, t * K + k)), s);
#pragma unroll
  for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o, 64);
  if (lane == 0) logits[i] = s;
}

// one wave per token: the top_k largest logits, ties to the lower id, NaN last
__global__ void __launch_bounds__(64) topk_kernel(const double *logits, int E, int top_k, int renorm, int32_t *ids,
                                                   float *weights) {
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x;
  const double *l = logits + t * E;
  double top = 0.0;
  float sum = 0.0f, mine = 0.0f;
  double last = 0.0;
  int last_id = -1;
  bool last_nan = false;
  for (int s = 0; s < top_k; ++s) {
    // the largest (value, lower id) after (last, last_id) in the order
    double bv = 0.0;
    int bi = -1;
    bool bn = false;
    for (int e = lane; e < E; e += 64) {
      const double v = l[e];
      const bool nan = v != v;
      const bool after = last_id < 0 || (nan ? (!last_nan || e > last_id)
                                             : (!last_nan && (v < last || (v == last && e > last_id))));
      if (!after) continue;
      if (bi < 0 || (bn && !nan) || (!bn && !nan && v > bv)) {
        bv = v;
        bi = e;
        bn = nan;
      }
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) {
      const double ov = __shfl_xor(bv, o, 64);
      const int oi = __shfl_xor(bi, o, 64);
      const bool on = __shfl_xor(static_cast<int>(bn), o, 64) != 0;
      const bool take = oi >= 0 && (bi < 0 || (bn != on ? bn : (!bn && ov != bv ? ov > bv : oi < bi)));
      if (take) {
        bv = ov;
        bi = oi;
        bn = on;
      }
    }
    last = bv;
    last_id = bi;
    last_nan = bn;
    if (s == 0) top = bv;
    const float p = expf(static_cast<float>(bv - top));
    sum += p;
    if (lane == s) mine = p;
    if (lane == 0) ids[t * top_k + s] = bi;
  }
  if (!renorm) {
    sum = 0.0f;
    for (int e = lane; e < E; e += 64) sum += expf(static_cast<float>(l[e] - top));
#pragma unroll
    for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o, 64);
  }
  if (lane < top_k) weights[t * top_k + lane] = mine / sum;
}

// One wave: 16 rows of gate and up for one (token, slot) pair; h = weight *
// silu(g) * u.  Every row of the A operand is the pair's token.
template <int F>
__global__ void __launch_bounds__(256) gate_up_kernel(const uint8_t *gate, const uint8_t *up, int64_t inter,
                                                       int64_t nb, int E, const _Float16 *tab, Tokens X,
                                                       int64_t npair, int top_k, const int32_t *ids,
                                                       const float *weights, float *h, int32_t *status) {
  __shared__ uint4 s_tab[Geo<F>::N];
  load_table<F>(s_tab, tab);
  __syncthreads();
  const int64_t nrt = inter / 16, w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int64_t p = w / nrt, rt = w - p * nrt;
  if (p >= npair) return;
  const int e = ids[p];
  if (e < 0 || e >= E) {
    raise_status(status, ST_BADID);
    return;
  }
  const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  const int64_t t = p / top_k, row = e * inter + rt * 16 + n;
  f32x4 ag = {0.0f, 0.0f, 0.0f, 0.0f}, au = ag;
  for (int64_t b = 0; b < nb; ++b) {
    const int x = X.ex[b * X.ntile * 16 + t], ex[4] = {x, x, x, x};
    block_product<F>(gate + (row * nb + b) * Geo<F>::BYTES, s_tab, X, b, t >> 4, t & 15, q, ag, ex);
    block_product<F>(up + (row * nb + b) * Geo<F>::BYTES, s_tab, X, b, t >> 4, t & 15, q, au, ex);
  }
  if (q == 0) h[p * inter + rt * 16 + n] = ag[0] / (1.0f + expf(-ag[0])) * au[0] * weights[p];
}

// One wave: 16 output columns of one token, over the token's experts.
template <int F>
__global__ void __launch_bounds__(256) down_kernel(const uint8_t *down, int64_t hidden, int64_t nb, int E,
                                                    const _Float16 *tab, Tokens H, int64_t T, int top_k,
                                                    const int32_t *ids, int dtype, void *y) {
  __shared__ uint4 s_tab[Geo<F>::N];
  load_table<F>(s_tab, tab);
  __syncthreads();
  const int64_t nrt = hidden / 16, w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int64_t t = w / nrt, rt = w - t * nrt;
  if (t >= T) return;
  const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = 0; s < top_k; ++s) {
    const int64_t p = t * top_k + s;
    const int e = ids[p];
    if (e < 0 || e >= E) continue;
    const int64_t row = e * hidden + rt * 16 + n;
    for (int64_t b = 0; b < nb; ++b) {
      const int x = H.ex[b * H.ntile * 16 + p], ex[4] = {x, x, x, x};
      block_product<F>(down + (row * nb + b) * Geo<F>::BYTES, s_tab, H, b, p >> 4, p & 15, q, acc, ex);
    }
  }
  if (q == 0) store1(y, dtype, t * hidden + rt * 16 + n, acc[0]);
}

// ---------------------------------------------------------------------------
// Workspaces
// ---------------------------------------------------------------------------
constexpr int64_t kMaxGrid = (int64_t(1) << 31) - 1;

struct TokensPlan {
  int64_t ntile;
  int parts;
  size_t xbytes, ebytes;
};
TokensPlan plan_tokens(int64_t T, int64_t cols, int dtype) {
  TokensPlan p;
  p.ntile = (T + 15) / 16;
  p.parts = dtype == IQ_DTYPE_F32 ? 2 : 1;
  p.xbytes = static_cast<size_t>(cols / 256) * p.ntile * p.parts * 8192;
  p.ebytes = static_cast<size_t>(cols / 256) * p.ntile * 64;
  return p;
}

struct MoePlan {
  TokensPlan x, h;
  size_t tab, tab2, xo, eo, lo, ho, hxo, heo, bytes;
};
MoePlan plan_moe(int fmt, int down_fmt, int64_t hidden, int64_t inter, int E, int dtype, int64_t T, int top_k) {
  MoePlan p;
  p.x = plan_tokens(T, hidden, dtype);
  p.h = plan_tokens(T * top_k, inter, dtype);
  p.tab = 0;
  p.tab2 = ws_up(static_cast<size_t>(kGridN[fmt]) * 16);
  p.xo = p.tab2 + ws_up(static_cast<size_t>(kGridN[down_fmt]) * 16);
  p.eo = p.xo + ws_up(p.x.xbytes);
  p.lo = p.eo + ws_up(p.x.ebytes);
  p.ho = p.lo + ws_up(static_cast<size_t>(T) * E * 8);
  p.hxo = p.ho + ws_up(static_cast<size_t>(T) * top_k * inter * 4);
  p.heo = p.hxo + ws_up(p.h.xbytes);
  p.bytes = p.heo + ws_up(p.h.ebytes) + kWsAlign;
  return p;
}

bool bad_fmt(int f) { return f < 0 || f > 4; }
bool bad_dtype(int d) { return d != IQ_DTYPE_F32 && d != IQ_DTYPE_BF16; }

int check_moe(int fmt, int down_fmt, int64_t hidden, int64_t inter, int E, int dtype, int64_t T, int top_k) {
  if (bad_fmt(fmt) || bad_fmt(down_fmt)) return IQ_ERR_FMT;
  if (bad_dtype(dtype)) return IQ_ERR_DTYPE;
  if (T < 0 || hidden <= 0 || hidden % 256 != 0 || inter <= 0 || inter % 256 != 0) return IQ_ERR_SHAPE;
  if (hidden > (int64_t(1) << 24) || inter > (int64_t(1) << 24)) return IQ_ERR_SHAPE;
  if (E < 1 || E > 4096 || top_k < 1 || top_k > 64) return IQ_ERR_ARG;
  const int64_t big = hidden > inter ? hidden : inter;
  if (T > (int64_t(1) << 24) || T * top_k * (big / 16) >= kMaxGrid || T * E >= kMaxGrid) return IQ_ERR_SHAPE;
  return IQ_OK;
}

int check_ws(size_t need, const void *ws, size_t have) {
  if (!ws) return IQ_ERR_NULL;
  return have < need ? IQ_ERR_WORKSPACE : IQ_OK;
}

dim3 waves4(int64_t n) { return dim3(static_cast<unsigned>((n + 3) / 4)); }

int launch_prep(const void *x, int dtype, int64_t T, int64_t cols, const Tokens &X, const float *g0, _Float16 *t0,
                int f0, const float *g1, _Float16 *t1, int f1, int32_t *status, hipStream_t stream) {
  PrepArgs P{};
  P.x = x;
  P.dtype = dtype;
  P.T = T;
  P.cols = cols;
  P.nconv = (T * (cols / 256) + 3) / 4;
  P.X = X;
  P.grid[0] = g0;
  P.grid[1] = g1;
  P.tab[0] = t0;
  P.tab[1] = t1;
  P.n[0] = kGridN[f0];
  P.n[1] = kGridN[f1];
  P.iq1[0] = f0 >= IQ1_S;
  P.iq1[1] = f1 >= IQ1_S;
  P.status = status;
  const int ntab = (g0 ? 1 : 0) + (g1 ? 1 : 0);
  hipLaunchKernelGGL(run_prep_kernel, dim3(static_cast<unsigned>(P.nconv + ntab)), dim3(256), 0, stream, P);
  return launched_ok() ? IQ_OK : IQ_ERR_HIP;
}

#define IQ_BY_FMT(fmt, CALL)                      \
  switch (fmt) {                                  \
    case IQ2_XXS: CALL(IQ2_XXS); break;           \
    case IQ2_XS: CALL(IQ2_XS); break;             \
    case IQ2_S: CALL(IQ2_S); break;               \
    case IQ1_S: CALL(IQ1_S); break;               \
    default: CALL(IQ1_M); break;                  \
  }

}  // namespace
}  // namespace iq

extern "C" {

int iq_moe_workspace_size(int fmt, int down_fmt, int64_t hidden, int64_t inter, int num_experts, int dtype,
                          int64_t T, int top_k, size_t *bytes) {
  const int rc = iq::check_moe(fmt, down_fmt, hidden, inter, num_experts, dtype, T, top_k);
  if (rc != IQ_OK) return rc;
  if (!bytes) return IQ_ERR_NULL;
  *bytes = T ? iq::plan_moe(fmt, down_fmt, hidden, inter, num_experts, dtype, T, top_k).bytes : 0;
  return IQ_OK;
}

int iq_moe(int fmt, int down_fmt, const uint8_t *gate, const uint8_t *up, const uint8_t *down, int64_t hidden,
           int64_t inter, int num_experts, const float *grid, const float *down_grid, const void *x, int dtype,
           int64_t T, const void *router, int router_dtype, int top_k, int renormalize, int32_t *ids,
           float *weights, void *y, void *workspace, size_t workspace_bytes, int32_t *status, hipStream_t stream) {
  using namespace iq;
  int rc = check_moe(fmt, down_fmt, hidden, inter, num_experts, dtype, T, top_k);
  if (rc != IQ_OK) return rc;
  if (router && bad_dtype(router_dtype)) return IQ_ERR_DTYPE;
  if (!grid || !down_grid || (T && (!gate || !up || !down || !x || !ids || !weights || !y))) return IQ_ERR_NULL;
  if (router && top_k > num_experts) return IQ_ERR_ARG;
  if (T == 0) return IQ_OK;
  const int E = num_experts;
  const MoePlan P = plan_moe(fmt, down_fmt, hidden, inter, E, dtype, T, top_k);
  if ((rc = check_ws(P.bytes, workspace, workspace_bytes)) != IQ_OK) return rc;
  char *base = ws_base(workspace);
  _Float16 *tab = reinterpret_cast<_Float16 *>(base + P.tab), *tab2 = reinterpret_cast<_Float16 *>(base + P.tab2);
  const Tokens X{reinterpret_cast<_Float16 *>(base + P.xo), reinterpret_cast<int32_t *>(base + P.eo), P.x.ntile,
                 P.x.parts};
  const Tokens H{reinterpret_cast<_Float16 *>(base + P.hxo), reinterpret_cast<int32_t *>(base + P.heo), P.h.ntile,
                 P.h.parts};
  double *logits = reinterpret_cast<double *>(base + P.lo);
  float *h = reinterpret_cast<float *>(base + P.ho);
  const int64_t np = T * top_k;
  if ((rc = launch_prep(x, dtype, T, hidden, X, grid, tab, fmt, down_grid, tab2, down_fmt, status, stream)) != IQ_OK)
    return rc;
  if (router) {
    hipLaunchKernelGGL(router_kernel, waves4(T * E), dim3(256), 0, stream, x, dtype, router, router_dtype, T, hidden,
                       E, logits);
    if (!launched_ok()) return IQ_ERR_HIP;
    hipLaunchKernelGGL(topk_kernel, dim3(static_cast<unsigned>(T)), dim3(64), 0, stream,
                       static_cast<const double *>(logits), E, top_k, renormalize, ids, weights);
    if (!launched_ok()) return IQ_ERR_HIP;
  }
#define CALL(F)                                                                                                     \
  hipLaunchKernelGGL(gate_up_kernel<F>, waves4(np * (inter / 16)), dim3(256), 0, stream, gate, up, inter,           \
                     hidden / 256, E, tab, X, np, top_k, static_cast<const int32_t *>(ids),                         \
                     static_cast<const float *>(weights), h, status)
  IQ_BY_FMT(fmt, CALL)
#undef CALL
  if (!launched_ok()) return IQ_ERR_HIP;
  if ((rc = launch_prep(h, IQ_DTYPE_F32, np, inter, H, nullptr, nullptr, 0, nullptr, nullptr, 0, status, stream)) !=
      IQ_OK)
    return rc;
#define CALL(F)                                                                                                    \
  hipLaunchKernelGGL(down_kernel<F>, waves4(T * (hidden / 16)), dim3(256), 0, stream, down, hidden, inter / 256, E, \
                     tab2, H, T, top_k, static_cast<const int32_t *>(ids), dtype, y)
  IQ_BY_FMT(down_fmt, CALL)
#undef CALL
  return launched_ok() ? IQ_OK : IQ_ERR_HIP;
}

}  // extern "C"
