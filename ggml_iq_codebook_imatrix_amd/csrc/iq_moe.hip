// iq_moe.hip -- iq_moe: a mixture-of-experts layer on encoded experts
// (include/iq_run.h).
//
// route_kernel brings the tokens into operand order, converts the codebooks and
// forms the router's logits in fp64.  For up to 8 tokens (and 256 experts) a
// launch costs more than picking the top_k does, so every workgroup of the next
// kernel picks them itself; for more, the choice is a launch of its own.  Up to
// 16 tokens a workgroup takes the expert of its rank among the chosen ones; for
// more it is given an expert, whose pairs it gathers from the ids.
//
// One token through 128 experts of 2,048 x 768 (eight of them, 9.7 MB of payload)
// takes 29 us: routing 5.5, gate and up 13 (2 of them the choice), down 10.  Each is
// a chain of waits: the launch, the logits, the payload, the sums.
//
// Gate and up (h in fp32, one row per pair):
//  up_split_kernel  16 rows of gate and up, the blocks of K split over the waves:
//                   where the chosen experts' rows alone would not fill the chip.
//  up_rows_kernel   128 rows, each wave 16 of them over the whole of K.
// Down:
//  down_split_kernel  16 columns of y; the (expert, block) pairs split over the
//                   waves, experts added up in the accumulators: no further launch.
//  down_rows_kernel 256 columns of one expert for the pairs routed to it, h
//                   converted once into LDS; sum_kernel adds each token's rows in
//                   the order of its ids.

#include <type_traits>

#include "iq_run.hpp"

namespace iq {
namespace {

// h is held as the sum of two fp16 values, for tokens of either type: one value's
// 2^-12 would change one bf16 output in twenty by a step.  The second costs matrix
// instructions beside the same decode: bf16, 1 token 28.7 us and 26.9 with one
// value, 64 tokens 106 and 101, 200 tokens 162 and 153.
constexpr int kHParts = 2;
constexpr int kFewTokens = 16, kFewExperts = 256, kMaxTopK = 64;

struct MoeArgs {
  const uint8_t *gate, *up, *down;
  int64_t hidden, inter;
  int E, top_k, renorm, pick;  // pick: few tokens' top_k is picked by the up kernel
  int64_t T, npair;
  const void *x, *router;
  int dtype, rdtype;
  Tokens X;
  const _Float16 *tab, *dtab;
  double *logits;          // [ks][T, E], sums over parts of K
  int ks;
  int32_t *ids;
  float *weights;
  float *h;                // [pairs, inter]
  float *z;                // [pairs, hidden] (down_rows_kernel)
  void *y;
  int32_t *status;
  Codebooks books;
  int64_t nconv;
};

// ---------------------------------------------------------------------------
// Routing
// ---------------------------------------------------------------------------
typedef double f64x4 __attribute__((ext_vector_type(4)));

// The logits of 16 tokens and 16 experts on the fp64 matrix cores, K split over
// ks workgroups (whose sums the choice adds) and each one's eight waves.  In fp64,
// so that the order of summation, which is the same for every expert, decides only
// between logits within 2 hidden 2^-53 of their terms' sum (5.5 us for up to 64 tokens by 128
// experts of 2,048, 8 for 200: latency).  v_mfma_f64_16x16x4: lane l holds k = l / 16
// of token (A) and expert (B) l % 16; D has lane l hold expert l % 16 and tokens l / 16 + 4 i.
template <int P>
__device__ __forceinline__ void route_logits(const MoeArgs &A, int64_t w, double *s_red) {
  constexpr int U = 4;  // loads in flight
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ne = (A.E + 15) / 16, ks = static_cast<int>(w % A.ks);
  const int b0 = static_cast<int>((A.hidden >> 8) * ks / A.ks), nb = static_cast<int>((A.hidden >> 8) * (ks + 1) / A.ks);
  w /= A.ks;
  const int64_t t0 = w / ne * 16, e0 = w % ne * 16;
  const int64_t k0 = wave * 32 + (lane >> 4) * 8;  // 32 of each 256 columns
  const int64_t xr = min(t0 + (lane & 15), A.T - 1) * A.hidden + k0;
  const int64_t rr = min(e0 + (lane & 15), static_cast<int64_t>(A.E) - 1) * A.hidden + k0;
  f64x4 acc = {0.0, 0.0, 0.0, 0.0};
  for (int b = b0; b < nb; b += U) {
    float x[U][8], r[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = min(b + u, nb - 1) * 256;
      load8u(A.x, P == 1, xr + at, x[u]);
      load8u(A.router, A.rdtype, rr + at, r[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (b + u < nb)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          acc = __builtin_amdgcn_mfma_f64_16x16x4f64(static_cast<double>(x[u][i]), static_cast<double>(r[u][i]), acc,
                                                     0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) s_red[(wave * 4 + i) * 64 + lane] = acc[i];
  __syncthreads();
  if (threadIdx.x < 256) {
    const int i = threadIdx.x >> 6;
    double s = s_red[i * 64 + lane];
    for (int v = 1; v < 8; ++v) s += s_red[(v * 4 + i) * 64 + lane];
    const int64_t t = t0 + (lane >> 4) + 4 * i, e = e0 + (lane & 15);
    if (t < A.T && e < A.E) A.logits[(ks * A.T + t) * A.E + e] = s;
  }
}

template <int P>
__global__ void __launch_bounds__(512) route_kernel(MoeArgs A) {
  __shared__ double s_red[8 * 4 * 64];
  int64_t w = blockIdx.x;
  if (w < A.nconv) {
    const int64_t t = w * 8 + (threadIdx.x >> 6);
    if (t < A.T) convert_token<P>(A.x, A.hidden, A.X, t, threadIdx.x & 63);
    return;
  }
  w -= A.nconv;
  if (w < A.books.wg[0] + A.books.wg[1]) {
    convert_codebook(A.books, static_cast<int>(w));
    return;
  }
  route_logits<P>(A, w - A.books.wg[0] - A.books.wg[1], s_red);
}

// fp64 as a whole number of the same order, from 1 (NaN) up; 0: taken
__device__ __forceinline__ uint64_t order_key(double v) {
  if (v != v) return 1;
  const int64_t b = __builtin_bit_cast(int64_t, v + 0.0);  // -0 as 0
  return b < 0 ? ~static_cast<uint64_t>(b) : static_cast<uint64_t>(b) | (uint64_t(1) << 63);
}
__device__ __forceinline__ double key_value(uint64_t k) {
  if (k == 1) return __builtin_nan("");
  return __builtin_bit_cast(double, (k >> 63) ? k & ~(uint64_t(1) << 63) : ~k);
}

// One wave picks a token's top_k (at most 64): largest logit first, equal ones
// by id, NaN last.  Lane l holds experts l + 64 j; a round finds the largest
// upper half by register permutes and looks at lower halves and ids only where
// several lanes tie.  ids, weights: where the token's choice goes.
template <int KPL>
__device__ __forceinline__ void pick_top(const MoeArgs &A, int64_t t, int32_t *ids, float *weights) {
  const int lane = threadIdx.x & 63, E = A.E, top_k = A.top_k;
  const double *l = A.logits + t * E;
  const auto logit = [&](int e) {
    double s = l[e];
    for (int k = 1; k < A.ks; ++k) s += l[k * A.T * E + e];
    return s;
  };
  uint64_t key[KPL];
#pragma unroll
  for (int j = 0; j < KPL; ++j) {
    const int e = lane + 64 * j;
    key[j] = e < E ? order_key(logit(e)) : 0;
  }
  double top = 0.0, mine = 0.0;
  int my_id = 0;
  for (int s = 0; s < top_k; ++s) {
    uint64_t best = key[0];
    int bj = 0;
#pragma unroll
    for (int j = 1; j < KPL; ++j)
      if (key[j] > best) {
        best = key[j];
        bj = j;
      }
    const uint32_t hi = static_cast<uint32_t>(best >> 32), lo = static_cast<uint32_t>(best);
    const uint32_t mhi = wave_max_u32(hi);
    uint64_t who = __ballot(hi == mhi);
    if (who & (who - 1)) {
      const uint32_t mlo = wave_max_u32(hi == mhi ? lo : 0u);
      const bool tied = hi == mhi && lo == mlo;
      who = __ballot(tied);
      if (who & (who - 1)) {  // the lowest id: the largest 4095 - id
        const uint32_t id = 4095u - static_cast<uint32_t>(lane + 64 * bj);
        const uint32_t mid = wave_max_u32(tied ? id : 0u);
        who = __ballot(tied && id == mid);
      }
    }
    const int from = static_cast<int>(__builtin_ctzll(who));
    const uint64_t won = (static_cast<uint64_t>(__builtin_amdgcn_readlane(static_cast<int>(hi), from)) << 32) |
                         static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(lo), from));
    const int wj = __builtin_amdgcn_readlane(bj, from);
#pragma unroll
    for (int j = 0; j < KPL; ++j)
      if (lane == from && j == wj) key[j] = 0;
    const double v = key_value(won);
    if (s == 0) top = v;
    if (lane == s) {
      mine = v;
      my_id = from + 64 * wj;
    }
  }
  const float p = lane < top_k ? expf(static_cast<float>(mine - top)) : 0.0f;
  float sum = p;
  if (!A.renorm) {
    sum = 0.0f;
    for (int e = lane; e < E; e += 64) sum += expf(static_cast<float>(logit(e) - top));
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o, 64);
  if (lane < top_k) {
    ids[lane] = my_id;
    weights[lane] = p / sum;
  }
}

__global__ void __launch_bounds__(64) topk_kernel(MoeArgs A) {
  const int64_t t = blockIdx.x;
  if (A.E <= 128)
    pick_top<2>(A, t, A.ids + t * A.top_k, A.weights + t * A.top_k);
  else if (A.E <= 256)
    pick_top<4>(A, t, A.ids + t * A.top_k, A.weights + t * A.top_k);
  else
    pick_top<64>(A, t, A.ids + t * A.top_k, A.weights + t * A.top_k);
}

// The four of a block's values whose place in the operand is the lane's: elements
// 4 (lane % 2) .. + 3 of group lane / 2.
__device__ __forceinline__ void load_h(const float *h, int lane, float v[4]) {
  const float *p = h + (lane >> 1) * 8 + (lane & 1) * 2;
  const float2 a = *reinterpret_cast<const float2 *>(p), b = *reinterpret_cast<const float2 *>(p + 4);
  v[0] = a.x;
  v[1] = b.x;
  v[2] = a.y;
  v[3] = b.y;
}

__device__ __forceinline__ float gated(float g, float u, float w) { return g / (1.0f + expf(-g)) * u * w; }

// ---------------------------------------------------------------------------
// The pairs of an expert
// ---------------------------------------------------------------------------
// What a workgroup knows of the routing of few tokens.
struct FewPairs {
  int ids[kFewTokens * kMaxTopK];   // the pairs' experts (-1: none)
  int list[kFewTokens * kMaxTopK];  // the pairs of this workgroup's expert, ascending
  float w[kFewTokens * kMaxTopK];
  uint32_t bits[kFewExperts / 32];  // the experts that occur
  int n;
};

// The pairs' experts into LDS: picked here from the logits, or read.
__device__ __forceinline__ void few_ids(const MoeArgs &A, FewPairs &S, bool pick) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), nw = blockDim.x >> 6;
  const int np = static_cast<int>(A.npair);
  if (threadIdx.x < kFewExperts / 32) S.bits[threadIdx.x] = 0;
  if (pick) {
    for (int t = wave; t < A.T; t += nw) {
      if (A.E <= 128)
        pick_top<2>(A, t, S.ids + t * A.top_k, S.w + t * A.top_k);
      else
        pick_top<4>(A, t, S.ids + t * A.top_k, S.w + t * A.top_k);
    }
  } else {
    for (int p = threadIdx.x; p < np; p += blockDim.x) {
      const int e = A.ids[p];
      const bool bad = e < 0 || e >= A.E;
      if (bad && blockIdx.x == 0) raise_status(A.status, ST_BADID);
      S.ids[p] = bad ? -1 : e;
      S.w[p] = A.weights[p];
    }
  }
  __syncthreads();
  for (int p = threadIdx.x; p < np; p += blockDim.x) {
    if (pick && blockIdx.x == 0) {
      A.ids[p] = S.ids[p];
      A.weights[p] = S.w[p];
    }
    if (S.ids[p] >= 0) atomicOr(&S.bits[S.ids[p] >> 5], 1u << (S.ids[p] & 31));
  }
  __syncthreads();
}

// The expert of rank `slot` among those that occur, and its pairs; -1: there are not as many.
__device__ __forceinline__ int few_expert(const MoeArgs &A, FewPairs &S, int slot) {
  const int lane = threadIdx.x & 63, np = static_cast<int>(A.npair);
  int e = -1;
#pragma unroll
  for (int i = 0; i < kFewExperts / 32; ++i) {
    uint32_t bits = __builtin_amdgcn_readfirstlane(S.bits[i]);
    const int c = __builtin_popcount(bits);
    if (e < 0 && slot < c) {
      for (int k = 0; k < slot; ++k) bits &= bits - 1;
      e = i * 32 + __builtin_ctz(bits);
    }
    if (e < 0) slot -= c;
  }
  if (e < 0) return -1;
  if (threadIdx.x < 64) {
    int n = 0;
    for (int p0 = 0; p0 < np; p0 += 64) {
      const bool hit = p0 + lane < np && S.ids[p0 + lane] == e;
      const uint64_t b = __ballot(hit);
      if (hit) S.list[n + __builtin_popcountll(b & ((uint64_t(1) << lane) - 1))] = p0 + lane;
      n += __builtin_popcountll(b);
    }
    if (lane == 0) S.n = n;
  }
  __syncthreads();
  return e;
}

// 16 rows of gate and up of one expert a row group, K split over its waves
// (split_blocks); h of its pairs.  For few experts' rows: the small layer (8 experts
// of 512 x 256, 5 tokens, float32) 9 us, with whole rows 11.
template <int F, int P>
__global__ void __launch_bounds__(512) up_split_kernel(MoeArgs A) {
  __shared__ uint4 s_tab[Geo<F>::N];
  __shared__ f32x4 s_red[8 * 2 * 64];
  __shared__ FewPairs S;
  load_table<F>(s_tab, A.tab);
  const int64_t nb = A.hidden >> 8, rowbytes = nb * Geo<F>::BYTES, stride = A.X.ntile * P * 4096;
  const Split W = split_of(nb);
  const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4, tiles = static_cast<int>(A.inter >> 4);
  const int per = (tiles + W.rw - 1) / W.rw, tile0 = static_cast<int>(blockIdx.x % per) * W.rw;
  few_ids(A, S, A.pick);
  const int e = few_expert(A, S, static_cast<int>(blockIdx.x / per));
  if (e < 0) return;
  const int64_t row = e * A.inter + min(tile0 + W.rg, tiles - 1) * 16 + n;
  for (int c0 = 0; c0 < S.n; c0 += 16) {
    const int *list = S.list + c0;
    const int count = min(16, S.n - c0);
    const int64_t t = list[min(n, count - 1)] / A.top_k;
    const _Float16 *x0 = A.X.x16 + (t >> 4) * P * 4096 + (q * 16 + (t & 15)) * 8;
    f32x4 acc[1][2][1] = {};
    split_blocks<F, P, 1, 1, 2>(
        nb, W, s_tab, [&](int m, int) { return (m ? A.up : A.gate) + row * rowbytes; },
        [&](int64_t b, Operand<P, 1> &x) __attribute__((always_inline)) {
          const _Float16 *const xp[1] = {x0 + b * stride};
          load_operand<P, 1>(x, xp);
        },
        acc);
    // the sums over a row group's waves, then h
#pragma unroll
    for (int j = 0; j < 2; ++j) s_red[((W.rg * W.kw + W.kg) * 2 + j) * 64 + lane] = acc[0][j][0];
    __syncthreads();
    for (int i = threadIdx.x; i < W.rw * 64; i += blockDim.x) {
      const int rg = i / 64, l = i & 63, tile = tile0 + rg;
      if (tile >= tiles) continue;
      const f32x4 *p = s_red + rg * W.kw * 2 * 64 + l;
      f32x4 g = p[0], u = p[64];
      for (int k = 1; k < W.kw; ++k) {
        g += p[k * 2 * 64];
        u += p[(k * 2 + 1) * 64];
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int at = (l >> 4) * 4 + k;
        if (at >= count) continue;
        const int64_t pair = list[at];
        const int ex = A.X.ex[pair / A.top_k];
        A.h[pair * A.inter + tile * 16 + (l & 15)] = gated(ldexpf(g[k], ex), ldexpf(u[k], ex), S.w[pair]);
      }
    }
    __syncthreads();  // the sums' memory is free again
  }
}

// Waves split (expert, block of inter): each stages its tokens' h of that block
// as the A operand (rows: tokens; absent ones zero) in LDS of its own.  One token
// through eight experts of 2,048 x 768: 10 us, latency.
constexpr int down_split_waves(int fmt) { return fmt >= IQ1_S ? 4 : 8; }  // 16 KiB of LDS a wave, beside the codebook
template <int F>
__global__ void __launch_bounds__(64 * down_split_waves(F)) down_split_kernel(MoeArgs A) {
  constexpr int NW = down_split_waves(F);
  __shared__ uint4 s_tab[Geo<F>::N];
  __shared__ uint4 s_x[NW][kHParts * 512];  // also the sums over the waves
  __shared__ int s_ex[NW][16], s_active[kFewExperts];
  __shared__ FewPairs S;
  load_table<F>(s_tab, A.dtab);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int np = static_cast<int>(A.npair), n = lane & 15, q = lane >> 4;
  for (int i = lane; i < kHParts * 512; i += 64) s_x[wave][i] = make_uint4(0, 0, 0, 0);
  if (lane < 16) s_ex[wave][lane] = 0;
  few_ids(A, S, false);
  int na = 0;
#pragma unroll
  for (int i = 0; i < kFewExperts / 32; ++i) {
    const uint32_t bits = __builtin_amdgcn_readfirstlane(S.bits[i]);
    if (wave == 0 && lane < 32 && ((bits >> lane) & 1u))
      s_active[na + __builtin_popcount(bits & ((1u << lane) - 1u))] = i * 32 + lane;
    na += __builtin_popcount(bits);
  }
  __syncthreads();
  const int nb = static_cast<int>(A.inter >> 8);
  const int64_t col0 = static_cast<int64_t>(blockIdx.x) * 16;
  _Float16 *xs = reinterpret_cast<_Float16 *>(&s_x[wave][0]);
  const int at = (((lane & 15) >> 1) * 64 + q * 16) * 8 + (lane & 1) * 4;  // the lane's place, token 0
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int task = wave; task < na * nb; task += NW) {
    const int e = __builtin_amdgcn_readfirstlane(s_active[task / nb]), b = task % nb;
    const Words words = load_words<F>(A.down + ((e * A.hidden + col0 + n) * nb + b) * Geo<F>::BYTES, q);
    uint32_t present = 0;
    const auto stage = [&](int t, const float *v) {  // token t's h: one wave, four columns a lane
      uint32_t x = 1;
#pragma unroll
      for (int j = 0; j < 4; ++j) x = max_exponent(x, v[j]);
      const int up = 141 - static_cast<int>(wave_max_u32(x));
      _Float16 hi[4], lo[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) to_parts(v[j], up, hi[j], lo[j]);
      *reinterpret_cast<uint2 *>(xs + at + t * 8) = __builtin_bit_cast(uint2, hi);
      *reinterpret_cast<uint2 *>(xs + 4096 + at + t * 8) = __builtin_bit_cast(uint2, lo);
      if (lane == 0) s_ex[wave][t] = -up;
      present |= 1u << t;
    };
    float v[4] = {};
    int token = -1;
    for (int p0 = 0; p0 < np; p0 += 64) {
      uint64_t hits = __ballot(p0 + lane < np && S.ids[p0 + lane] == e);
      while (hits) {
        const int p = p0 + static_cast<int>(__builtin_ctzll(hits));
        hits &= hits - 1;
        const int t = p / A.top_k;
        if (t != token) {  // an expert named twice by a token: its rows are added
          if (token >= 0) stage(token, v);
          token = t;
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = 0.0f;
        }
        float f[4];
        load_h(A.h + p * A.inter + b * 256, lane, f);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += f[j];
      }
    }
    stage(token, v);
    const _Float16 *const xp[1] = {xs + lane * 8};
    Raw raw[1];
    raw[0] = unpack<F>(words, q);
    f32x4 part[1][1];
    block_mma<F, kHParts, 1, 1>(raw, s_tab, xp, part);
    const float d = block_scale<F>(raw[0]);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if ((present >> (q * 4 + k)) & 1u) acc[k] += ldexpf(d * part[0][0][k], s_ex[wave][q * 4 + k]);
    for (uint32_t m = present; m; m &= m - 1) {  // leave the rows zero again
      const int t = __builtin_ctz(m);
      *reinterpret_cast<uint2 *>(xs + at + t * 8) = make_uint2(0, 0);
      *reinterpret_cast<uint2 *>(xs + 4096 + at + t * 8) = make_uint2(0, 0);
    }
  }
  const Split W{NW, 1, wave, 0};
  reduce_split<1, 1>(&acc, reinterpret_cast<f32x4 *>(&s_x[0][0]), W, [&](int, int, int l, const f32x4 &s) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int t = (l >> 4) * 4 + k;
      if (t < A.T) store1(A.y, A.dtype, t * A.hidden + col0 + (l & 15), s[k]);
    }
  });
}

// Walks the pairs of one expert in ascending order, N at a time: f(list, count).
// The ids are searched, a workgroup's width at a time.
template <int N> struct PairWalk {
  int list[512 + N], cnt[8];  // up to eight waves
};
template <int N, class Fn>
__device__ __forceinline__ void for_pairs(const MoeArgs &A, int e, PairWalk<N> &S, Fn f) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nw = blockDim.x >> 6;
  int have = 0;
  for (int64_t p0 = 0; p0 < A.npair; p0 += blockDim.x) {
    const int64_t p = p0 + threadIdx.x;
    const bool hit = p < A.npair && A.ids[p] == e;
    const uint64_t b = __ballot(hit);
    if (lane == 0) S.cnt[wave] = __builtin_popcountll(b);
    __syncthreads();
    int at = have, total = 0;
    for (int w = 0; w < nw; ++w) {
      const int c = S.cnt[w];
      if (w < wave) at += c;
      total += c;
    }
    if (hit) S.list[at + __builtin_popcountll(b & ((uint64_t(1) << lane) - 1))] = static_cast<int>(p);
    have += total;
    __syncthreads();
    const bool last = p0 + blockDim.x >= A.npair;
    int head = 0;
    while (have - head >= N || (last && have > head)) {
      f(S.list + head, min(N, have - head));
      head += min(N, have - head);
    }
    if (head) {  // what is left moves to the front
      const int rest = have - head;
      int keep = 0;
      if (static_cast<int>(threadIdx.x) < rest) keep = S.list[head + threadIdx.x];
      __syncthreads();
      if (static_cast<int>(threadIdx.x) < rest) S.list[threadIdx.x] = keep;
      have = rest;
      __syncthreads();
    }
  }
}

// 16 NW rows of gate and up of one expert: NW waves, 16 rows each over the whole
// of K.  The pairs' tokens come through LDS, KC blocks at a time for all waves;
// a wave keeps the payload of the next two blocks on its way in registers (with
// one, waiting for HBM was a third of the time).  64 tokens through 128 experts of
// 2,048 x 768, IQ2_XXS: 51 us for 102 MB of payload (2.0 TB/s).  The decode bounds it:
// 19,400 vector instructions a SIMD at 4.9 cycles are 0.85 of its time, LDS is busy
// 0.45 of it.  Sharing the blocks of K between the waves instead took 119 us: every
// wave then reads all tokens from memory.
template <int F, int P, int C, int NW, bool FEW>
__global__ void __launch_bounds__(64 * NW, NW == 4 ? 2 / P : P * C == 1 ? 4 : 2) up_rows_kernel(MoeArgs A) {
  constexpr int N = 16 * C, KC = C * P >= 4 ? 1 : 2, kUnits = 512 / (64 * NW), XU = KC * C * P * kUnits;
  __shared__ uint4 s_tab[Geo<F>::N];
  __shared__ u32x4 s_x[2][XU * 64 * NW];
  __shared__ typename std::conditional<FEW, FewPairs, PairWalk<N>>::type S;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, q = lane >> 4;
  const int64_t nb = A.hidden >> 8, per = A.inter / (16 * NW), part = blockIdx.x % per;
  int e = static_cast<int>(blockIdx.x / per);
  load_table<F>(s_tab, A.tab);
  if constexpr (FEW) {
    few_ids(A, S, A.pick);
    e = few_expert(A, S, e);
    if (e < 0) return;
  }
  const int64_t col = part * 16 * NW + wave * 16 + n, row = e * A.inter + col;
  const uint8_t *rp[2] = {A.gate + row * nb * Geo<F>::BYTES, A.up + row * nb * Geo<F>::BYTES};
  Words words[3][2];  // the block in hand and the next two
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int r = 0; r < 2; ++r) words[k][r] = load_words<F>(rp[r] + min(static_cast<int64_t>(k), nb - 1) * Geo<F>::BYTES, q);
  bool fresh = true;
  const auto body = [&](const int *list, int count) __attribute__((always_inline)) {
    if (!fresh) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          words[k][r] = load_words<F>(rp[r] + min(static_cast<int64_t>(k), nb - 1) * Geo<F>::BYTES, q);
    }
    fresh = false;
    const int m = threadIdx.x & 15;  // a thread copies the same row of every tile
    int64_t from[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t t = list[min(c * 16 + m, count - 1)] / A.top_k;
      from[c] = (t >> 4) * P * 512 + (threadIdx.x & ~15) + (t & 15);
    }
    u32x4 xr[XU];
    // unit i: part i / kUnits of the chunk's [block][tile][part] 8 KiB pieces
    const auto load_x = [&](int64_t b0) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < XU; ++i) {
        const int piece = i / kUnits, c = piece / P % C;
        const int64_t b = min(b0 + piece / (C * P), nb - 1);
        if (c * 16 + m < count)
          xr[i] = reinterpret_cast<const u32x4 *>(
              A.X.x16)[b * A.X.ntile * P * 512 + piece % P * 512 + i % kUnits * (64 * NW) + from[c]];
      }
    };
    const auto store_x = [&](u32x4 *to) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < XU; ++i)
        if (i / kUnits / P % C * 16 + m < count) to[i * 64 * NW + threadIdx.x] = xr[i];
    };
    f32x4 acc[2][C] = {};
    load_x(0);
    store_x(s_x[0]);
    int cur = 0;
    for (int64_t b0 = 0; b0 < nb; b0 += KC) {
      __syncthreads();  // the chunk is there, and the one before read
      if (b0 + KC < nb) load_x(b0 + KC);
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        const int64_t b = b0 + k;
        if (b >= nb) break;
#pragma unroll
        for (int r = 0; r < 2; ++r) words[2][r] = load_words<F>(rp[r] + min(b + 2, nb - 1) * Geo<F>::BYTES, q);
        __builtin_amdgcn_sched_barrier(0);  // the loads above go out before the work below, not after it
        const _Float16 *xp[C];
#pragma unroll
        for (int c = 0; c < C; ++c)
          xp[c] = reinterpret_cast<const _Float16 *>(s_x[cur] + (k * C + c) * P * 512 + lane);
        f32x4 sum[2][C];
        Raw raw[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) raw[r] = unpack<F>(words[0][r], q);
        block_mma<F, P, C, 2>(raw, s_tab, xp, sum);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
          for (int c = 0; c < C; ++c) scale_add(acc[r][c], sum[r][c], block_scale<F>(raw[r]));
          words[0][r] = words[1][r];
          words[1][r] = words[2][r];
        }
      }
      cur ^= 1;
      if (b0 + KC < nb) store_x(s_x[cur]);
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = c * 16 + q * 4 + k;
        if (i >= count) continue;
        const int64_t p = list[i];
        float w;
        if constexpr (FEW)
          w = S.w[p];
        else
          w = A.weights[p];
        const int ex = A.X.ex[p / A.top_k];
        A.h[p * A.inter + col] = gated(ldexpf(acc[0][c][k], ex), ldexpf(acc[1][c][k], ex), w);
      }
    __syncthreads();  // the tokens' memory and the list may change
  };
  if constexpr (FEW) {
    for (int c0 = 0; c0 < S.n; c0 += N) body(S.list + c0, min(N, S.n - c0));
  } else {
    for_pairs<N>(A, e, S, body);
  }
}

// 32 NW columns of y of one expert: NW waves, 32 columns each.  The pairs' h
// goes to LDS as the A operand, KB blocks at a time: a wave converts one pair's
// block, so the conversion is repeated only by an expert's hidden / (32 NW)
// workgroups.  z: one row per pair.  64 tokens as above: 36 us, the decode 0.75 of it.
template <int F, int C, int NW, bool FEW>
__global__ void __launch_bounds__(64 * NW, C == 1 ? 4 : 2) down_rows_kernel(MoeArgs A) {
  constexpr int N = 16 * C, KB = C == 4 ? 1 : 2;
  __shared__ uint4 s_tab[Geo<F>::N];
  __shared__ _Float16 s_h[KB][C][kHParts * 4096];
  __shared__ int s_ex[KB][N];
  __shared__ typename std::conditional<FEW, FewPairs, PairWalk<N>>::type S;
  load_table<F>(s_tab, A.dtab);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, q = lane >> 4;
  const int nb = static_cast<int>(A.inter >> 8);
  const int64_t per = A.hidden / (32 * NW), part = blockIdx.x % per;
  int e = static_cast<int>(blockIdx.x / per);
  if constexpr (FEW) {
    few_ids(A, S, false);
    e = few_expert(A, S, e);
    if (e < 0) return;
  }
  const int64_t col = part * 32 * NW + wave * 32 + n;
  const uint8_t *rp[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) rp[r] = A.down + (e * A.hidden + col + r * 16) * nb * Geo<F>::BYTES;
  Words words[3][2];  // the block in hand and the next two
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int r = 0; r < 2; ++r) words[k][r] = load_words<F>(rp[r] + min(k, nb - 1) * Geo<F>::BYTES, q);
  bool fresh = true;
  const auto body = [&](const int *list, int count) __attribute__((always_inline)) {
    f32x4 acc[2][C] = {};
    if (!fresh) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int r = 0; r < 2; ++r) words[k][r] = load_words<F>(rp[r] + min(k, nb - 1) * Geo<F>::BYTES, q);
    }
    fresh = false;
    for (int b0 = 0; b0 < nb; b0 += KB) {
      const int kb = min(KB, nb - b0);
      if (b0) __syncthreads();  // the blocks before are read
      for (int i = wave; i < count * kb; i += NW) {
        const int m = i / kb, j = i - m * kb;
        float v[4];
        load_h(A.h + list[m] * A.inter + (b0 + j) * 256, lane, v);
        uint32_t x = 1;
#pragma unroll
        for (int k = 0; k < 4; ++k) x = max_exponent(x, v[k]);
        const int up = 141 - static_cast<int>(wave_max_u32(x));
        _Float16 hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) to_parts(v[k], up, hi[k], lo[k]);
        _Float16 *o = &s_h[j][m >> 4][((n >> 1) * 64 + q * 16 + (m & 15)) * 8 + (n & 1) * 4];
        *reinterpret_cast<uint2 *>(o) = __builtin_bit_cast(uint2, hi);
        *reinterpret_cast<uint2 *>(o + 4096) = __builtin_bit_cast(uint2, lo);
        if (lane == 0) s_ex[j][m] = -up;
      }
      __syncthreads();
      for (int j = 0; j < kb; ++j) {
        const int bn = min(b0 + j + 2, nb - 1);
#pragma unroll
        for (int r = 0; r < 2; ++r) words[2][r] = load_words<F>(rp[r] + bn * Geo<F>::BYTES, q);
        __builtin_amdgcn_sched_barrier(0);  // the loads above go out before the work below, not after it
        const _Float16 *xp[C];
#pragma unroll
        for (int c = 0; c < C; ++c) xp[c] = &s_h[j][c][lane * 8];
        f32x4 sum[2][C];
        Raw raw[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) raw[r] = unpack<F>(words[0][r], q);
        block_mma<F, kHParts, C, 2>(raw, s_tab, xp, sum);
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int ex = s_ex[j][c * 16 + q * 4 + k];  // past count: of rows not stored
#pragma unroll
            for (int r = 0; r < 2; ++r) acc[r][c][k] += ldexpf(block_scale<F>(raw[r]) * sum[r][c][k], ex);
          }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          words[0][r] = words[1][r];
          words[1][r] = words[2][r];
        }
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = c * 16 + q * 4 + k;
        if (i >= count) continue;
        const int64_t p = list[i];
#pragma unroll
        for (int r = 0; r < 2; ++r) A.z[p * A.hidden + col + r * 16] = acc[r][c][k];
      }
    __syncthreads();  // s_h is free again
  };
  if constexpr (FEW) {
    for (int c0 = 0; c0 < S.n; c0 += N) body(S.list + c0, min(N, S.n - c0));
  } else {
    for_pairs<N>(A, e, S, body);
  }
}

// y[t] = the sum of its pairs' rows, in the order of its ids: no atomics, so that
// a call repeats bit for bit (4 to 5 us, a launch).
__global__ void __launch_bounds__(256) sum_kernel(MoeArgs A) {
  const int64_t per = A.hidden / 4, i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= A.T * per) return;
  const int64_t t = i / per, c = (i - t * per) * 4;
  float s[4] = {};
  for (int k0 = 0; k0 < A.top_k; k0 += 8) {  // eight rows in flight
    float4 v[8];
    bool ok[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t p = t * A.top_k + min(k0 + k, A.top_k - 1);
      v[k] = *reinterpret_cast<const float4 *>(A.z + p * A.hidden + c);
      const int e = A.ids[p];
      ok[k] = e >= 0 && e < A.E;  // a pair without an expert has no row
      if (!ok[k] && c == 0) raise_status(A.status, ST_BADID);
      ok[k] = ok[k] && k0 + k < A.top_k;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      s[0] += ok[k] ? v[k].x : 0.0f;
      s[1] += ok[k] ? v[k].y : 0.0f;
      s[2] += ok[k] ? v[k].z : 0.0f;
      s[3] += ok[k] ? v[k].w : 0.0f;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) store1(A.y, A.dtype, t * A.hidden + c + j, s[j]);
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
// The rules below, measured with 128 experts of 2,048 x 768, eight a token, bf16,
// unless another layer is named.
//
// Few tokens name few experts: a workgroup per chosen expert, not per expert (1
// token 26 us and 49, 8 tokens 59 and 71, 16 tokens 73 and 84).  Past 256 experts a
// launch takes all of them (1 token: 256 experts 32 us, 512 127).
bool is_few(int64_t T, int E) { return T <= kFewTokens && E <= kFewExperts; }
// A wave picks a token's experts in 2 us, a launch for it takes 4 to 5 and as much
// of the host's time: picked in the next kernel while its eight waves do it in one
// go (8 tokens 59 us and 58, 9 tokens 63 and 58, 16 tokens 94 and 74).
bool is_pick(int64_t T, int E) { return T <= 8 && E <= kFewExperts; }
// Experts that np pairs reach at most.
int64_t reached(int64_t np, int E) { return np < E ? np : E; }
// Gate and up with K split over the waves, where whole rows would leave half of
// the 1,024 SIMDs without a wave: 384 row tiles 26 us and 30 with whole rows, 512
// (16 experts of 1,024 x 512, 16 tokens) 28 and 30, 768 38 and 36.
bool split_up(const MoeArgs &A) { return is_few(A.T, A.E) && reached(A.npair, A.E) * (A.inter / 16) <= 512; }
// Down with the (expert, block) pairs split over the waves, no launch for the sums:
// a wave converts every pair's block, so while these are few: 16 of them (16
// experts of 1,024 x 512, 4 tokens) 23 us and 26 with whole rows, 24 29 and 34, 48
// 41 and 40, 72 52 and 46.  The IQ1 codebooks leave LDS for half the waves: 16 of
// them 27 and 27, 24 34 and 35, 48 48 and 41.  Whole rows of few large experts leave
// CUs without work: two of eight experts of 4,096 x 14,336, one token, are 32
// workgroups, and the layer takes 174 us for 90 MB of payload.
bool split_down(int64_t T, int E, int top_k, int64_t inter, int down_fmt) {
  return is_few(T, E) && T * top_k * (inter / 256) <= (down_split_waves(down_fmt) == 4 ? 24 : 48);
}

struct MoePlan {
  TokensPlan x;
  int ks;
  size_t tab, dtab, xo, eo, lo, ho, zo, bytes;
};
MoePlan plan_moe(int fmt, int down_fmt, int64_t hidden, int64_t inter, int E, int dtype, int64_t T, int top_k) {
  MoePlan p;
  const size_t np = static_cast<size_t>(T) * top_k;
  p.x = plan_tokens(T, hidden, dtype);
  p.tab = 0;
  p.dtab = ws_up(static_cast<size_t>(kCodebook[fmt]) * 16);
  p.xo = p.dtab + ws_up(static_cast<size_t>(kCodebook[down_fmt]) * 16);
  p.eo = p.xo + ws_up(p.x.xbytes);
  p.lo = p.eo + ws_up(p.x.ebytes);
  p.ks = hidden >= 4 * 256 ? 4 : 1;  // eight workgroups alone would route 16 tokens to 128 experts: 3 to 5 us more
  p.ho = p.lo + ws_up(static_cast<size_t>(p.ks) * T * E * 8);
  p.zo = p.ho + ws_up(np * inter * 4);
  p.bytes = p.zo + ws_up(split_down(T, E, top_k, inter, down_fmt) ? 0 : np * hidden * 4) + kWsAlign;
  return p;
}

int check_moe(int fmt, int down_fmt, int64_t hidden, int64_t inter, int E, int dtype, int64_t T, int top_k) {
  if (run_bad_fmt(fmt) || run_bad_fmt(down_fmt)) return IQ_ERR_FMT;
  if (run_bad_dtype(dtype)) return IQ_ERR_DTYPE;
  if (T < 0 || hidden <= 0 || hidden % 256 != 0 || inter <= 0 || inter % 256 != 0) return IQ_ERR_SHAPE;
  if (hidden > (int64_t(1) << 24) || inter > (int64_t(1) << 24)) return IQ_ERR_SHAPE;
  if (E < 1 || E > 4096 || top_k < 1 || top_k > kMaxTopK) return IQ_ERR_ARG;
  const int64_t ntile = (T + 15) / 16, np = T * top_k;
  if (T > (int64_t(1) << 24)) return IQ_ERR_SHAPE;
  // pairs are counted in 32 bits; then the launches: routing, up, down, sum
  if (np >= (int64_t(1) << 31) - 1 || (T + 7) / 8 + 8 + ((E + 15) / 16) * ntile * 4 >= kMaxWG ||
      E * (inter / 128) >= kMaxWG || E * (hidden / 256) >= kMaxWG || T * (hidden / 4) / 512 >= kMaxWG)
    return IQ_ERR_SHAPE;
  return IQ_OK;
}

template <int F, int P, int C, int NW, bool FEW>
void launch_up_rows(const MoeArgs &A, int64_t experts, hipStream_t stream) {
  hipLaunchKernelGGL((up_rows_kernel<F, P, C, NW, FEW>), dim3(static_cast<unsigned>(experts * (A.inter / (16 * NW)))),
                     dim3(64 * NW), 0, stream, A);
}
template <int F, int C, int NW, bool FEW>
void launch_down_rows(const MoeArgs &A, int64_t experts, hipStream_t stream) {
  hipLaunchKernelGGL((down_rows_kernel<F, C, NW, FEW>),
                     dim3(static_cast<unsigned>(experts * (A.hidden / (32 * NW)))), dim3(64 * NW), 0, stream, A);
}
// Tiles of 16 pairs that a workgroup multiplies at once, by an expert's pairs on
// average: as many as most experts fill, since every pass decodes the rows again.
// Measured (128 experts of 2,048 x 768, IQ1_M): 12.5 pairs with one tile 173 us and
// 164 with two; 16 with two 200 and 204 with four; 31 with two 313 and 300 with
// four; 250 with two 2,152 and 1,822 with four.  Gate and up of float32 have no room
// for four.
int pair_tiles(int64_t npair, int64_t E) { return npair <= 8 * E ? 1 : npair <= 28 * E ? 2 : 4; }

template <int F, int P> void launch_up(const MoeArgs &A, hipStream_t stream) {
  const int64_t experts = reached(A.npair, A.E);
  const int pairs = pair_tiles(A.npair, A.E);
  if (split_up(A)) {
    const int64_t nb = A.hidden / 256, rows = split_rw(nb) * 16, per = (A.inter + rows - 1) / rows;
    hipLaunchKernelGGL((up_split_kernel<F, P>), dim3(static_cast<unsigned>(experts * per)),
                       dim3(static_cast<unsigned>(64 * split_kw(nb) * split_rw(nb))), 0, stream, A);
    return;
  }
  if (is_few(A.T, A.E))  // four waves: 8 tokens 59 us and 62 with eight, 9 tokens 58 and 64, 16 tokens 73 and 73
    launch_up_rows<F, P, 1, 4, true>(A, experts, stream);
  else if (pairs == 1)
    launch_up_rows<F, P, 1, 8, false>(A, A.E, stream);
  else if (P == 2 || pairs == 2)
    launch_up_rows<F, P, 2, 8, false>(A, A.E, stream);
  else if constexpr (P == 1)
    launch_up_rows<F, P, 4, 8, false>(A, A.E, stream);
}

template <int F> void launch_down(const MoeArgs &A, hipStream_t stream) {
  const int pairs = pair_tiles(A.npair, A.E);
  if (split_down(A.T, A.E, A.top_k, A.inter, F)) {
    hipLaunchKernelGGL((down_split_kernel<F>), dim3(static_cast<unsigned>(A.hidden / 16)),
                       dim3(64 * down_split_waves(F)), 0, stream, A);
    return;
  }
  if (is_few(A.T, A.E))
    launch_down_rows<F, 1, 8, true>(A, reached(A.npair, A.E), stream);
  else if (pairs == 1)
    launch_down_rows<F, 1, 8, false>(A, A.E, stream);
  else if (pairs == 2)
    launch_down_rows<F, 2, 8, false>(A, A.E, stream);
  else
    launch_down_rows<F, 4, 8, false>(A, A.E, stream);
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
  if (router && run_bad_dtype(router_dtype)) return IQ_ERR_DTYPE;
  if (!grid || !down_grid || (T && (!gate || !up || !down || !x || !ids || !weights || !y))) return IQ_ERR_NULL;
  if (router && top_k > num_experts) return IQ_ERR_ARG;
  if (T == 0) return IQ_OK;
  if ((reinterpret_cast<uintptr_t>(gate) | reinterpret_cast<uintptr_t>(up) | reinterpret_cast<uintptr_t>(down)) & 1)
    return IQ_ERR_ARG;
  const MoePlan P = plan_moe(fmt, down_fmt, hidden, inter, num_experts, dtype, T, top_k);
  if ((rc = run_check_ws(P.bytes, workspace, workspace_bytes)) != IQ_OK) return rc;
  char *base = ws_base(workspace);
  MoeArgs A{};
  A.gate = gate;
  A.up = up;
  A.down = down;
  A.hidden = hidden;
  A.inter = inter;
  A.E = num_experts;
  A.top_k = top_k;
  A.renorm = renormalize;
  A.pick = router != nullptr && is_pick(T, num_experts);
  A.T = T;
  A.npair = T * top_k;
  A.x = x;
  A.router = router;
  A.dtype = dtype;
  A.rdtype = router_dtype;
  A.X = Tokens{reinterpret_cast<_Float16 *>(base + P.xo), reinterpret_cast<int32_t *>(base + P.eo), P.x.ntile};
  _Float16 *tab = reinterpret_cast<_Float16 *>(base + P.tab), *dtab = reinterpret_cast<_Float16 *>(base + P.dtab);
  A.tab = tab;
  A.dtab = dtab;
  A.logits = reinterpret_cast<double *>(base + P.lo);
  A.ks = P.ks;
  A.ids = ids;
  A.weights = weights;
  A.h = reinterpret_cast<float *>(base + P.ho);
  A.z = reinterpret_cast<float *>(base + P.zo);
  A.y = y;
  A.status = status;
  A.books = one_codebook(fmt, grid, tab, status);
  const Codebooks second = one_codebook(down_fmt, down_grid, dtab, status);
  A.books.grid[1] = second.grid[0];
  A.books.tab[1] = second.tab[0];
  A.books.n[1] = second.n[0];
  A.books.iq1[1] = second.iq1[0];
  A.books.wg[1] = second.wg[0];
  A.nconv = (T + 7) / 8;
  const int64_t nroute = router ? ((num_experts + 15) / 16) * P.x.ntile * P.ks : 0;
  const dim3 wgs(static_cast<unsigned>(A.nconv + A.books.wg[0] + A.books.wg[1] + nroute));
  if (dtype == IQ_DTYPE_F32)
    hipLaunchKernelGGL(route_kernel<2>, wgs, dim3(512), 0, stream, A);
  else
    hipLaunchKernelGGL(route_kernel<1>, wgs, dim3(512), 0, stream, A);
  if (!run_launched()) return IQ_ERR_HIP;
  if (router && !A.pick) {
    hipLaunchKernelGGL(topk_kernel, dim3(static_cast<unsigned>(T)), dim3(64), 0, stream, A);
    if (!run_launched()) return IQ_ERR_HIP;
  }
#define CALL(F) dtype == IQ_DTYPE_F32 ? launch_up<F, 2>(A, stream) : launch_up<F, 1>(A, stream)
  IQ_BY_FMT(fmt, CALL)
#undef CALL
  if (!run_launched()) return IQ_ERR_HIP;
#define CALL(F) launch_down<F>(A, stream)
  IQ_BY_FMT(down_fmt, CALL)
#undef CALL
  if (!run_launched()) return IQ_ERR_HIP;
  if (!split_down(T, num_experts, top_k, inter, down_fmt)) {
    hipLaunchKernelGGL(sum_kernel, dim3(static_cast<unsigned>((T * (hidden / 4) + 255) / 256)), dim3(256), 0,
                       stream, A);
    if (!run_launched()) return IQ_ERR_HIP;
  }
  return IQ_OK;
}

}  // extern "C"
