// iq_glu.hip -- iq_glu and iq_glu_backward: a gated feed-forward block's two
// projections, activation and product on encoded weights (include/iq_train.h).
//
// Forward, two launches: tokens and codebook into operand order, then both
// products, whose sums meet in registers and leave as h.  Backward, three (four
// where few tokens split the rows): the same product, whose sums leave as the
// gradients by g and u in the operand order of the product over rows (iq_rows.hip)
// that gives dx.

#include <type_traits>

#include "iq_train.hpp"

namespace iq {
namespace {

struct GluArgs {
  const uint8_t *packed[2];  // gate, up
  int64_t rows, nb, T;
  const _Float16 *tab;
  Tokens X;
  int act, dtype;
  void *h;
  // backward (dh not null)
  const void *dh;
  Grads G;
};

struct GluPrepArgs {
  Source S;
  int64_t T, cols, nconv;
  Tokens X;
  Codebooks books;
  // backward: the bound on the weights; the products find the largest of their gradients from zero on
  int fmt, bytes, backward;
  const uint8_t *packed[2];
  int64_t rows;
  Bound B;
  uint32_t *most;
};

// Everything the products want beforehand, a wave a token: 4,096 tokens x 5,120 in bf16 20 us (63 MB, 3.1 TB/s: a token's
// largest magnitude has to be known before its first value is written); backward, of a checkpoint, 36, which reads the
// payloads' block scales for their bound as well.
__global__ void __launch_bounds__(512) glu_prep_kernel(GluPrepArgs A) {
  __shared__ uint32_t s_red[8];
  int64_t w = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (A.backward) {
    if (w < kScaleSlots) {
      bound_scales(A.fmt, A.bytes, A.packed, 2, A.rows * (A.cols >> 8), A.B, static_cast<int>(w), s_red);
      return;
    }
    w -= kScaleSlots;
  }
  if (w < A.nconv) {
    const int64_t t = w * 8 + wave;
    if (t >= A.T) return;
    if (A.backward && lane == 0) A.most[t] = 0;
    if (A.S.ex)
      convert_checkpoint(static_cast<const int8_t *>(A.S.x), A.S.ex, A.cols, A.X, t, lane);
    else if (A.S.dtype == IQ_DTYPE_F32)
      convert_token<2>(A.S.x, A.cols, A.X, t, lane);
    else
      convert_token<1>(A.S.x, A.cols, A.X, t, lane);
    return;
  }
  w -= A.nconv;
  convert_codebook(A.books, static_cast<int>(w));
  if (A.backward) bound_codebook(A.books, A.B, static_cast<int>(w), s_red);
}

// ---------------------------------------------------------------------------
// Activations
// ---------------------------------------------------------------------------
// act(g), and with `back` its derivative in slope.  exp as a power of two (2^-23 |z| of its value) and one reciprocal
// (an ulp) leave a sigmoid s within 2^-24 |z| s (1 - s) and an ulp.  A sigmoid of 0 or 1 leaves no 0 * inf.
__device__ __forceinline__ float activation(int act, float g, bool back, float &slope) {
  slope = 0.0f;
  if (act == IQ_ACT_GELU) {
    const float phi = 0.5f * erfcf(-0.70710678f * g);
    if (back) slope = phi + g * (0.39894228f * expf(-0.5f * g * g));
    return g * phi;
  }
  float z = g, dz = 1.0f;
  if (act == IQ_ACT_GELU_TANH) {  // (1 + tanh(y)) / 2 is the sigmoid of 2 y
    constexpr float c = 1.5957691f, a = 0.044715f;
    const float g2 = g * g;
    z = c * (g + a * g * g2);
    dz = c * (1.0f + 3.0f * a * g2);
  }
  const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * z));
  if (back) {
    const float r = s * (1.0f - s);
    slope = s + (r == 0.0f ? 0.0f : g * r * dz);
  }
  return g * s;
}

// ---------------------------------------------------------------------------
// Results
// ---------------------------------------------------------------------------
// One value of h, or of both gradients, whose largest magnitude's bits are the result.  (dh meets u and the slope last: a
// dh * u that is infinite would make NaN of a slope of zero.)
__device__ __forceinline__ uint32_t put1(const GluArgs &A, int64_t t, int64_t row, float g, float u) {
  if (t >= A.T) return 0;
  float slope;
  const float a = activation(A.act, g, A.dh, slope);
  if (!A.dh) {
    if (row < A.rows) store1(A.h, A.dtype, t * A.rows + row, a * u);
    return 0;
  }
  const int64_t chunks = row_chunks(A.rows);
  if (row >= chunks * 64) return 0;
  float v[2] = {0.0f, 0.0f};
  if (row < A.rows) {
    const float d = load1(A.dh, A.dtype, t * A.rows + row);
    v[0] = d * (u * slope);
    v[1] = d * a;
  }
  const int in = static_cast<int>(row & 63);
  float *to = static_cast<float *>(A.G.g) + ((row >> 6) * A.G.ntile + (t >> 4)) * 1024 + (in >> 5) * 512 +
              ((in & 7) >> 2) * 256 + (((in & 31) >> 3) * 16 + (t & 15)) * 4 + (in & 3);
#pragma unroll
  for (int m = 0; m < 2; ++m) to[m * chunks * A.G.ntile * 1024] = v[m];
  return max_bits(max_bits(0, v[0]), v[1]);
}

// Eight rows of one token from row on (row a multiple of eight).
__device__ __forceinline__ uint32_t put8(const GluArgs &A, int64_t t, int64_t row, const float (&g)[8],
                                         const float (&u)[8]) {
  const int64_t chunks = row_chunks(A.rows), at = t * A.rows + row;
  const bool whole = row + 8 <= A.rows;
  float a[8], slope[8], d[8];
  if (A.dh) {
    if (row >= chunks * 64) return 0;
    if (whole) {
      load8u(A.dh, A.dtype, at, d);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) d[k] = row + k < A.rows ? load1(A.dh, A.dtype, at + k) : 0.0f;
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) a[k] = activation(A.act, g[k], A.dh, slope[k]);
  if (!A.dh) {
#pragma unroll
    for (int k = 0; k < 8; ++k) a[k] *= u[k];
    if (whole) {
      store8u(A.h, A.dtype, at, a);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (row + k < A.rows) store1(A.h, A.dtype, at + k, a[k]);
    }
    return 0;
  }
  uint32_t most = 0;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    float v[8];  // rows past the last: zeros, whatever was summed there
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[k] = row + k < A.rows ? (m ? d[k] * a[k] : d[k] * (u[k] * slope[k])) : 0.0f;
      most = max_bits(most, v[k]);
    }
    put_grads(A.G, m * chunks, t, row, v);
  }
  return most;
}

// The largest magnitude of each of a workgroup's N tokens, collected in LDS, into A.G.most (maxima, in any order alike).
template <int N> __device__ __forceinline__ void put_most(const GluArgs &A, int64_t t0, const uint32_t *s_most) {
  __syncthreads();
  const int64_t t = t0 + threadIdx.x;
  if (A.dh && threadIdx.x < N && t < A.T && s_most[threadIdx.x]) atomicMax(A.G.most + t, s_most[threadIdx.x]);
}

// ---------------------------------------------------------------------------
// Few tokens: the waves split K (split_blocks), a row tile of both weights each, so
// that many small loads are on their way at once.  Bound by latency: 5,632 x 2,048
// (IQ2_XS), one token, 8.7 us for 6.7 MB of payload, of which about 3 are the launch
// and the codebook's way to LDS; waves wait 0.44 of the time.
// ---------------------------------------------------------------------------
template <int F, int P, int C>
__global__ void __launch_bounds__(512) glu_split_kernel(GluArgs A) {
  constexpr int kTab = Geo<F>::N, kRed = 8 * 2 * 64;
  __shared__ uint4 s_mem[kTab > kRed ? kTab : kRed];
  __shared__ uint32_t s_most[16 * C];
  load_table<F>(s_mem, A.tab);
  if (threadIdx.x < 16 * C) s_most[threadIdx.x] = 0;
  const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  const Split S = split_of(A.nb);
  const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * S.rw + S.rg) * 16;
  const int64_t tt0 = static_cast<int64_t>(blockIdx.y) * C;
  const int64_t rowbytes = A.nb * Geo<F>::BYTES, stride = A.X.ntile * P * 4096;
  const int64_t at = min(row0 + n, A.rows - 1) * rowbytes;
  const _Float16 *x0[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int64_t t = min((tt0 + c) * 16 + n, A.T - 1);
    x0[c] = A.X.x16 + (t >> 4) * P * 4096 + (q * 16 + (t & 15)) * 8;
  }
  f32x4 acc[1][2][C] = {};
  __syncthreads();
  split_blocks<F, P, C, 1, 2>(
      A.nb, S, s_mem, [&](int m, int) { return A.packed[m] + at; },
      [&](int64_t b, Operand<P, C> &x) __attribute__((always_inline)) {
        const _Float16 *xp[C];
#pragma unroll
        for (int c = 0; c < C; ++c) xp[c] = x0[c] + b * stride;
        load_operand<P, C>(x, xp);
      },
      acc);
  f32x4 *red = reinterpret_cast<f32x4 *>(s_mem);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    __syncthreads();  // what the memory held before is read
#pragma unroll
    for (int m = 0; m < 2; ++m) red[((S.rg * S.kw + S.kg) * 2 + m) * 64 + lane] = acc[0][m][c];
    __syncthreads();
    for (int i = threadIdx.x; i < S.rw * 64; i += blockDim.x) {
      const int rg = i >> 6, l = i & 63;
      f32x4 s[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const f32x4 *p = red + (rg * S.kw * 2 + m) * 64 + l;
        s[m] = p[0];
        for (int k = 1; k < S.kw; ++k) s[m] += p[k * 128];
      }
      const int64_t row = (static_cast<int64_t>(blockIdx.x) * S.rw + rg) * 16 + (l & 15);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t t = (tt0 + c) * 16 + (l >> 4) * 4 + k;
        if (t >= A.T) continue;
        const int e = A.X.ex[t];
        const uint32_t most = put1(A, t, row, ldexpf(s[0][k], e), ldexpf(s[1][k], e));
        if (most) atomicMax(s_most + c * 16 + (l >> 4) * 4 + k, most);
      }
    }
  }
  put_most<16 * C>(A, tt0 * 16, s_most);
}

// load_words loads at least so many times.
constexpr int kWordLoads = 2;

// ---------------------------------------------------------------------------
// A batch of tokens: a wave has one row tile of one weight, RT row tiles of both are
// a workgroup, and all its C token tiles meet a weight in the registers of the wave
// that decoded it.  The tokens of half a block lie in LDS for all waves, the next
// half's on their way.  d scales a block's sums.  Bound by the decode's issue and the
// waits around it (0.54 of the time): 17,408 x 5,120 (IQ1_M), 48 tokens, 43 us, 0.40
// PFLOP/s; in workgroups of four row tiles 59 at 64 tokens where six take 50, see
// batch_cost.
// ---------------------------------------------------------------------------
template <int F, int P, int C, int RT>
__global__ void __launch_bounds__(128 * RT, RT < 4 ? 2 : RT / 2) glu_batch_kernel(GluArgs A) {
  constexpr int NW = 2 * RT, NP = C * P * 4, NPW = (NP + NW - 1) / NW;  // pieces of 1 KiB of half a block's tokens
  constexpr int kX = 2 * NP * 64, kRed = NW * C * 64;
  __shared__ uint4 s_tab[Geo<F>::N];
  __shared__ u32x4 s_x[kX > kRed ? kX : kRed];  // [half % 2][tile][part][step][lane]
  static_assert(16 * C <= 64 * NW, "a thread a token");
  const uint32_t x_at = IQ_LDS_ADDRESS(s_x);
  load_table<F>(s_tab, A.tab);
  const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), m = wave & 1, rt = wave >> 1;
  const int64_t rblk = static_cast<int64_t>(blockIdx.x) * (16 * RT), tt0 = static_cast<int64_t>(blockIdx.y) * C;
  const uint8_t *rp = A.packed[m] + min(rblk + rt * 16 + n, A.rows - 1) * A.nb * Geo<F>::BYTES;
  const char *xbase = reinterpret_cast<const char *>(A.X.x16) + tt0 * P * 8192;
  const int64_t xblock = A.X.ntile * P * 8192;
  uint32_t xoff[NPW];
#pragma unroll
  for (int i = 0; i < NPW; ++i) {
    const int p = i * NW + wave, most = static_cast<int>(min(A.X.ntile - tt0, static_cast<int64_t>(C))) - 1;
    xoff[i] = static_cast<uint32_t>((min(p / (P * 4), most) * P + p / 4 % P) * 8192 + p % 4 * 1024 + lane * 16);
  }
  const auto fetch = [&](int64_t b, int half) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NPW; ++i)
      if (NP % NW == 0 || i * NW + wave < NP)
        load_to_lds(xbase + b * xblock + half * 4096, xoff[i], x_at + (half * NP + i * NW + wave) * 1024);
  };
  f32x4 acc[C], part[C];
#pragma unroll
  for (int c = 0; c < C; ++c) acc[c] = part[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  Words words = load_words<F>(rp, q);
  fetch(0, 0);
  wait_loads<0>();
  __syncthreads();
  for (int64_t b = 0; b < A.nb; ++b) {
    const Raw raw = unpack<F>(words, q);
    half8v w[2];
    w[0] = group_half8<F>(raw, 0, s_tab);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (half == 0)
        fetch(b, 1);
      else if (b + 1 < A.nb)
        fetch(b + 1, 0);
      // after the tokens, which are waited for first: the payload comes from further away
      if (half == 0) words = load_words<F>(rp + min(b + 1, A.nb - 1) * Geo<F>::BYTES, q);
      __builtin_amdgcn_sched_barrier(0);  // the loads above go out before the work below
      const u32x4 *xs = s_x + half * NP * 64 + lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int g = half * 4 + i;
        half8v x[C][P];
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int p = 0; p < P; ++p) x[c][p] = __builtin_bit_cast(half8v, xs[((c * P + p) * 4 + i) * 64]);
        if (g < 7) w[(g + 1) & 1] = group_half8<F>(raw, g + 1, s_tab);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int p = 0; p < P; ++p)
            part[c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[c][p], w[g & 1], part[c], 0, 0, 0);
      }
      if (half == 1) {
        const float d = block_scale<F>(raw);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          scale_add(acc[c], part[c], d);
          part[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
      }
      if (half == 0)
        wait_loads<kWordLoads>();
      else
        wait_loads<0>();
      __syncthreads();  // the next half is there, this one free
    }
  }
  // both sums of an output in one lane: tile [row tile][weight][token tile], lane l's row l % 16, tokens 4 (l / 16) + k
  const float *all = reinterpret_cast<const float *>(s_x);
#pragma unroll
  for (int c = 0; c < C; ++c) s_x[((rt * 2 + m) * C + c) * 64 + lane] = __builtin_bit_cast(u32x4, acc[c]);
  uint32_t *s_most = reinterpret_cast<uint32_t *>(s_tab);  // the codebook has done its work
  if (threadIdx.x < 16 * C) s_most[threadIdx.x] = 0;
  __syncthreads();
#pragma unroll 1
  for (int i = threadIdx.x; i < 32 * RT * C; i += 64 * NW) {
    const int o = i % (2 * RT), tok = i / (2 * RT) & 15, c = i / (32 * RT);  // eight rows, token, token tile
    const int64_t t = (tt0 + c) * 16 + tok, row = rblk + o * 8;
    if (t >= A.T || row >= (A.dh ? row_chunks(A.rows) * 64 : A.rows)) continue;
    const int e = A.X.ex[t];
    const float *at = all + (((o >> 1) * 2 * C + c) * 64 + (tok >> 2) * 16 + (o & 1) * 8) * 4 + (tok & 3);
    float g[8], u[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      g[k] = ldexpf(at[k * 4], e);
      u[k] = ldexpf(at[C * 256 + k * 4], e);
    }
    const uint32_t most = put8(A, t, row, g, u);
    if (most) atomicMax(s_most + c * 16 + tok, most);
  }
  put_most<16 * C>(A, tt0 * 16, s_most);
}

// weights_half8 begun: the fields of group i, which is the same in all lanes but not known to the compiler, and its
// codebook entry, which comes from LDS some time later.
struct Entry {
  uint4 e;
  GroupFields g;
  uint32_t keep;
};
template <int F> __device__ __forceinline__ Entry lookup(const Raw &r, int i, const uint4 *tab, uint32_t keep) {
  Raw s = r;  // the words that hold it, where group_fields looks for those of groups 0 .. 3
  if (i & 4) {
    s.a[0] = F == IQ2_XXS || F == IQ2_XS ? r.a[2] : r.a[1];
    s.a[1] = r.a[3];
    if (F == IQ2_S) s.a[2] = r.a[3];
    if (F == IQ1_S || F == IQ1_M) s.a[2] = r.a[2] >> 16;
  }
  const int lo = i & 3;
  if (F == IQ2_XS) {
    s.a[0] = (lo & 2 ? s.a[1] : s.a[0]) >> (16 * (lo & 1));
    s.s = r.s >> (4 * (i >> 1));
  } else {
    s.a[0] >>= 8 * lo;
    if (F == IQ2_XXS) s.a[1] = ((s.a[1] >> (7 * lo)) & 127u) | (s.a[1] & 0xf0000000u);
    if (F == IQ2_S) {
      s.a[2] >>= 8 * lo;
      s.s = ((r.s >> (2 * i)) & 3u) | ((r.s >> (4 * (i >> 1))) & 0xffff0000u);
    }
    if (F == IQ1_S) s.a[2] = ((s.a[2] >> (3 * lo)) & 7u) | (s.a[2] & 0xf000u);
    if (F == IQ1_M) {
      s.a[2] >>= 4 * lo;
      s.s = r.s >> (3 * (i >> 1));
    }
  }
  Entry t;
  t.g = group_fields<F>(s, 0);
  t.e = tab[t.g.k];
  t.keep = keep;
  return t;
}

// ---------------------------------------------------------------------------
// Many tokens: a workgroup's weights are decoded once and reach its waves through
// LDS.  WT token groups of C tiles by WR row groups of R row tiles, half of them of
// the gate and half of the up projection, so that a wave's registers end up with
// both sums of an output.  Weights are the A operand here: a lane has four
// consecutive rows of one token.
//
// A stage is a step of 32 columns.  While the matrix cores work on stage s, the wave
// decodes its R / WT row tiles of stage s + 2 between their instructions and the
// tokens of stage s + 3 are on their way to LDS; its operands are read a group of W
// row tiles ahead, the first of a stage before the barrier that opens it (its buffers
// were full a barrier earlier), so that no wave waits for LDS at a barrier.
//
// 17,408 x 5,120 (IQ1_S), 4,096 tokens: 1,382 us, 1.06 PFLOP/s, where a library's large
// product of fp16 reaches 1.20.  Matrix cores are busy 0.43 of the time, LDS 0.33, and
// the decode issues 297,000 vector instructions a SIMD (0.37); waves wait 0.28.  With
// the decode and the operands' reads in the stage that needs them a call took 1,648 us
// instead of 1,433.  Backward (IQ1_M) 1,630 to 1,710: it writes both gradients in fp32, 560 MB where h is 140.
//
// Sums are kept in units of the block's d, as in iq_linear's prompts (P == 1, bf16
// calls); for f32 tokens a block has sums of its own, which are scaled and added (kept
// in one sum, 5,120 columns came to 1e-6 of h in the norm, near twice 32-bit
// arithmetic's).
// ---------------------------------------------------------------------------
template <int F, int P, int WT, int WR, int C, int R>
__global__ void __launch_bounds__(64 * WT * WR, WT * WR / 4) glu_tile_kernel(GluArgs A) {
  constexpr int NW = WT * WR, DR = R / WT, TA = WT * C, TB = WR * R;
  constexpr int W = R < 4 ? R : 4, NG = R / W;               // groups of row tiles whose operands are read together
  constexpr int NP = TA * P, NPW = (NP + NW - 1) / NW;       // pieces of 1 KiB of a stage's tokens, a wave's share
  static_assert(R % WT == 0 && R % 2 == 0 && R % W == 0, "whole row tiles to decode, as many of either weight");
  static_assert(NP % NW == 0 || NP < NW, "waves wait for the same number of loads, or have none");
  __shared__ uint4 s_tab[Geo<F>::N];
  __shared__ u32x4 s_a[4][NP * 64];  // tokens [stage % 4][tile][part][lane]
  __shared__ u32x4 s_b[3][TB * 64];  // weights [stage % 3][tile][lane]
  __shared__ f32x4 s_ratio[2][TB * 4], s_unit[TB * 4];
  static_assert(16 * TA <= 64 * NW, "a thread a token");
  const uint32_t x_at = IQ_LDS_ADDRESS(s_a);
  load_table<F>(s_tab, A.tab);
  const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wt = wave / WR, wr = wave % WR;
  const int64_t rblk = static_cast<int64_t>(blockIdx.x) * (TB / 2) * 16;  // first row of the workgroup
  const int64_t tt0 = static_cast<int64_t>(blockIdx.y) * TA, rowbytes = A.nb * Geo<F>::BYTES;
  const int stages = static_cast<int>(A.nb) * 8;
  // Tile i of the workgroup: row group i / R, within it R / 2 tiles of the gate, then of the up projection.
  const auto tile_row = [&](int i) { return rblk + ((i / R) * (R / 2) + i % R % (R / 2)) * 16; };
  const uint8_t *rp[DR];
#pragma unroll
  for (int i = 0; i < DR; ++i) {
    const int ti = wave * DR + i;
    rp[i] = A.packed[ti % R / (R / 2)] + min(tile_row(ti) + n, A.rows - 1) * rowbytes;
  }
  const char *xbase = reinterpret_cast<const char *>(A.X.x16) + tt0 * P * 8192;
  const int64_t xblock = A.X.ntile * P * 8192;  // bytes of a block of columns
  uint32_t xoff[NPW];
#pragma unroll
  for (int i = 0; i < NPW; ++i) {
    const int p = i * NW + wave, most = static_cast<int>(min(A.X.ntile - tt0, static_cast<int64_t>(TA))) - 1;
    xoff[i] = static_cast<uint32_t>((min(p / P, most) * P + p % P) * 8192 + lane * 16);
  }
  // Stages in turn, each call the next (past the last some bytes that are not read).
  const char *xnext = xbase;
  int fetched = 0;
  const auto fetch = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NPW; ++i)
      if (NP % NW == 0 || i * NW + wave < NP)
        load_to_lds(xnext, xoff[i], x_at + ((fetched & 3) * NP + i * NW + wave) * 1024);
    ++fetched;
    xnext += 1024;
    if ((fetched & 7) == 0) xnext += fetched < stages ? xblock - 8192 : -8192;
  };
  Words words[DR];
  Raw raw[DR];
  float unit[DR];
  uint32_t keep[DR];
  const auto load_block = [&](int64_t b) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < DR; ++i) words[i] = load_words<F>(rp[i] + min(b, A.nb - 1) * Geo<F>::BYTES, q);
  };
  // The block whose words are there becomes the one to decode; its d against the one before.  (Past the last block
  // the last comes again, which changes nothing that is read.)
  const auto open_block = [&](int par) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < DR; ++i) {
      raw[i] = unpack<F>(words[i], q);
      const float d = block_scale<F>(raw[i]);
      keep[i] = d != 0.0f ? ~0u : 0u;
      const float ratio = P == 2 ? d : keep[i] ? unit[i] / d : 1.0f;
      unit[i] = P == 2 ? 1.0f : keep[i] ? d : unit[i];
      if (q == 0) reinterpret_cast<float *>(s_ratio[par])[(wave * DR + i) * 16 + n] = ratio;
    }
  };
  const auto put_weights = [&](const Entry &t, int i, int buf) __attribute__((always_inline)) {
    s_b[buf][(wave * DR + i) * 64 + lane] = __builtin_bit_cast(u32x4, weights_half8<F>(t.g, t.e, t.keep));
  };
  half8v x[2][C][P], w[2][W];
  const auto read_x = [&](int u, int s) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int p = 0; p < P; ++p) x[u][c][p] = __builtin_bit_cast(half8v, s_a[s & 3][((wt * C + c) * P + p) * 64 + lane]);
  };
  const auto read_w = [&](int u, int g, int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[u][i] = __builtin_bit_cast(half8v, s_b[buf][(wr * R + g * W + i) * 64 + lane]);
  };

  f32x4 acc[R][C], part[P == 2 ? R : 1][C];  // part: a block's sums
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < C; ++c) acc[r][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < DR; ++i) unit[i] = 0.0f;
  load_block(0);
  fetch();
  fetch();
  fetch();
  __syncthreads();  // the codebook
  open_block(0);
  load_block(1);
#pragma unroll
  for (int d = 0; d < 2; ++d)
#pragma unroll
    for (int i = 0; i < DR; ++i) put_weights(lookup<F>(raw[i], d, s_tab, keep[i]), i, d);
  Entry t[DR];  // begun: the row tiles of stage s + 2
#pragma unroll
  for (int i = 0; i < DR; ++i) t[i] = lookup<F>(raw[i], 2, s_tab, keep[i]);
  wait_loads<0>();
  __syncthreads();
  read_x(0, 0);
  read_w(0, 0, 0);
  // Of a SIMD's two waves the first goes first: while it works on its addresses the other has the matrix cores.
  if (wave < NW / 2) __builtin_amdgcn_s_setprio(1);
  int b0 = 0, b1 = 1, b2 = 2;  // buffers of the weights of stages s, s + 1, s + 2
  const auto stage = [&](auto parity, int s) __attribute__((always_inline)) {
    constexpr int U = decltype(parity)::value;
    const int d = s + 2;
    if ((s & 7) == 0) {
      const int par = (s >> 3) & 1;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const f32x4 f = s_ratio[par][(wr * R + r) * 4 + q];
#pragma unroll
        for (int c = 0; c < C; ++c) {
          if (P == 2)
            part[r % (P == 2 ? R : 1)][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
          else
            acc[r][c] *= f;
        }
      }
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      constexpr int first = U * NG;  // groups alternate between two sets of registers
      // Before the last group's products the next stage's first operands and entries are requested.
      if (g + 1 < NG) {
        read_w((first + g + 1) & 1, g + 1, b0);
      } else {
        read_x(U ^ 1, s + 1);
        read_w((first + g + 1) & 1, 0, b1);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < DR; ++i)
        if (i * NG / DR == g) put_weights(t[i], i, b2);
#pragma unroll
      for (int i = 0; i < W; ++i)
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int p = 0; p < P; ++p) {
            f32x4 &to = P == 2 ? part[(g * W + i) % (P == 2 ? R : 1)][c] : acc[g * W + i][c];
            to = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[(first + g) & 1][i], x[U][c][p], to, 0, 0, 0);
          }
      __builtin_amdgcn_sched_barrier(0);
      if (g == 0) {
        if ((d & 7) == 1 && s > 0) load_block((d >> 3) + 1);
        fetch();
      }
    }
    if (((d + 1) & 7) == 0) open_block(((d + 1) >> 3) & 1);
#pragma unroll
    for (int i = 0; i < DR; ++i) t[i] = lookup<F>(raw[i], (d + 1) & 7, s_tab, keep[i]);
    if (P == 2 && (s & 7) == 7) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const f32x4 f = s_ratio[(s >> 3) & 1][(wr * R + r) * 4 + q];
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[r][c][k] = fmaf(f[k], part[r % (P == 2 ? R : 1)][c][k], acc[r][c][k]);
      }
    }
    // The tokens of stage s + 2 have to be there; what was requested after them may be on its way: those of stage
    // s + 3, and in one stage of eight the next block's payload, which comes from further away.
    if (s > 0 && (d & 7) == 1)
      wait_loads<NPW + DR * kWordLoads>();
    else
      wait_loads<NPW>();
    __syncthreads();
    const int old = b0;
    b0 = b1;
    b1 = b2;
    b2 = old;
  };
  for (int s = 0; s < stages; s += 2) {
    stage(std::integral_constant<int, 0>{}, s);
    stage(std::integral_constant<int, 1>{}, s + 1);
  }
  wait_loads<0>();  // the memory is used again below
#pragma unroll
  for (int i = 0; i < DR; ++i)
    if (q == 0) reinterpret_cast<float *>(s_unit)[(wave * DR + i) * 16 + n] = unit[i];
  uint32_t *s_most = reinterpret_cast<uint32_t *>(s_tab);  // the codebook has done its work
  if (threadIdx.x < 16 * TA) s_most[threadIdx.x] = 0;
  __syncthreads();
  // A token tile's sums at a time through LDS, in which a lane finds eight rows of one token; one copy of the code
  // for all of them (16 in a row were 160 KB of instructions, and took as long as twelve stages).
  static_assert(4 * NP >= NW * R, "a wave's sums of a token tile fit");
  f32x4 *own = reinterpret_cast<f32x4 *>(s_a) + wave * R * 64;
#pragma unroll 1
  for (int c = 0; c < C; ++c) {
#pragma unroll
    for (int k = 0; k < C; ++k) {
      if (k != c) continue;
#pragma unroll
      for (int r = 0; r < R; ++r) own[r * 64 + lane] = acc[r][k] * s_unit[(wr * R + r) * 4 + q];
    }
#pragma unroll 1
    for (int i = lane; i < 16 * R; i += 64) {
      const int m = i & 15, o = i >> 4;  // token, and its eight rows
      const int64_t t = (tt0 + wt * C + c) * 16 + m, row = tile_row(wr * R) + o * 8;
      if (t >= A.T || row >= (A.dh ? row_chunks(A.rows) * 64 : A.rows)) continue;
      const int e = A.X.ex[t];
      float g[8], u[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // row tile o / 2, quarters 2 (o % 2) + h
        const f32x4 *at = own + (o >> 1) * 64 + ((o & 1) * 2 + h) * 16 + m;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          g[h * 4 + k] = ldexpf(at[0][k], e);
          u[h * 4 + k] = ldexpf(at[R / 2 * 64][k], e);
        }
      }
      const uint32_t most = put8(A, t, row, g, u);
      if (most) atomicMax(s_most + (wt * C + c) * 16 + m, most);
    }
  }
  put_most<16 * TA>(A, tt0 * 16, s_most);
}

template <int F, int P, int C> void launch_split(const GluArgs &A, hipStream_t stream) {
  const int64_t rw = split_rw(A.nb), rows = rw * 16, all = A.dh ? row_chunks(A.rows) * 64 : A.rows;
  hipLaunchKernelGGL((glu_split_kernel<F, P, C>),
                     dim3(static_cast<unsigned>((all + rows - 1) / rows),
                          static_cast<unsigned>((A.X.ntile + C - 1) / C)),
                     dim3(static_cast<unsigned>(64 * split_kw(A.nb) * rw)), 0, stream, A);
}

template <int F, int P, int WT, int WR, int C, int R>
void launch_tile(const GluArgs &A, hipStream_t stream) {
  constexpr int rows = WR * R / 2 * 16;
  const int64_t all = A.dh ? row_chunks(A.rows) * 64 : A.rows;
  hipLaunchKernelGGL((glu_tile_kernel<F, P, WT, WR, C, R>),
                     dim3(static_cast<unsigned>((all + rows - 1) / rows),
                          static_cast<unsigned>((A.X.ntile + WT * C - 1) / (WT * C))),
                     dim3(64 * WT * WR), 0, stream, A);
}

template <int F, int P, int C, int RT> void launch_batch(const GluArgs &A, hipStream_t stream) {
  const int64_t all = A.dh ? row_chunks(A.rows) * 64 : A.rows;
  hipLaunchKernelGGL((glu_batch_kernel<F, P, C, RT>),
                     dim3(static_cast<unsigned>((all + 16 * RT - 1) / (16 * RT)),
                          static_cast<unsigned>((A.X.ntile + C - 1) / C)),
                     dim3(128 * RT), 0, stream, A);
}

// What a batch costs with RT row tiles a workgroup: the rounds of its workgroups over 256 CUs times a workgroup's
// waves on a SIMD, in eighths.  Measured at 17,408 x 5,120 (IQ1_M) with RT = 2, 4, 6, us: 64 tokens 67, 59, 50 (3, 4 and
// 3 waves on the fullest CU's SIMDs); 128 tokens 97, 89, 91; 256 tokens 158, 138, 132; at 5,632 x 2,048 (IQ2_S): 64
// tokens 20, 23, 27; 128 tokens 25, 24, 27; 256 tokens 32, 35, 31.  So workgroups of two row tiles, which bring as many
// tokens to LDS as others, count a quarter more where several share a CU (with two token tiles they do not: 39, 47,
// 44 at 32 tokens), six a tenth.
inline int64_t batch_cost(const GluArgs &A, int C, int RT) {
  const int64_t rounds = ((A.rows + 16 * RT - 1) / (16 * RT) * ((A.X.ntile + C - 1) / C) + 255) / 256;
  return rounds * (RT == 2 ? (rounds > 1 && C > 2 ? 10 : 8) : RT == 4 ? 16 : 26);
}

template <int F, int P, int C> void launch_batches(const GluArgs &A, hipStream_t stream) {
  const int64_t two = batch_cost(A, C, 2), four = batch_cost(A, C, 4), six = batch_cost(A, C, 6);
  if (two < four && two <= six) return launch_batch<F, P, C, 2>(A, stream);
  if (four <= six) return launch_batch<F, P, C, 4>(A, stream);
  launch_batch<F, P, C, 6>(A, stream);
}

template <int F, int P> void launch_glu(const GluArgs &A, hipStream_t stream) {
  const int64_t ntile = A.X.ntile;
  if (ntile == 1) return launch_split<F, P, 1>(A, stream);
  if (ntile == 2) return launch_batches<F, P, 2>(A, stream);
  // Three token tiles a workgroup where they leave less of it empty than four, us with two, three and four: 17,408 x
  // 5,120 (IQ1_M), 48 tokens 57, 42, 46 (f32 91, 55, 65), 80 tokens 82, 73, 82 (122, 101, 139), 96 tokens 81, 72, 80 (119,
  // 101, 135); 5,632 x 2,048 (IQ2_S) 16, 14, 15, 20, 18, 20 and 20, 18, 21.
  if (ntile == 3 || ntile == 5 || ntile == 6) return launch_batches<F, P, 3>(A, stream);
  // Tiles, a workgroup a CU, take 16 us a round and 7.2 more for each block of columns; batches 0.08 and 0.09 (f32
  // 0.155) of their cost.  5,632 x 2,048 (IQ2_S), batches and tiles, us: 500 tokens 49 and 83, 2,048 tokens 150 and
  // 167, 4,096 tokens 286 and 244 (f32: 512 tokens 70 and 84, 2,048 tokens 228 and 236); 17,408 x 5,120 (IQ1_M): 512
  // tokens 255 and 335, 1,024 tokens 493 and 522.
  constexpr int C = P == 2 ? 2 : 4;
  // A checkpoint's tokens in an f32 call want a block's own sums as well.  Tiles of 128 of them took 67 and 410 us for 512
  // and 4,096 tokens of 5,632 x 2,048 (IQ2_S) where batches, which have them, take 48 and 328; 17,408 x 5,120 (IQ1_M),
  // 2,048 tokens 1,220 and 975.
  if (P == 1 && A.dtype == IQ_DTYPE_F32) return launch_batches<F, P, 4>(A, stream);
  int64_t batch = batch_cost(A, 4, 2);
  for (int RT = 4; RT <= 6; RT += 2) batch = min(batch, batch_cost(A, 4, RT));
  const int64_t rounds = ((A.rows + 127) / 128 * ((ntile + 4 * C - 1) / (4 * C)) + 255) / 256;
  if (batch * (16 + (P == 2 ? 31 : 18) * A.nb) <= rounds * (3200 + 1440 * A.nb)) return launch_batches<F, P, 4>(A, stream);
  launch_tile<F, P, 4, 2, C, 8>(A, stream);
}

struct GluPlan {
  TokensPlan x;
  RowsPlan rows;
  size_t xo, eo, bo, go, geo, po, bytes;
};
GluPlan plan_glu(int fmt, int64_t inter, int64_t hidden, int dtype, int64_t T, bool backward) {
  GluPlan p{};
  p.x = plan_tokens(T, hidden, dtype);  // a checkpoint of f32 tokens needs half of it
  p.xo = ws_up(static_cast<size_t>(kCodebook[fmt]) * 16);
  p.eo = p.xo + ws_up(p.x.xbytes);
  p.bo = p.eo + ws_up(p.x.ebytes);
  p.bytes = p.bo + kWsAlign;
  if (!backward) return p;
  const int64_t chunks = 2 * row_chunks(inter);
  p.rows = plan_rows(T, hidden / 256, chunks, dtype, true);
  p.go = p.bo + ws_up(kBoundBytes);
  p.geo = p.go + ws_up(grads_bytes(chunks, p.x.ntile, true));
  p.po = p.geo + ws_up(p.x.ebytes);
  p.bytes = p.po + ws_up(p.rows.bytes) + kWsAlign;
  return p;
}

int check_glu(int fmt, int64_t inter, int64_t hidden, int dtype, int64_t T) {
  if (run_bad_fmt(fmt)) return IQ_ERR_FMT;
  if (run_bad_dtype(dtype)) return IQ_ERR_DTYPE;
  if (inter < 0 || T < 0 || hidden <= 0 || hidden % 256 != 0) return IQ_ERR_SHAPE;
  if (inter > (int64_t(1) << 24) || hidden > (int64_t(1) << 24) || T > (int64_t(1) << 24)) return IQ_ERR_SHAPE;
  const int64_t ntile = (T + 15) / 16;
  if (ntile > 4 * 65535) return IQ_ERR_SHAPE;  // token tiles of the products
  if (T * (hidden / 256) >= (int64_t(1) << 26)) return IQ_ERR_SHAPE;  // the tiles of dx
  return IQ_OK;
}

int run_glu(int fmt, const uint8_t *gate, const uint8_t *up, int64_t inter, int64_t hidden, const float *grid,
            const void *x, const uint8_t *exponents, const void *dh, int dtype, int64_t T, int act, void *out,
            bool backward, void *workspace, size_t workspace_bytes, int32_t *status, hipStream_t stream) {
  int rc = check_glu(fmt, inter, hidden, dtype, T);
  if (rc != IQ_OK) return rc;
  if (act < IQ_ACT_SILU || act > IQ_ACT_GELU_TANH) return IQ_ERR_ARG;
  const bool nothing = T == 0 || (inter == 0 && !backward), zeros = !nothing && inter == 0;
  if (!grid || (!nothing && !zeros && (!gate || !up || !x || (backward && !dh))) || (!nothing && !out))
    return IQ_ERR_NULL;
  if (nothing) return IQ_OK;
  if (zeros) return launch_zero(out, static_cast<size_t>(T) * hidden * (dtype == IQ_DTYPE_F32 ? 4 : 2), stream);
  if ((reinterpret_cast<uintptr_t>(gate) | reinterpret_cast<uintptr_t>(up)) & 1) return IQ_ERR_ARG;
  const GluPlan P = plan_glu(fmt, inter, hidden, dtype, T, backward);
  if ((rc = run_check_ws(P.bytes, workspace, workspace_bytes)) != IQ_OK) return rc;
  char *base = ws_base(workspace);
  _Float16 *tab = reinterpret_cast<_Float16 *>(base);
  const Tokens X{reinterpret_cast<_Float16 *>(base + P.xo), reinterpret_cast<int32_t *>(base + P.eo), P.x.ntile};
  GluPrepArgs A{};
  A.S = Source{x, exponents, dtype};
  A.T = T;
  A.cols = hidden;
  A.nconv = (T + 7) / 8;
  A.X = X;
  A.books = one_codebook(fmt, grid, tab, status);
  A.fmt = fmt;
  A.bytes = block_bytes(fmt);
  A.backward = backward;
  A.packed[0] = gate;
  A.packed[1] = up;
  A.rows = inter;
  GluArgs M{};
  M.packed[0] = gate;
  M.packed[1] = up;
  M.rows = inter;
  M.nb = hidden / 256;
  M.T = T;
  M.tab = tab;
  M.X = X;
  M.act = act;
  M.dtype = dtype;
  M.h = out;
  if (backward) {
    A.B = Bound{reinterpret_cast<uint32_t *>(base + P.bo), reinterpret_cast<uint32_t *>(base + P.bo) + kScaleSlots,
                A.books.wg[0], fmt >= IQ1_S};
    A.most = reinterpret_cast<uint32_t *>(base + P.geo);
    M.dh = dh;
    M.G = Grads{base + P.go, A.most, P.x.ntile};
  }
  const int64_t wgs = A.nconv + A.books.wg[0] + (backward ? kScaleSlots : 0);
  hipLaunchKernelGGL(glu_prep_kernel, dim3(static_cast<unsigned>(wgs)), dim3(512), 0, stream, A);
  if (!run_launched()) return IQ_ERR_HIP;
#define CALL(F) source_parts(A.S) == 2 ? launch_glu<F, 2>(M, stream) : launch_glu<F, 1>(M, stream)
  IQ_BY_FMT(fmt, CALL)
#undef CALL
  if (!run_launched()) return IQ_ERR_HIP;
  if (!backward) return IQ_OK;
  RowsArgs D{};
  D.packed[0] = gate;
  D.packed[1] = up;
  D.nmat = 2;
  D.rows = inter;
  D.nb = hidden / 256;
  D.T = T;
  D.tab = tab;
  D.G = M.G;
  D.B = A.B;
  D.out = out;
  D.partial = reinterpret_cast<float *>(base + P.po);
  D.plan = P.rows;
  return launch_rows(fmt, dtype, D, stream);
}

int glu_size(int fmt, int64_t inter, int64_t hidden, int dtype, int64_t T, bool backward, size_t *bytes) {
  const int rc = check_glu(fmt, inter, hidden, dtype, T);
  if (rc != IQ_OK) return rc;
  if (!bytes) return IQ_ERR_NULL;
  *bytes = inter && T ? plan_glu(fmt, inter, hidden, dtype, T, backward).bytes : 0;
  return IQ_OK;
}

}  // namespace
}  // namespace iq

extern "C" {

int iq_glu_workspace_size(int fmt, int64_t inter, int64_t hidden, int dtype, int64_t T, size_t *bytes) {
  return iq::glu_size(fmt, inter, hidden, dtype, T, false, bytes);
}

int iq_glu(int fmt, const uint8_t *gate, const uint8_t *up, int64_t inter, int64_t hidden, const float *grid,
           const void *x, int dtype, int64_t T, int act, void *h, void *workspace, size_t workspace_bytes,
           int32_t *status, hipStream_t stream) {
  return iq::run_glu(fmt, gate, up, inter, hidden, grid, x, nullptr, nullptr, dtype, T, act, h, false, workspace,
                     workspace_bytes, status, stream);
}

int iq_glu_backward_workspace_size(int fmt, int64_t inter, int64_t hidden, int dtype, int64_t T, size_t *bytes) {
  return iq::glu_size(fmt, inter, hidden, dtype, T, true, bytes);
}

int iq_glu_backward(int fmt, const uint8_t *gate, const uint8_t *up, int64_t inter, int64_t hidden,
                    const float *grid, const void *x, const uint8_t *exponents, const void *dh, int dtype,
                    int64_t T, int act, void *dx, void *workspace, size_t workspace_bytes, int32_t *status,
                    hipStream_t stream) {
  return iq::run_glu(fmt, gate, up, inter, hidden, grid, x, exponents, dh, dtype, T, act, dx, true, workspace,
                     workspace_bytes, status, stream);
}

}  // extern "C"
