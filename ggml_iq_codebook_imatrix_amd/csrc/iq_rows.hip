// iq_rows.hip -- dx = G W: gradients by encoded weights, summed over the weights'
// rows (iq_linear_backward, and iq_glu_backward for two weights one after the
// other).
//
// A weight is d m v, d its block's scale.  m v is exact in fp16.  d differs from row to
// row, so it cannot scale a sum; but a workgroup's columns are one block of each row,
// so that d belongs to a row there, as the gradients do: G d is formed in fp32 for the
// workgroup and enters as the sum of two fp16 values (2^-23 of the value), under
// one power of two per token, of its largest gradient, and one for the payload's scales.  The weight as an fp16
// operand in the place of m v would have been rounded twice; two values of it, beside
// gradients of two values, take three products and twice the LDS.
//
// The matrix instruction wants eight consecutive rows of one column from a lane; a
// payload gives eight consecutive columns of one row.  A thread therefore decodes
// the same group of four consecutive rows, which makes two pairs of rows of each of
// its eight columns by byte permutations, and eight such columns are the eight
// operands that a group's lane has in eight instructions: operand j of half h holds
// columns 128 h + 8 n + j of a block, n the lane's place, so that its results are
// eight consecutive columns of dx.  Decoded once for all tokens of a workgroup, the
// weights reach the waves through LDS; a wave's gradients are its own tokens', and
// come from memory to its registers.  For f32 the sums of four chunks are added to the
// whole ones, so that fewer additions round at a whole sum's size.

#include <algorithm>
#include <type_traits>

#include "iq_train.hpp"

namespace iq {
namespace {

// acc[j][c] += p A of the adapters that the wave's tokens (tiles tt .. tt + C - 1) name, columns col + j of the lane's
// eight.  32 ranks at a time: a lane has eight ranks of its eight columns, which byte permutations make operands of
// (bf16; p is the sum of three bf16 values, without a rounding), or four ranks at a time on the fp32 cores.  Rows of
// tokens with other adapters are zeros; where A is not finite (wild), 0 * A would reach them, and what they give is dropped.
template <bool F32, int C>
__device__ __forceinline__ void add_adapters(const RowsArgs &A, int64_t tt, int64_t col, f32x4 (&acc)[8][C]) {
  const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  const int64_t cols = A.nb * 256, mytok = tt * 16 + lane, cb = col >> 8;
  const int mine = lane < 16 * C && mytok < A.T ? A.ids[mytok] : -1;
  const int tiles = (A.rank + 15) >> 4;
  uint64_t todo = __ballot(mine >= 0);
  while (todo) {
    const int a = __builtin_amdgcn_readlane(mine, __builtin_ctzll(todo));
    const uint64_t group = __ballot(mine == a);
    todo &= ~group;
    for (int r0 = 0; r0 < A.rank; r0 += F32 ? 4 : 32) {
      const uint32_t *wild = A.wild + (static_cast<int64_t>(a) * tiles + (r0 >> 4)) * A.nb + cb;
      const bool drop = wild[0] | wild[!F32 && r0 + 16 < A.rank ? A.nb : 0];
      if constexpr (!F32) {
        const uint16_t *from = static_cast<const uint16_t *>(A.a) + static_cast<int64_t>(a) * A.rank * cols + col;
        u32x4 w[8];  // ranks r0 + 8 q + i; zeros past the last, as p is there
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = ldu<u32x4>(from + min(r0 + 8 * q + i, A.rank - 1) * cols);
        if (r0 + 32 > A.rank) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (r0 + 8 * q + i >= A.rank) w[i] = u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const uint32_t tokens = static_cast<uint32_t>(group >> (16 * c)) & 0xffffu;
          if (!tokens) continue;
          const uint16_t *p = A.parts + ((tt + c) * ((A.rank + 31) >> 5) + (r0 >> 5)) * 1536 + lane * 8;
          const uint32_t keep = (tokens >> n) & 1u ? ~0u : 0u;
          bf16x8 v[3];
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            u32x4 t = ldu<u32x4>(p + k * 512);
#pragma unroll
            for (int i = 0; i < 4; ++i) t[i] &= keep;
            v[k] = __builtin_bit_cast(bf16x8, t);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t sel = j & 1 ? 0x07060302u : 0x05040100u;
            u32x4 o;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = __builtin_amdgcn_perm(w[2 * i + 1][j >> 1], w[2 * i][j >> 1], sel);
            f32x4 d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[0], __builtin_bit_cast(bf16x8, o), acc[j][c], 0, 0, 0);
            if (drop) {  // the first part of p has met what is not finite; the others may be zeros
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if ((o[i] & 0x7f80u) == 0x7f80u) o[i] &= 0xffff0000u;
                if ((o[i] & 0x7f800000u) == 0x7f800000u) o[i] &= 0xffffu;
              }
            }
#pragma unroll
            for (int k = 1; k < 3; ++k)
              d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[k], __builtin_bit_cast(bf16x8, o), d, 0, 0, 0);
            if (drop) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (!((tokens >> (4 * q + k)) & 1u)) d[k] = acc[j][c][k];
            }
            acc[j][c] = d;
          }
        }
      } else {
        float w[8];
        load8u(A.a, 0, (static_cast<int64_t>(a) * A.rank + min(r0 + q, A.rank - 1)) * cols + col, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = r0 + q < A.rank ? w[j] : 0.0f;  // as v is there
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const uint32_t tokens = static_cast<uint32_t>(group >> (16 * c)) & 0xffffu;
          if (!tokens) continue;
          const float v = r0 + q < A.rank && ((tokens >> n) & 1u) ? A.p[(r0 + q) * A.tpad + (tt + c) * 16 + n] : 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            f32x4 d = __builtin_amdgcn_mfma_f32_16x16x4f32(v, w[j], acc[j][c], 0, 0, 0);
            if (drop) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (!((tokens >> (4 * q + k)) & 1u)) d[k] = acc[j][c][k];
            }
            acc[j][c] = d;
          }
        }
      }
    }
  }
}

// Two gradients times their rows' scales, as the sums of two fp16 values each, to 2^-23 of the product; where it is
// infinite the second value, inf - inf, becomes a number, which leaves the infinity.
template <class V>
__device__ __forceinline__ void scaled_parts(V g0, V g1, float d0, float d1, uint32_t &hi, uint32_t &lo) {
  // written as fma, a product and its rounding are one instruction for each half of a register
  const half2v h = {static_cast<_Float16>(__builtin_fmaf(static_cast<float>(g0), d0, 0.0f)),
                    static_cast<_Float16>(__builtin_fmaf(static_cast<float>(g1), d1, 0.0f))};
  hi = __builtin_bit_cast(uint32_t, h);
  asm("" : "+v"(hi));  // both halves are taken from here
  const half2v k = __builtin_bit_cast(half2v, hi);
  const half2v l = {static_cast<_Float16>(__builtin_fmaf(static_cast<float>(g0), d0, -static_cast<float>(k[0]))),
                    static_cast<_Float16>(__builtin_fmaf(static_cast<float>(g1), d1, -static_cast<float>(k[1])))};
  const half2v most = {static_cast<_Float16>(65504.0f), static_cast<_Float16>(65504.0f)};
  lo = __builtin_bit_cast(uint32_t, __builtin_elementwise_min(l, most));
}

// Eight waves, each C tiles of 16 tokens and the block's 256 columns.  WIDE: the gradients are fp32, else fp16.  F32: dx
// is.  LORA: with adapters.
//
// A stage is a step of 32 rows, a chunk two.  Chunk c + 1 is decoded in the odd stage of chunk c - 1 (a thread's first
// two rows) and the even stage of chunk c (the others, and both pairs to LDS); the next stage's gradients meet their
// scales in each stage, and those of the stage after it are requested when that is done.  Payload is requested in the odd
// stage four chunks before its own.  The work stands between the matrix instructions, and weights are read a group of G
// columns ahead, a stage's first before the barrier that opens it.
//
// With 256 tokens bound by the matrix cores at the rate that a large product sustains here: 176 chunks by 256 tiles
// (IQ2_XS, fp16 gradients) 638 us, 1.18 PFLOP/s of its two products (a library's product of fp16: 1.20).  With 128 tokens
// the decode, which is the same for half the products, counts as much as they do: 455 us, 0.83.
template <int F, bool WIDE, int C, bool F32, bool LORA>
__global__ void __launch_bounds__(512, 2) rows_kernel(RowsArgs A) {
  constexpr int NT = 512, TA = 8 * C;
  constexpr int W = (Geo<F>::BYTES + 5) / 4, NR = (64 * W + NT - 1) / NT;  // words of a row's block, a thread's share
  constexpr int NB = 3;                                                    // chunks of payload in LDS
  constexpr int GL = WIDE ? 2 : 1;                                         // a lane's loads of a tile's step
  __shared__ uint4 s_tab[Geo<F>::N];
  __shared__ u32x4 s_b[2][2][16 * 64];     // m v [chunk % 2][step][column 8 half + j][lane]
  __shared__ uint32_t s_raw[NB][NR * NT];  // [chunk % NB][row][word]
  __shared__ f32x4 s_d[2][16];             // the rows' scales [chunk % 2][row / 4]
  const uint32_t raw_at = IQ_LDS_ADDRESS(s_raw);
  const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool whole = blockIdx.x < A.plan.full;
  const int64_t rest = blockIdx.x - A.plan.full, place = whole ? blockIdx.x : A.plan.full + rest / A.plan.splits;
  const int splits = whole ? 1 : A.plan.splits, split = whole ? 0 : static_cast<int>(rest % A.plan.splits);
  const int64_t cb = place % A.nb, tt0 = place / A.nb * TA;
  const int64_t cols = A.nb * 256, rowbytes = A.nb * Geo<F>::BYTES;
  const int64_t per = (A.rows + 63) / 64, chunks = per * A.nmat;
  const int64_t share = (chunks + splits - 1) / splits, ch0 = split * share;
  const int count = static_cast<int>(max(min(share, chunks - ch0), static_cast<int64_t>(0)));
  const bool more = count > NB;  // payload is requested in the loop as well
  // Waves past the last token decode, and multiply nothing (5,120 x 17,408, one token 49 us instead of 70, 64 tokens 57
  // instead of 69); in the tiles of many tokens the branch would cost registers that are not there.
  const bool active = C == 2 || tt0 + wave * C < A.G.ntile;
  const uint8_t *const p0 = A.packed[0] + cb * Geo<F>::BYTES, *const p1 = A.packed[A.nmat - 1] + cb * Geo<F>::BYTES;

  // The first row of chunk c of the workgroup's, and whether it is the second weight's; past the last chunk the last.
  const auto chunk_of = [&](int c, bool &second) __attribute__((always_inline)) {
    const int64_t ch = ch0 + min(c, count - 1);
    second = ch >= per;
    return (second ? ch - per : ch) * 64;
  };
  // Its blocks, whole aligned words (rows past the last read the last's) into buffer `buf`.  64 rows are a multiple of
  // four bytes, so a lane's offsets are the same for all whole chunks of a weight.
  uint32_t roff[NR];
  int rkey = -1;
  const auto fetch_raw = [&](int c, int buf) __attribute__((always_inline)) {
    bool second;
    const int64_t row0 = chunk_of(c, second);
    const uintptr_t base = reinterpret_cast<uintptr_t>(second ? p1 : p0);
    const int most = static_cast<int>(min(A.rows - 1 - row0, static_cast<int64_t>(63))), key = most * 2 + second;
    if (key != rkey) {
      rkey = key;
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const int u = i * NT + static_cast<int>(threadIdx.x), r = min(u / W, most), w = u % W;
        const uint32_t at = static_cast<uint32_t>(base & 2) + static_cast<uint32_t>(r) * static_cast<uint32_t>(rowbytes);
        roff[i] = (at & ~3u) + 4 * min(w, static_cast<int>(((at & 2) + Geo<F>::BYTES - 1) >> 2));
      }
    }
    const char *from = reinterpret_cast<const char *>(base & ~uintptr_t(3)) + row0 * rowbytes;
#pragma unroll
    for (int i = 0; i < NR; ++i) load_words_to_lds(from, roff[i], raw_at + ((buf * NR + i) * NT + wave * 64) * 4);
  };
  // The wave's gradients of a step of the chunk at `from`, and with their scales as operands.
  const int64_t gchunk = A.G.ntile * (GL * 2048);
  const char *gbase = reinterpret_cast<const char *>(A.G.g) + (ch0 * A.G.ntile + tt0) * (GL * 2048);
  uint32_t goff[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int most = static_cast<int>(min(A.G.ntile - tt0, static_cast<int64_t>(TA))) - 1;
    goff[c] = static_cast<uint32_t>(min(wave * C + c, most) * (GL * 2048) + lane * 16);
  }
  u32x4 grad[C][GL];
  const auto load_grads = [&](const char *from, int step) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < GL; ++i)
        grad[c][i] = ld_global<u32x4, 16>(reinterpret_cast<uintptr_t>(from) + (step * GL + i) * 1024 + goff[c]);
  };
  // of the lane's tokens, and of the payload
  float power[C];
#pragma unroll
  for (int c = 0; c < C; ++c)
    power[c] = ldexpf(1.0f, grad_power(A.G.most[min(tt0 + wave * C + c, A.G.ntile - 1) * 16 + n], true));
  half8v x[2][C][2];
  f32x4 scale[2];
  const auto read_scales = [&](int c, int step) __attribute__((always_inline)) {
    scale[0] = s_d[c & 1][step * 8 + q * 2];
    scale[1] = s_d[c & 1][step * 8 + q * 2 + 1];
  };
  const auto convert = [&](int u, int c) __attribute__((always_inline)) {
    u32x4 hi, lo;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float d0 = scale[i >> 1][2 * (i & 1)], d1 = scale[i >> 1][2 * (i & 1) + 1];
      uint32_t h, l;
      if constexpr (WIDE) {
        const u32x4 &g = grad[c][(i >> 1) % GL];
        scaled_parts(__uint_as_float(g[2 * (i & 1)]) * power[c], __uint_as_float(g[2 * (i & 1) + 1]) * power[c], d0, d1, h, l);
      } else {
        const half2v g = __builtin_bit_cast(half2v, static_cast<uint32_t>(grad[c][0][i]));
        scaled_parts(g[0], g[1], d0, d1, h, l);
      }
      hi[i] = h;
      lo[i] = l;
    }
    x[u][c][0] = __builtin_bit_cast(half8v, hi);
    x[u][c][1] = __builtin_bit_cast(half8v, lo);
  };
  // The thread's group and four rows of each chunk: fields and entries of two rows at a time, weights, and both pairs
  // of rows to operand [quad / 8][half][column], lane 16 ((quad % 8) / 2) + n, half quad % 2.
  const int group = (wave & 1) * 16 + n, quad = (wave >> 1) * 4 + q;
  Fields f[2];
  uint4 e[2];
  uint32_t wv[4][4];
  int last = 0;  // of the rows in `f`'s chunk
  const int odd0 = static_cast<int>(reinterpret_cast<uintptr_t>(p0)) & 2, odd1 = static_cast<int>(reinterpret_cast<uintptr_t>(p1)) & 2;
  const auto read_rows = [&](int c, int j0, int buf) __attribute__((always_inline)) {
    bool second;
    const int64_t row0 = chunk_of(c, second);
    last = static_cast<int>(min(A.rows - 1 - row0, static_cast<int64_t>(63)));
    const int step = static_cast<int>(rowbytes) & 2, odd = second ? odd1 : odd0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = quad * 4 + j0 + j, half = ((min(r, last) << 1) & step) ^ odd;  // the block's address modulo four
      f[j] = read_fields<F>(reinterpret_cast<const uint8_t *>(&s_raw[buf][r * W]) + half, group, half);
    }
  };
  const auto look_up = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 2; ++j) e[j] = s_tab[f[j].k];
  };
  const int ed = scale_exponent(A.B), shift = codebook_shift(A.B);
  const _Float16 shrink = static_cast<_Float16>(ldexpf(1.0f, -shift));
  const auto weigh = [&](int c, int j0) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 2; ++j) row_weights<F>(f[j], e[j], half2v{shrink, shrink}, wv[j0 + j]);
    if (group == 0) {  // zeros past the last row, whose scale need not be finite
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float d = f16_bits_to_f32(static_cast<uint16_t>(f[j].d16)) * (Geo<F>::IQ1 ? 1.0f : 0.125f);
        reinterpret_cast<float *>(s_d[c & 1])[quad * 4 + j0 + j] = quad * 4 + j0 + j <= last ? ldexpf(d, -ed) : 0.0f;
      }
    }
  };
  const auto put = [&](int c) __attribute__((always_inline)) {
    uint2 *to = reinterpret_cast<uint2 *>(s_b[c & 1][quad / 8]) + ((wave & 1) * 8 * 64 + (quad % 8) / 2 * 16 + n) * 2 + quad % 2;
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
      for (int k = 0; k < 2; ++k) {  // column p + 4 k
        const uint32_t sel = k ? 0x07060302u : 0x05040100u;
        to[(p + 4 * k) * 128] = make_uint2(__builtin_amdgcn_perm(wv[1][p], wv[0][p], sel),
                                           __builtin_amdgcn_perm(wv[3][p], wv[2][p], sel));
      }
  };
  constexpr int G = C == 1 && !F32 ? 4 : 2, NG = 16 / G;  // columns whose weights are read together
  half8v w[2][G];
  const auto read_w = [&](int u, int g, int c, int step) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < G; ++j) w[u][j] = __builtin_bit_cast(half8v, s_b[c & 1][step][(g * G + j) * 64 + lane]);
  };

  f32x4 acc[2][8][C], part[F32 ? 16 : 1][C];
#pragma unroll
  for (int j = 0; j < 16; ++j)
#pragma unroll
    for (int c = 0; c < C; ++c) acc[j >> 3][j & 7][c] = part[F32 ? j : 0][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  int r1 = 1, r2 = 2;  // the buffers of the payload of chunks c + 1 and c + 2
  const char *g1 = gbase + (count > 1 ? gchunk : 0);  // the gradients of chunk c + 1; past the last its
  const auto stage = [&](auto step, int c) __attribute__((always_inline)) {
    constexpr int U = decltype(step)::value;
    const int next = c + 1 + U;  // the chunk whose rows are decoded in this stage
    read_rows(next, U ? 0 : 2, U ? r2 : r1);
    if (U == 1 && more) fetch_raw(c + 4, r1);  // chunk c + 1's is decoded
    if (active) {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (g + 1 < NG)
          read_w((g + 1) & 1, g + 1, c, U);
        else  // the next stage's first
          read_w(0, 0, c + U, U ^ 1);
        __builtin_amdgcn_sched_barrier(0);
        if (g == NG / 4) weigh(next, U ? 0 : 2);
        if (g == NG / 2 - 1 && U == 0) put(next);
        if (g == NG - C - 1) read_scales(c + U, U ^ 1);
        if (g >= NG - C) convert(U ^ 1, g - (NG - C));
#pragma unroll
        for (int j = 0; j < G; ++j)
#pragma unroll
          for (int cc = 0; cc < C; ++cc) {
            const int col = g * G + j;
            f32x4 &to = F32 ? part[F32 ? col : 0][cc] : acc[col >> 3][col & 7][cc];
#pragma unroll
            for (int p = 0; p < 2; ++p) to = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[U][cc][p], w[g & 1][j], to, 0, 0, 0);
          }
        __builtin_amdgcn_sched_barrier(0);
        if (g == 0) {
          look_up();
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    } else {
      look_up();
      weigh(next, U ? 0 : 2);
      if (U == 0) put(next);
    }
    load_grads(g1, U);
    if (F32 && U == 1 && ((c & 3) == 3 || c + 1 == count)) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
#pragma unroll
        for (int cc = 0; cc < C; ++cc) {
          f32x4 &p = part[F32 ? j : 0][cc];
          acc[j >> 3][j & 7][cc] += p;
          p = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
    }
    // The payload of chunk c + 2, which the next stage reads, has to be there; of what was requested after it the newest
    // may be on its way: chunk c + 3's payload and this stage's gradients.
    if (U == 0 && more) wait_loads<C * GL + NR>();
    __syncthreads();
    if (U == 1) {
      r1 = r2;
      r2 = r2 + 1 == NB ? 0 : r2 + 1;
      if (c + 2 < count) g1 += gchunk;
    }
  };
  if (count) {
    fetch_raw(0, 0);
    if (count > 1) fetch_raw(1, 1);
    if (count > 2) fetch_raw(2, 2);
    load_grads(gbase, 0);
  }
  load_table<F>(s_tab, A.tab);
  if (count) {
    wait_loads<0>();
    __syncthreads();
    read_rows(0, 0, 0);
    look_up();
    weigh(0, 0);
    read_rows(0, 2, 0);
    look_up();
    weigh(0, 2);
    put(0);
    read_rows(1, 0, 1);  // of a single chunk there is none: what lies there is decoded, and not used
    look_up();
    weigh(1, 0);
    __syncthreads();  // chunk 0 is there, its payload read
    if (more) fetch_raw(3, 0);
    read_scales(0, 0);
#pragma unroll
    for (int c = 0; c < C; ++c) convert(0, c);
    load_grads(gbase, 1);
    read_w(0, 0, 0, 0);
    // Of a SIMD's two waves the first goes first: while it works on its addresses the other has the matrix cores.
    if (wave < 4) __builtin_amdgcn_s_setprio(1);
    for (int c = 0; c < count; ++c) {
      stage(std::integral_constant<int, 0>{}, c);
      stage(std::integral_constant<int, 1>{}, c);
    }
    wait_loads<0>();  // none is on its way to memory that another workgroup may be given
  }
  // tokens 4 q + k of tile c, columns 8 n + j of either half
  const int64_t tw = tt0 + wave * C;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const uint4 e4 = *reinterpret_cast<const uint4 *>(A.G.most + min((tw + c) * 16 + q * 4, A.G.ntile * 16 - 4));
    const uint32_t most[4] = {e4.x, e4.y, e4.z, e4.w};
#pragma unroll
    for (int j = 0; j < 16; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[j >> 3][j & 7][c][k] = ldexpf(acc[j >> 3][j & 7][c][k], ed + shift - grad_power(most[k], WIDE));
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t col = cb * 256 + h * 128 + 8 * n;
    if (LORA && split == 0) add_adapters<F32, C>(A, tw, col, acc[h]);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t t0 = (tw + c) * 16 + q * 4;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (t0 + k >= A.T) continue;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = acc[h][j][c][k];
        if (whole)
          store8u(A.out, !F32, (t0 + k) * cols + col, v);
        else
          store8u(A.partial + (rest * min(A.T, static_cast<int64_t>(TA * 16)) + t0 + k - tt0 * 16) * 256, 0, h * 128 + 8 * n, v);
      }
    }
  }
}

// The splits' sums, in their order: a workgroup has eight tokens of one tile of the rest.  Bound by memory: 64 tiles in 4
// splits 13 us (67 MB read, half of it from caches), 26 splits of 19 tokens' 5, a load's latency four times.
template <bool F32> __global__ void __launch_bounds__(256) rows_join_kernel(RowsArgs A) {
  const int64_t held = min(A.T, static_cast<int64_t>(A.plan.tiles) * 16), per = (held + 7) / 8, size = held * 256;
  const int64_t rest = blockIdx.x / per, i = blockIdx.x % per * 2048 + threadIdx.x * 8;
  const int64_t place = A.plan.full + rest, t = place / A.nb * A.plan.tiles * 16 + i / 256;
  if (t >= A.T) return;
  const float *from = A.partial + rest * A.plan.splits * size + i;
  float v[8] = {};
  for (int s0 = 0; s0 < A.plan.splits; s0 += 8) {
    float w[8][8];
#pragma unroll
    for (int s = 0; s < 8; ++s) load8u(from, 0, min(s0 + s, A.plan.splits - 1) * size, w[s]);
    __builtin_amdgcn_sched_barrier(0);  // all of them on their way together
#pragma unroll
    for (int s = 0; s < 8; ++s)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (s0 + s < A.plan.splits) v[j] += w[s][j];
  }
  store8u(A.out, !F32, (t * A.nb + place % A.nb) * 256 + i % 256, v);
}

// An empty sum's result (a fill by the runtime is no kernel, and would enter a captured graph as another node).
__global__ void __launch_bounds__(256) zero_kernel(uint16_t *p, size_t n) {
  for (size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<size_t>(gridDim.x) * 256)
    p[i] = 0;
}

template <int F, bool WIDE, int C, bool F32, bool LORA> void launch_tile(const RowsArgs &A, hipStream_t stream) {
  hipLaunchKernelGGL((rows_kernel<F, WIDE, C, F32, LORA>),
                     dim3(static_cast<unsigned>(A.plan.full + A.plan.rest * A.plan.splits)), dim3(512), 0, stream, A);
}

template <int F> void launch_fmt(int dtype, const RowsArgs &A, hipStream_t stream) {
  if (dtype == IQ_DTYPE_F32)
    return A.rank ? launch_tile<F, true, 1, true, true>(A, stream) : launch_tile<F, true, 1, true, false>(A, stream);
  if (A.nmat == 2)  // a gated block's
    return A.plan.tiles == 8 ? launch_tile<F, true, 1, false, false>(A, stream) : launch_tile<F, true, 2, false, false>(A, stream);
  if (A.plan.tiles == 8)
    return A.rank ? launch_tile<F, false, 1, false, true>(A, stream) : launch_tile<F, false, 1, false, false>(A, stream);
  A.rank ? launch_tile<F, false, 2, false, true>(A, stream) : launch_tile<F, false, 2, false, false>(A, stream);
}

}  // namespace

// The tiles of 128 or 256 tokens that cost least: whole rounds of them over 256 CUs, and the rest in as many splits of
// the rows as fill a round or do better.  A round is 8 us and per chunk of 64 rows what stands below, from 256 tiles of
// 88 and of 176 chunks (IQ2_XS; IQ1_S up to 9% less): 241 and 455 us with 128 tokens of fp16 gradients, 253 and 464 of
// fp32, 267 and 473 for dx in f32; with 256 tokens 317 and 638, and 333 and 686.  A split rest also costs the joining
// launch's 3 us and the way of its sums there and back (4 TB/s).  Its sums take 128 MiB at most: over six sizes of weights
// and up to 9,000 tokens that costs 0.1% of a call by this reckoning (64 MiB 0.7, none would take 327 MB in places).
RowsPlan plan_rows(int64_t T, int64_t nb, int64_t chunks, int dtype, bool wide) {
  struct Tile {
    int tiles;
    double chunk;
  };
  constexpr int64_t kMostBytes = int64_t(1) << 27;
  const bool f32 = dtype == IQ_DTYPE_F32;
  const Tile kinds[2] = {{8, f32 ? 2.6 : 2.5}, {16, wide ? 3.9 : 3.6}};
  const int64_t ntile = (T + 15) / 16;
  RowsPlan best{};
  size_t most = 0;
  double least = 0.0;
  for (int k = 0; k < (f32 ? 1 : 2); ++k) {
    const Tile &tile = kinds[k];
    const int64_t all = nb * ((ntile + tile.tiles - 1) / tile.tiles);
    const int64_t full = all / 256 * 256, rest = all - full, size = std::min(T, static_cast<int64_t>(tile.tiles) * 16) * 256 * 4;
    const int64_t splits = std::min(chunks, static_cast<int64_t>(64));
    // what any smaller T could take, so that a workspace for more tokens serves fewer
    most = std::max(most, static_cast<size_t>(std::min(all * splits * size, kMostBytes)));
    const double whole = static_cast<double>(full / 256) * (8.0 + static_cast<double>(chunks) * tile.chunk);
    for (int s = 1; s <= splits; ++s) {
      if (s > 1 && (!rest || rest * s * size > kMostBytes)) break;
      double us = whole;
      if (rest)
        us += static_cast<double>((rest * s + 255) / 256) * (8.0 + static_cast<double>((chunks + s - 1) / s) * tile.chunk);
      if (s > 1) us += 3.0 + static_cast<double>(s * rest * size) * 2.0 / 4e6;
      if (!best.tiles || us < least) {
        least = us;
        best = RowsPlan{tile.tiles, s > 1 ? full : all, s > 1 ? rest : 0, s, 0};
      }
    }
  }
  best.bytes = most;
  return best;
}

int launch_zero(void *p, size_t bytes, hipStream_t stream) {
  const size_t n = bytes / 2, wgs = (n + 2047) / 2048;
  if (!n) return IQ_OK;
  hipLaunchKernelGGL(zero_kernel, dim3(static_cast<unsigned>(wgs < 4096 ? wgs : 4096)), dim3(256), 0, stream,
                     static_cast<uint16_t *>(p), n);
  return run_launched() ? IQ_OK : IQ_ERR_HIP;
}

int launch_rows(int fmt, int dtype, const RowsArgs &A, hipStream_t stream) {
#define CALL(F) launch_fmt<F>(dtype, A, stream)
  IQ_BY_FMT(fmt, CALL)
#undef CALL
  if (!run_launched()) return IQ_ERR_HIP;
  if (A.plan.splits > 1) {
    const int64_t held = std::min(A.T, static_cast<int64_t>(A.plan.tiles) * 16);
    const dim3 wgs(static_cast<unsigned>(A.plan.rest * ((held + 7) / 8)));
    if (dtype == IQ_DTYPE_F32)
      hipLaunchKernelGGL(rows_join_kernel<true>, wgs, dim3(256), 0, stream, A);
    else
      hipLaunchKernelGGL(rows_join_kernel<false>, wgs, dim3(256), 0, stream, A);
    if (!run_launched()) return IQ_ERR_HIP;
  }
  return IQ_OK;
}

}  // namespace iq
