// iq_rows.hip -- dx = G W: gradients by encoded weights, summed over the weights'
// rows (iq_linear_backward, and iq_glu_backward for two weights one after the
// other).
//
// The matrix instruction wants eight consecutive rows of one column from a lane; a
// payload gives eight consecutive columns of one row.  A thread therefore decodes
// the same group of four consecutive rows, which makes two pairs of rows of each of
// its eight columns by byte permutations, and eight such columns are the eight
// operands that a group's lane has in eight instructions: operand j of half h holds
// columns 128 h + 8 n + j of a block, n the lane's place, so that its results are
// eight consecutive columns of dx.  Decoded once for all tokens of a workgroup, the
// weights reach the waves through LDS.
//
// d differs from row to row, so it cannot scale a sum: the operand is the whole
// weight, d m v, in fp16 under one power of two for the payload (bf16), or the sum of
// two fp16 values (f32, three products; the sums of four chunks are added to the whole
// ones, so that fewer additions round at a whole sum's size).

#include <type_traits>

#include "iq_train.hpp"

namespace iq {
namespace {

// acc[j][c] += p A of the adapters that the wave's tokens (tiles tt .. tt + C - 1) name, columns col + j of the lane's
// eight.  32 ranks at a time: a lane has eight ranks of its eight columns, which byte permutations make operands of
// (bf16; p is the sum of three bf16 values, without a rounding), or four ranks at a time on the fp32 cores.  Rows of
// tokens with other adapters are zeros; where A is not finite, 0 * A would reach them, and what they give is dropped.
template <int P, int C>
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
    for (int r0 = 0; r0 < A.rank; r0 += P == 1 ? 32 : 4) {
      const uint32_t *wild = A.wild + (static_cast<int64_t>(a) * tiles + (r0 >> 4)) * A.nb + cb;
      const bool drop = wild[0] | wild[P == 1 && r0 + 16 < A.rank ? A.nb : 0];
      if constexpr (P == 1) {
        const uint16_t *from = static_cast<const uint16_t *>(A.a) + static_cast<int64_t>(a) * A.rank * cols + col;
        u32x4 w[8];  // ranks r0 + 8 q + i; past the last p is zero
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = ldu<u32x4>(from + min(r0 + 8 * q + i, A.rank - 1) * cols);
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
            f32x4 d = acc[j][c];
#pragma unroll
            for (int k = 0; k < 3; ++k)
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

// Waves: 4 token groups (of C tiles) by H halves of a block's columns.  LORA: with adapters.
//
// A stage is a step of 32 rows, a chunk two.  Chunk c + 1 is decoded in the odd stage of chunk c - 1 (a thread's first
// two rows) and the even stage of chunk c (the others, and both pairs to LDS).  Its payload is requested in an odd
// stage NA chunks before chunk c + 1's, and the gradients NA - 1 stages ahead.  As in iq_glu's tiles the work stands
// between the matrix instructions, and operands are read a group of four ahead, a stage's first before the barrier that
// opens it.
//
// Two weights of 17,408 x 5,120 (IQ1_M), 4,096 tokens: 1,379 us, 1.06 PFLOP/s (a library's large product of fp16: 1.20),
// matrix cores busy 0.46 of the time, LDS 0.45, waves waiting 0.28; 5,120 x 17,408 (IQ1_S) with four adapters 715, 1.02.
// Without the decode a chunk of IQ1_S takes 1.65 us of its 2.3, with a quarter of the products 1.85: neither bounds it
// alone.
// Larger tiles would decode less for each product, but 512 tokens' gradients do not fit LDS beside a codebook.
template <int F, int P, int C, int H, bool LORA>
__global__ void __launch_bounds__(256 * H, H) rows_kernel(RowsArgs A) {
  constexpr int NW = 4 * H, NT = 64 * NW, TA = 4 * C, NP = TA * P, NPW = (NP + NW - 1) / NW;
  constexpr int NA = Geo<F>::N > 512 ? 3 : 4;  // stages of gradients in LDS, beside a large codebook one fewer
  constexpr int W = (Geo<F>::BYTES + 5) / 4, NR = (64 * W + NT - 1) / NT;  // words of a row's block, a thread's share
  constexpr int NB = NA - 1;                    // chunks of payload in LDS
  __shared__ uint4 s_tab[Geo<F>::N];
  __shared__ u32x4 s_a[NA][NP * 64];            // [stage % NA][tile][part][lane]
  __shared__ u32x4 s_b[2][2][H * 8 * P * 64];   // [chunk % 2][step][half][column j][part][lane]
  __shared__ uint32_t s_raw[NB][NR * NT];       // [chunk % NB][row][word]
  const uint32_t grad_at = IQ_LDS_ADDRESS(s_a), raw_at = IQ_LDS_ADDRESS(s_raw);
  load_table<F>(s_tab, A.tab);
  const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wt = wave / H, wh = wave % H;
  const bool whole = blockIdx.x < A.plan.full;
  const int64_t rest = blockIdx.x - A.plan.full, place = whole ? blockIdx.x : A.plan.full + rest / A.plan.splits;
  const int splits = whole ? 1 : A.plan.splits, split = whole ? 0 : static_cast<int>(rest % A.plan.splits);
  const int64_t across = place % A.plan.across, tt0 = place / A.plan.across * TA;
  const int64_t cb = across / (2 / H), cols = A.nb * 256, rowbytes = A.nb * Geo<F>::BYTES;
  const int half0 = H == 2 ? 0 : static_cast<int>(across & 1);  // the first half that the workgroup takes
  const int64_t per = (A.rows + 63) / 64, chunks = per * A.nmat;
  const int64_t share = (chunks + splits - 1) / splits, ch0 = split * share;
  const int count = static_cast<int>(max(min(share, chunks - ch0), static_cast<int64_t>(0)));
  const int ew = weight_exponent(A.B);
  const int unit = 15 - ew - (Geo<F>::IQ1 ? 0 : 3);
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
  // Step `step` of the gradients of the chunk at `from` into buffer `buf`.
  const char *gbase = reinterpret_cast<const char *>(A.G.g16) + (ch0 * A.G.ntile + tt0) * P * 2048;
  const int64_t gchunk = A.G.ntile * P * 2048;
  uint32_t goff[NPW];
#pragma unroll
  for (int i = 0; i < NPW; ++i) {
    const int p = i * NW + wave, most = static_cast<int>(min(A.G.ntile - tt0, static_cast<int64_t>(TA))) - 1;
    goff[i] = static_cast<uint32_t>((min(p / P, most) * P + p % P) * 2048 + lane * 16);
  }
  const auto fetch = [&](const char *from, int step, int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NPW; ++i)
      if (NP % NW == 0 || i * NW + wave < NP)
        load_to_lds(from + step * 1024, goff[i], grad_at + (buf * NP + i * NW + wave) * 1024);
  };
  // The thread's group and four rows of each chunk: fields and entries of two rows at a time, weights, and both pairs
  // of rows to operand [quad / 8][wave % H][column], lane 16 ((quad % 8) / 2) + n, half quad % 2.
  const int group = (half0 + wave % H) * 16 + n, quad = (wave / H) * 4 + q;
  Fields f[2];
  uint4 e[2];
  uint32_t hi[4][4], lo[4][4];
  const int odd0 = static_cast<int>(reinterpret_cast<uintptr_t>(p0)) & 2, odd1 = static_cast<int>(reinterpret_cast<uintptr_t>(p1)) & 2;
  const auto read_rows = [&](int c, int j0, int buf) __attribute__((always_inline)) {
    bool second;
    const int64_t row0 = chunk_of(c, second);
    const int most = static_cast<int>(min(A.rows - 1 - row0, static_cast<int64_t>(63)));
    const int step = static_cast<int>(rowbytes) & 2, odd = second ? odd1 : odd0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = quad * 4 + j0 + j, half = ((min(r, most) << 1) & step) ^ odd;  // the block's address modulo four
      f[j] = read_fields<F>(reinterpret_cast<const uint8_t *>(&s_raw[buf][r * W]) + half, group, half);
    }
  };
  const auto look_up = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 2; ++j) e[j] = s_tab[f[j].k];
  };
  const auto weigh = [&](int j0) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 2; ++j) whole_weights<F, P>(f[j], e[j], unit, hi[j0 + j], lo[j0 + j]);
  };
  const auto put = [&](int c) __attribute__((always_inline)) {
    uint2 *to = reinterpret_cast<uint2 *>(s_b[c & 1][quad / 8]) +
                ((wave % H) * 8 * P * 64 + (quad % 8) / 2 * 16 + n) * 2 + quad % 2;
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
      for (int k = 0; k < 2; ++k) {  // column p + 4 k
        const uint32_t sel = k ? 0x07060302u : 0x05040100u;
#pragma unroll
        for (int part = 0; part < P; ++part) {
          const uint32_t(&v)[4][4] = part ? lo : hi;
          to[((p + 4 * k) * P + part) * 128] = make_uint2(__builtin_amdgcn_perm(v[1][p], v[0][p], sel),
                                                          __builtin_amdgcn_perm(v[3][p], v[2][p], sel));
        }
      }
  };
  constexpr int G = P == 1 ? 4 : 2, NG = 8 / G;  // columns whose operands are read together
  half8v x[2][C][P], w[2][G][P];
  const auto read_x = [&](int u, int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int p = 0; p < P; ++p) x[u][c][p] = __builtin_bit_cast(half8v, s_a[buf][((wt * C + c) * P + p) * 64 + lane]);
  };
  const auto read_w = [&](int u, int g, int c, int step) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < G; ++j)
#pragma unroll
      for (int p = 0; p < P; ++p)
        w[u][j][p] = __builtin_bit_cast(half8v, s_b[c & 1][step][((wh * 8 + g * G + j) * P + p) * 64 + lane]);
  };

  f32x4 acc[8][C], part[P == 2 ? 8 : 1][C];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int c = 0; c < C; ++c) acc[j][c] = part[j % (P == 2 ? 8 : 1)][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  int a0 = 0;  // the buffer of the stage's gradients
  const auto buffer = [&](int ahead) __attribute__((always_inline)) {
    const int b = a0 + ahead;
    return b >= NA ? b - NA : b;
  };
  int r1 = 1 % NB, r2 = 2 % NB;  // the buffers of the payload of chunks c + 1 and c + 2
  const char *g1 = gbase + (count > 1 ? gchunk : 0), *g2 = g1 + (count > 2 ? gchunk : 0);  // their gradients; past the last its
  const auto stage = [&](auto step, int c) __attribute__((always_inline)) {
    constexpr int U = decltype(step)::value;
    const int next = c + 1 + U;  // the chunk whose rows are decoded in this stage
    read_rows(next, U ? 0 : 2, U ? r2 : r1);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      constexpr int first = U * NG;  // groups alternate between two sets of registers
      if (g + 1 < NG) {
        read_w((first + g + 1) & 1, g + 1, c, U);
      } else {  // the next stage's first
        read_x(U ^ 1, buffer(1));
        read_w((first + g + 1) & 1, 0, c + U, U ^ 1);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (g + 1 == NG) {
        weigh(U ? 0 : 2);
        if (U == 0) put(next);
      }
#pragma unroll
      for (int j = 0; j < G; ++j)
#pragma unroll
        for (int cc = 0; cc < C; ++cc) {
          f32x4 &to = P == 2 ? part[(g * G + j) % (P == 2 ? 8 : 1)][cc] : acc[g * G + j][cc];
          const half8v(&ww)[P] = w[(first + g) & 1][j];
          to = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[U][cc][0], ww[0], to, 0, 0, 0);
          if (P == 2) {
            to = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[U][cc][P - 1], ww[0], to, 0, 0, 0);
            to = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[U][cc][0], ww[P - 1], to, 0, 0, 0);
          }
        }
      __builtin_amdgcn_sched_barrier(0);
      if (g == 0) {
        look_up();
        fetch(NA == 3 || U == 0 ? g1 : g2, NA == 3 ? U : U ^ 1, buffer(NA - 1));
        if (U == 1) fetch_raw(c + NA, r1);  // chunk c + 1's is decoded
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (P == 2 && U == 1 && ((c & 3) == 3 || c + 1 == count)) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int cc = 0; cc < C; ++cc) {
          f32x4 &p = part[j % (P == 2 ? 8 : 1)][cc];
          acc[j][cc] += p;
          p = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
    }
    // What the stage after the next needs has to be there.  Four buffers: the gradients requested a stage ago, so that
    // those of this stage and a payload requested since may be on their way (as many as the wave has: with more allowed,
    // the end of an earlier payload could be among them); three: the gradients of this stage, but not a payload requested
    // after them.
    if (NA == 4 && (NP % NW == 0 || wave < NP % NW))
      wait_loads<NPW + NR>();
    else if (NA == 4)
      wait_loads<NPW - 1 + NR>();
    else if (U == 1)
      wait_loads<NR>();
    else
      wait_loads<0>();
    __syncthreads();
    a0 = buffer(1);
    if (U == 1) {
      const int next2 = r2 + 1 == NB ? 0 : r2 + 1;
      r1 = r2;
      r2 = next2;
      g1 = g2;
      if (c + 3 < count) g2 += gchunk;
    }
  };
  if (count) {
    fetch_raw(0, 0);
    fetch_raw(1, 1 % NB);
#pragma unroll
    for (int s = 0; s < NA - 1; ++s) fetch(s < 2 ? gbase : g1, s & 1, s);
    wait_loads<0>();
    __syncthreads();
    read_rows(0, 0, 0);
    look_up();
    weigh(0);
    read_rows(0, 2, 0);
    look_up();
    weigh(2);
    put(0);
    read_rows(1, 0, 1 % NB);
    look_up();
    weigh(0);
    __syncthreads();  // chunk 0 is there, its payload read
    for (int c = 2; c < NA; ++c) fetch_raw(c, c % NB);
    wait_loads<0>();
    __syncthreads();
    read_x(0, 0);
    read_w(0, 0, 0, 0);
    // Of a SIMD's two waves the first goes first: while it works on its addresses the other has the matrix cores.
    if (wave < NW / 2) __builtin_amdgcn_s_setprio(1);
    for (int c = 0; c < count; ++c) {
      stage(std::integral_constant<int, 0>{}, c);
      stage(std::integral_constant<int, 1>{}, c);
    }
    wait_loads<0>();  // none is on its way to memory that another workgroup may be given
  }
  // tokens 4 q + k of tile c, columns 8 n + j of the wave's half
  const int64_t col = cb * 256 + (half0 + wh) * 128 + 8 * n, tw = tt0 + wt * C;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int4 e4 = *reinterpret_cast<const int4 *>(A.G.ex + min((tw + c) * 16 + q * 4, A.G.ntile * 16 - 4));
    const int ex[4] = {e4.x, e4.y, e4.z, e4.w};
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[j][c][k] = ldexpf(acc[j][c][k], ex[k] + ew - 15);
  }
  if (LORA && split == 0) add_adapters<P, C>(A, tw, col, acc);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int64_t t0 = (tw + c) * 16 + q * 4;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (t0 + k >= A.T) continue;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = acc[j][c][k];
      if (whole)
        store8u(A.out, P == 1, (t0 + k) * cols + col, v);
      else
        store8u(A.partial + (rest * TA * 16 + t0 + k - tt0 * 16) * (128 * H), 0, wh * 128 + 8 * n, v);
    }
  }
}

// The splits' sums, in their order: a workgroup has 2,048 values of one tile of the rest.  Bound by memory: 64 tiles in 4
// splits 13 us (67 MB read, half of it from caches), 26 splits of 19 tokens' 5, a load's latency four times.
template <int P> __global__ void __launch_bounds__(256) rows_join_kernel(RowsArgs A) {
  constexpr int width = P == 2 ? 128 : 256;
  const int64_t size = static_cast<int64_t>(A.plan.tiles) * 16 * width, per = size / 2048;
  const int64_t rest = blockIdx.x / per, i = blockIdx.x % per * 2048 + threadIdx.x * 8;
  const int64_t place = A.plan.full + rest, t = place / A.plan.across * A.plan.tiles * 16 + i / width;
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
  store8u(A.out, P == 1, t * A.nb * 256 + place % A.plan.across * width + i % width, v);
}

// An empty sum's result (a fill by the runtime is no kernel, and would enter a captured graph as another node).
__global__ void __launch_bounds__(256) zero_kernel(uint16_t *p, size_t n) {
  for (size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<size_t>(gridDim.x) * 256)
    p[i] = 0;
}

template <int F, int P, int C, int H, bool LORA> void launch_tile(const RowsArgs &A, hipStream_t stream) {
  hipLaunchKernelGGL((rows_kernel<F, P, C, H, LORA>),
                     dim3(static_cast<unsigned>(A.plan.full + A.plan.rest * A.plan.splits)), dim3(256 * H), 0, stream, A);
}

template <int F, bool LORA> void launch_fmt(int dtype, const RowsArgs &A, hipStream_t stream) {
  if (dtype == IQ_DTYPE_F32) return launch_tile<F, 2, (Geo<F>::N > 1024 ? 1 : 2), 1, LORA>(A, stream);
  if (A.plan.tiles == 4) return launch_tile<F, 1, 1, 2, LORA>(A, stream);
  if (A.plan.tiles == 8) return launch_tile<F, 1, 2, 2, LORA>(A, stream);
  if (A.plan.tiles == 12) return launch_tile<F, 1, 3, 2, LORA>(A, stream);
  launch_tile<F, 1, 4, 2, LORA>(A, stream);
}

}  // namespace

// The tiles of 64 to 256 tokens that cost least: whole rounds of them over 256 CUs, and the rest in as many splits of
// the rows as fill a round or do better.  A round is 8 us and per chunk of 64 rows what stands below, from 256 tiles of
// 88 and of 176 chunks (IQ2_XS; IQ1 within 15%): 155 and 294 us with 64 tokens, 153 and 292 with 128, 194 and 363 with
// 192, 208 and 413 with 256 (f32: 458 for 176 chunks of 128 tokens by 128 columns, 383 of 64 beside a codebook of
// 2,048 entries).  A split rest also costs the joining launch's 3 us and the way of its sums there and back (4 TB/s).
// With 192 tokens as well 5,632 x 5,120 (IQ2_XS) by 1,500 tokens took 128 us, without 150.
RowsPlan plan_rows(int fmt, int64_t T, int64_t cols, int64_t chunks, int dtype) {
  struct Tile {
    int tiles;
    double chunk;
  };
  const bool f32 = dtype == IQ_DTYPE_F32;
  constexpr Tile bf16s[4] = {{4, 1.55}, {8, 1.6}, {12, 1.95}, {16, 2.3}};
  const Tile single = {kCodebook[fmt] > 1024 ? 4 : 8, kCodebook[fmt] > 1024 ? 2.0 : 2.7};
  const int64_t ntile = (T + 15) / 16;
  RowsPlan best{};
  double least = 0.0;
  for (int k = 0; k < (f32 ? 1 : 4); ++k) {
    const Tile &tile = f32 ? single : bf16s[k];
    const int64_t across = cols / (f32 ? 128 : 256), all = across * ((ntile + tile.tiles - 1) / tile.tiles);
    const int64_t full = all / 256 * 256, rest = all - full, size = static_cast<int64_t>(tile.tiles) * 16 * (f32 ? 128 : 256) * 4;
    const double whole = static_cast<double>(full / 256) * (8.0 + static_cast<double>(chunks) * tile.chunk);
    for (int s = 1; s <= 64 && s <= chunks; ++s) {
      if (s > 1 && !rest) break;
      double us = whole;
      if (rest)
        us += static_cast<double>((rest * s + 255) / 256) * (8.0 + static_cast<double>((chunks + s - 1) / s) * tile.chunk);
      if (s > 1) us += 3.0 + static_cast<double>(s * rest * size) * 2.0 / 4e6;
      if (!best.tiles || us < least) {
        least = us;
        best = RowsPlan{tile.tiles, across, s > 1 ? full : all, s > 1 ? rest : 0, s,
                        s > 1 ? static_cast<size_t>(s * rest * size) : 0};
      }
    }
  }
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
#define CALL(F) A.rank ? launch_fmt<F, true>(dtype, A, stream) : launch_fmt<F, false>(dtype, A, stream)
  IQ_BY_FMT(fmt, CALL)
#undef CALL
  if (!run_launched()) return IQ_ERR_HIP;
  if (A.plan.rest) {
    const int64_t size = static_cast<int64_t>(A.plan.tiles) * 16 * (dtype == IQ_DTYPE_F32 ? 128 : 256);
    const dim3 wgs(static_cast<unsigned>(A.plan.rest * (size / 2048)));
    if (dtype == IQ_DTYPE_F32)
      hipLaunchKernelGGL(rows_join_kernel<2>, wgs, dim3(256), 0, stream, A);
    else
      hipLaunchKernelGGL(rows_join_kernel<1>, wgs, dim3(256), 0, stream, A);
    if (!run_launched()) return IQ_ERR_HIP;
  }
  return IQ_OK;
}

}  // namespace iq
