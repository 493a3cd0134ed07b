// iq_backward.hip -- iq_linear_backward: the gradients by an encoded projection's
// tokens and by its low-rank adapters (include/iq_train.h).
//
// Launches: dy and the adapters into operand order, with the bound on the weights;
// the rank-wide products p = s dy B and v = s x A^T; dx (iq_rows.hip, with p A added
// to its sums); and dA, dB as sums over the tokens.

#include "iq_train.hpp"

namespace iq {
namespace {

struct Adapters {
  const void *a, *b;
  const float *scale;
  const int32_t *ids;
  int n, rank;
};

struct BackPrepArgs {
  const void *dy;
  int dtype, fmt, bytes;
  int64_t T, rows, nb, nconv;
  const uint8_t *packed;
  Grads G;
  Bound B;
  Codebooks books;
  int convert;  // dx is wanted
  Adapters L;
  // OUT, A and B for the rank-wide products [adapter][tile of 16 ranks][64 of k][half][lane][8], of dtype: lane 16 q + n
  // of half h holds rank n, k = 16 q + 8 h on; zeros past the last rank and row
  void *ao, *bo;
  int tiles;
  int64_t cols, rowpad;
  uint32_t *wild;  // OUT [adapter][tile of 16 ranks][256 columns of A]: not all of them are finite
};

// One wave brings one token's gradient into the order of Grads.
template <int P>
__device__ __forceinline__ void convert_grad(const BackPrepArgs &A, int64_t t, int lane) {
  const int64_t all = row_chunks(A.rows) * 64;
  const auto load = [&](int64_t r, float (&v)[8]) __attribute__((always_inline)) {
    if (r + 8 <= A.rows) {
      load8u(A.dy, A.dtype, t * A.rows + r, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = r + j < A.rows ? load1(A.dy, A.dtype, t * A.rows + r + j) : 0.0f;
    }
  };
  uint32_t most = 0;
  if (P == 1) {
    most = row_exponent(A.dy, A.dtype, A.rows, t, lane) << 23;
    const int n = grad_power(most, false);
    for (int64_t r = lane * 8; r < all; r += 512) {
      float v[8];
      load(r, v);
      half8v o;
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = static_cast<_Float16>(ldexpf(v[j], n));
      const int in = static_cast<int>(r & 63);
      *reinterpret_cast<half8v *>(static_cast<_Float16 *>(A.G.g) + ((r >> 6) * A.G.ntile + (t >> 4)) * 1024 +
                                  ((in >> 5) * 64 + ((in & 31) >> 3) * 16 + (t & 15)) * 8) = o;
    }
  } else {
    for (int64_t r = lane * 8; r < all; r += 512) {
      float v[8];
      load(r, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) most = max_bits(most, v[j]);
      put_grads(A.G, 0, t, r, v);
    }
    most = wave_max_u32(most);
  }
  if (lane == 0) A.G.most[t] = most;
}

// A wave a token of dy, which it goes through twice (the largest magnitude first).  4,096 tokens of 5,120 columns, four
// adapters of rank 32 beside 17,408 columns: 30 us for 107 MB, 3.6 TB/s; 2,048 of 2,048 7 us.
template <int P> __global__ void __launch_bounds__(512) back_prep_kernel(BackPrepArgs A) {
  __shared__ uint32_t s_red[8];
  int64_t w = blockIdx.x;
  if (A.convert) {
    if (w < kScaleSlots) {
      const uint8_t *const packed[2] = {A.packed, A.packed};
      bound_scales(A.fmt, A.bytes, packed, 1, A.rows * A.nb, A.B, static_cast<int>(w), s_red);
      return;
    }
    w -= kScaleSlots;
    if (w < A.nconv) {
      const int64_t t = w * 8 + (threadIdx.x >> 6);
      if (t < A.T) convert_grad<P>(A, t, threadIdx.x & 63);
      return;
    }
    w -= A.nconv;
    if (w < A.books.wg[0]) {
      convert_codebook(A.books, static_cast<int>(w));
      bound_codebook(A.books, A.B, static_cast<int>(w), s_red);
      return;
    }
    w -= A.books.wg[0];
  }
  // 256 rows of B or columns of A, of a tile of 16 ranks
  int64_t per = A.rowpad >> 8;
  const bool of_a = w >= A.L.n * A.tiles * per;
  if (of_a) {
    w -= A.L.n * A.tiles * per;
    per = A.cols >> 8;
  }
  const int64_t tile = w / per, a = tile / A.tiles;
  const int lane = threadIdx.x & 63, h = (threadIdx.x >> 6) & 1, rank = static_cast<int>(tile % A.tiles) * 16 + (lane & 15);
  const int64_t block = w % per * 4 + (threadIdx.x >> 7), k = block * 64 + (lane >> 4) * 16 + h * 8;
  float v[8];
  if (of_a && rank < A.L.rank) {
    load8u(A.L.a, P == 1, (a * A.L.rank + rank) * A.cols + k, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = !of_a && rank < A.L.rank && k + j < A.rows ? load1(A.L.b, P == 1, (a * A.rows + k + j) * A.L.rank + rank) : 0.0f;
  }
  if (of_a) {
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) bad |= !finite_f(v[j]);
    const int any = __syncthreads_or(bad);
    if (threadIdx.x == 0) A.wild[w] = any;
  }
  const int64_t to = ((tile * per * 4 + block) * 2 + h) * 512 + lane * 8;
  if (P == 1) {  // as they were: a NaN keeps its bits' top half
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = __builtin_amdgcn_perm(__float_as_uint(v[2 * j + 1]), __float_as_uint(v[2 * j]), 0x07060302u);
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(of_a ? A.ao : A.bo) + to) = make_uint4(o[0], o[1], o[2], o[3]);
  } else {
    __builtin_memcpy(static_cast<float *>(of_a ? A.ao : A.bo) + to, v, 32);
  }
}

// ---------------------------------------------------------------------------
// Rank-wide products
// ---------------------------------------------------------------------------
struct Shrink {
  Source s;         // tokens [T, k]
  int64_t k;
  const void *w;    // adapters as BackPrepArgs has them
  int64_t kpad;     // a multiple of 256
  float *out;       // f32: [ranks, in 32s][tpad]
  uint16_t *parts;  // three bf16 values each [32 tokens][16 ranks, 32s of them][3][lane][8]
};
struct ShrinkArgs {
  Shrink of[2];  // dy by B, x by A
  int dtype;
  int64_t T, tpad;
  Adapters L;
  int rgroups, slots;  // 32 ranks a workgroup
  int32_t *ids;  // OUT [tpad]: the tokens' adapters, -1 for none or another id
  int2 *range;   // OUT [tpad / 32]: the least and the largest of 32 tokens'
  uint16_t *parts;  // OUT, bf16: p [tile of 16 tokens][32 ranks][3][lane][8]
  int32_t *status;
};

// Eight values of a source from column k on; past the row's end zeros.
__device__ __forceinline__ void source8(const Source &s, int64_t cols, int64_t t, int64_t k, float v[8]) {
  const int64_t at = t * cols + k;
  if (s.ex) {  // whole blocks of 32
    decode_codes(ldu<uint2>(static_cast<const int8_t *>(s.x) + at), s.ex[t * (cols >> 5) + (k >> 5)] - 133, v);
  } else if (k + 8 <= cols) {
    load8u(s.x, s.dtype, at, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = k + j < cols ? load1(s.x, s.dtype, at + j) : 0.0f;
  }
}
// The same in bf16, exact for bf16 tokens and checkpoints.
__device__ __forceinline__ bf16x8 source8_bf16(const Source &s, int64_t cols, int64_t t, int64_t k) {
  if (!s.ex && k + 8 <= cols) return ldu<bf16x8>(static_cast<const uint16_t *>(s.x) + t * cols + k);
  float v[8];
  source8(s, cols, t, k, v);
  u32x4 o;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    o[j] = __builtin_amdgcn_perm(__float_as_uint(v[2 * j + 1]), __float_as_uint(v[2 * j]), 0x07060302u);
  return __builtin_bit_cast(bf16x8, o);
}

// Eight values of a checkpoint in bf16 (exact).
__device__ __forceinline__ bf16x8 codes_bf16(uint32_t lo, uint32_t hi, int e) {
  float v[8];
  decode_codes(make_uint2(lo, hi), e - 133, v);
  u32x4 o;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    o[j] = __builtin_amdgcn_perm(__float_as_uint(v[2 * j + 1]), __float_as_uint(v[2 * j]), 0x07060302u);
  return __builtin_bit_cast(bf16x8, o);
}

enum SourceKind { FROM_F32, FROM_BF16, FROM_CHECKPOINT };
// 4,096 tokens, 5,120 and 17,408 columns, four adapters of rank 32: 63 us with an adapter's tokens together, 130 in random
// order; 2,048 tokens, 2,048 and 5,632 columns, eight adapters of rank 16 24 and 53.  Each token's values once, from
// memory, would take 22 of the 63.  With the tokens together one slot of eight finds work, 256 workgroups of 2,048, of
// which the 128 of x A^T are 3.4 times as long as those of dy B; in random order each adapter among 32 tokens goes through
// their rows again.  Factors in operand order, 1 KiB in a row, made 84 us of 108.
//
// 32 tokens (A, two tiles) by 32 ranks (B) of the adapter of token `slot`, K split
// over the eight waves, each lane 16 columns at a time (64 bytes of a row a load);
// results of tokens with other adapters are dropped.  Nothing in the loop depends on the kind of tokens or on a row's
// end: a value that one of two branches loads is waited for where they meet.
// (Each product is a call of its own: of a chosen one the compiler would not see that its pointers are to global memory.)
template <int KIND, bool BF16>
__device__ __forceinline__ void shrink(const ShrinkArgs &A, const Shrink &S, bool of_x, int first, int64_t w, f32x4 *s_red) {
  const int64_t tt = w / A.rgroups;
  const int rg = static_cast<int>(w % A.rgroups), r0 = rg * 32;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, q = lane >> 4;
  const int64_t mytok = tt * 32 + (lane & 31);
  const bool once = first == 0 && rg == 0 && !of_x && threadIdx.x < 64;
  int mine = -1;
  if (mytok < A.T) {
    const int id = A.L.ids[mytok];
    if (id >= 0 && id < A.L.n)
      mine = id;
    else if (id != -1 && once)
      raise_status(A.status, ST_BADID);
  }
  if (once) {
    int least = mine, most = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      least = min(least, __shfl_xor(least, d, 64));
      most = max(most, __shfl_xor(most, d, 64));
    }
    if (lane < 32) A.ids[mytok] = mine;
    if (lane == 0) A.range[tt] = make_int2(least, most);
  }
  const uint32_t with = static_cast<uint32_t>(__ballot(mine >= 0));  // the tokens twice, once in either half of the wave
  // Value r of token tok's 32 in fp32, and as the three bf16 values that add up to it: in the order of the operands of
  // the sums over tokens, and of p for dx.
  const auto put_ranks = [&](int64_t step, int tok, int r, float f) __attribute__((always_inline)) {
    if (S.out) S.out[(r0 + r) * A.tpad + step * 32 + tok] = f;
    uint16_t *u = S.parts + ((step * A.rgroups + rg) * 2 + (r >> 4)) * 1536 + ((tok >> 3) * 16 + (r & 15)) * 8 + (tok & 7);
    uint16_t *v = A.parts + ((2 * step + (tok >> 4)) * A.rgroups + rg) * 1536 + ((r >> 3) * 16 + (tok & 15)) * 8 + (r & 7);
#pragma unroll
    for (int d = 0; d < 3; ++d) {
      const uint32_t top = __float_as_uint(f) & 0xffff0000u;
      u[d * 512] = static_cast<uint16_t>(top >> 16);
      if (BF16 && !of_x) v[d * 512] = static_cast<uint16_t>(top >> 16);
      f = finite_f(f) ? f - __uint_as_float(top) : 0.0f;  // inf - inf would be NaN
    }
  };
  if (first == 0) {  // zeros for tokens without an adapter
    const int tok = threadIdx.x & 31;
    if (!((with >> tok) & 1u))
      for (int r = threadIdx.x >> 5; r < 32; r += 16) put_ranks(tt, tok, r, 0.0f);
  }
  for (int slot = first; slot < 32; slot += A.slots) {
    const int a = __builtin_amdgcn_readlane(mine, slot);
    const uint32_t group = static_cast<uint32_t>(__ballot(mine == a));
    if (a < 0 || (group & ((1u << slot) - 1u))) continue;  // done with an earlier token
    const bool tile[2] = {(group & 0xffffu) != 0, (group >> 16) != 0};
    const int tiles = (A.L.rank + 15) >> 4;
    int64_t t[2], wr[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {  // rows of other tokens read this one's
      t[r] = tt * 32 + (((group >> (16 * r + n)) & 1u) ? 16 * r + n : slot);
      wr[r] = (static_cast<int64_t>(a) * tiles + min(2 * rg + r, tiles - 1)) * S.kpad * 16 + lane * 8;
    }
    f32x4 acc[4] = {};  // [token tile][rank tile]
    if constexpr (BF16) {
      // A round of the waves is 512 columns; two rounds are on their way while one multiplies (past the end the last
      // columns again).
      constexpr int H = KIND == FROM_CHECKPOINT ? 1 : 2;  // loads of a lane's 16 columns
      const int64_t whole = S.k & ~int64_t(63);
      const uint8_t *row[2], *ex[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        row[r] = static_cast<const uint8_t *>(S.s.x) + t[r] * S.k * H;
        ex[r] = S.s.ex + t[r] * (S.k >> 5);
      }
      u32x4 x[3][2][H], b[3][2][2];
      int e[3][2];
      const auto load = [&](int u, int64_t k0) __attribute__((always_inline)) {
        const int64_t block = min(k0, whole - 64), k = block + q * 16;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
          for (int h = 0; h < H; ++h) x[u][r][h] = ldu<u32x4>(row[r] + k * H + 16 * h);
          if (KIND == FROM_CHECKPOINT) e[u][r] = ex[r][k >> 5];
#pragma unroll
          for (int h = 0; h < 2; ++h) b[u][r][h] = ldu<u32x4>(static_cast<const uint16_t *>(S.w) + wr[r] + block * 16 + 512 * h);
        }
      };
      const auto multiply = [&](int i, bf16x8 v, const u32x4 &w) __attribute__((always_inline)) {
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, __builtin_bit_cast(bf16x8, w), acc[i], 0, 0, 0);
      };
      if (wave * 64 < whole) {
        load(0, wave * 64);
        load(1, wave * 64 + 512);
      }
      for (int64_t k0 = wave * 64; k0 < whole; k0 += 3 * 512)
#pragma unroll
        for (int u = 0; u < 3; ++u) {
          if (k0 + u * 512 >= whole) break;
          load((u + 2) % 3, k0 + (u + 2) * 512);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const u32x4 &w = x[u][r][h % H];
              const bf16x8 v = H == 1 ? codes_bf16(w[2 * h], w[2 * h + 1], e[u][r]) : __builtin_bit_cast(bf16x8, w);
#pragma unroll
              for (int i = 0; i < 2; ++i) multiply(2 * r + i, v, b[u][i][h]);
            }
        }
      if ((S.k & 63) && (whole >> 6) % 8 == wave) {  // the last columns (of dy: a checkpoint has whole blocks of 256)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const bf16x8 v = source8_bf16(S.s, S.k, t[r], whole + q * 16 + 8 * h);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              multiply(2 * r + i, v, ldu<u32x4>(static_cast<const uint16_t *>(S.w) + wr[i] + whole * 16 + 512 * h));
          }
      }
    } else {
      for (int64_t k0 = wave * 64; k0 < S.kpad; k0 += 512)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t k = k0 + q * 16 + 8 * h;
          float x[2][8], b[2][8];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            if (tile[r]) source8(S.s, S.k, t[r], k, x[r]);
            load8u(S.w, 0, wr[r] + k0 * 16 + 512 * h, b[r]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (tile[i >> 1])
#pragma unroll
              for (int j = 0; j < 8; ++j)
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i >> 1][j], b[i & 1][j], acc[i], 0, 0, 0);
        }
    }
    const float scale = A.L.scale ? A.L.scale[a] : 1.0f;
    const Split P{8, 1, wave, 0};
    reduce_split<4, 4>(acc, s_red, P, [&](int, int i, int l, const f32x4 &s) {
      const int r = (i & 1) * 16 + (l & 15), j = r0 + r;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int tok = (i >> 1) * 16 + (l >> 4) * 4 + k;
        if (!((group >> tok) & 1u)) continue;
        put_ranks(tt, tok, r, j < A.L.rank ? s[k] * scale : 0.0f);
      }
    });
  }
}

// KIND of x; dy is of its tensors' type (BF16).
template <int KIND, bool BF16> __global__ void __launch_bounds__(512) back_shrink_kernel(ShrinkArgs A) {
  __shared__ f32x4 s_red[8 * 4 * 64];
  const int64_t steps = (A.tpad >> 5) * A.rgroups, w = blockIdx.x % (2 * steps);
  const int first = static_cast<int>(blockIdx.x / (2 * steps));
  if (w < steps)
    shrink<BF16 ? FROM_BF16 : FROM_F32, BF16>(A, A.of[0], false, first, w, s_red);
  else
    shrink<KIND, BF16>(A, A.of[1], true, first, w - steps, s_red);
}

// ---------------------------------------------------------------------------
// Gradients by the adapters: sums over the tokens
// ---------------------------------------------------------------------------
struct Outer {
  Source s;        // [T, k]
  int64_t k, blocks;  // workgroups' columns: 128 each
  const float *w;         // f32: [ranks, in 32s][tpad]
  const uint16_t *parts;  // Shrink's
  void *out;       // by rank: [adapter][rank][k]; else [adapter][k][rank]
  int by_rank;
};
struct OuterArgs {
  Outer of[2];
  int64_t T, tpad;
  int dtype, rank, rgroups;
  const int32_t *ids;   // [tpad]
  const int2 *range;    // [tpad / 32]
  int splits;           // of the tokens
  float *partial;       // [split][both gradients], where there are several
  int64_t before[2], all;  // where each gradient begins in a split's, and its size
};

// The first of a lane's eight columns: the last lanes of a row overlap, so that every load is whole.
__device__ __forceinline__ int64_t outer_col(const Outer &O, int64_t blk, int m) {
  return max(min(blk * 128 + m * 8, O.k - 8), static_cast<int64_t>(0));
}

// out[j][c] = sum of w[j][t] s[t][c] over adapter a's tokens: 128 columns (A, eight a
// lane, brought from eight tokens each into operands by byte permutations) by 16 RT
// ranks (B; three bf16 values each).  The tokens in steps of 32 are dealt to the splits and their eight
// waves; a step whose tokens' adapters cannot be a is passed over, and where all
// are a none is masked out.  f32 tokens go through the fp32 cores.  4,096 tokens, 5,120
// and 17,408 columns, four adapters: 47 us with an adapter's tokens together, 149 in
// random order, where every adapter's workgroups go through all tokens; 2,048 tokens,
// 2,048 and 5,632 columns, one adapter 13, eight 14 and 45.  With the next step's loads
// ahead registers spill: 88 us.
struct OuterMemory {
  f32x4 red[8 * 4 * 64];
  float out[16][132];
};
template <int RT, int KIND>
__device__ __forceinline__ void outer_sums(const OuterArgs &A, const Outer &O, int which, int64_t blk, OuterMemory &mem) {
  const int a = blockIdx.y, rt0 = static_cast<int>(blockIdx.z / A.splits) * RT, split = blockIdx.z % A.splits;
  const int lane = threadIdx.x & 63, m = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t c0 = outer_col(O, blk, m);
  f32x4 acc[RT][8];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[r][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const auto one_step = [&](int64_t t0, bool all) __attribute__((always_inline)) {
    if constexpr (KIND == FROM_F32) {
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const int64_t t = t0 + 4 * s + q;
        const bool mine = all || A.ids[t] == a;  // false past the last token
        float x[8];
        if (O.k >= 8) {
          load8u(O.s.x, 0, (mine ? t : 0) * O.k + c0, x);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = j < O.k ? load1(O.s.x, 0, (mine ? t : 0) * O.k + j) : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = mine ? x[j] : 0.0f;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const float w = mine ? O.w[(static_cast<int64_t>(rt0 + r) * 16 + m) * A.tpad + t] : 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[r][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[j], w, acc[r][j], 0, 0, 0);
        }
      }
      return;
    }
    uint32_t mine = 255u;
    if (!all) {
      mine = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) mine |= static_cast<uint32_t>(A.ids[t0 + 8 * q + i] == a) << i;
    }
    u32x4 w[RT][3];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int k = 0; k < 3; ++k)
        w[r][k] = ldu<u32x4>(O.parts + ((t0 >> 5) * 2 * A.rgroups + rt0 + r) * 1536 + k * 512 + lane * 8);
    u32x4 x[8];
    if constexpr (KIND == FROM_CHECKPOINT) {
      uint2 codes[8];
      int e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t t = (mine >> i) & 1u ? t0 + 8 * q + i : 0;
        codes[i] = ldu<uint2>(static_cast<const int8_t *>(O.s.x) + t * O.k + c0);
        e[i] = O.s.ex[t * (O.k >> 5) + (c0 >> 5)];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float v[8];
        decode_codes(codes[i], e[i] - 133, v);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[i][j] = __builtin_amdgcn_perm(__float_as_uint(v[2 * j + 1]), __float_as_uint(v[2 * j]), 0x07060302u);
      }
    } else if (O.k >= 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[i] = ldu<u32x4>(static_cast<const uint16_t *>(O.s.x) + ((mine >> i) & 1u ? t0 + 8 * q + i : 0) * O.k + c0);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[i] = __builtin_bit_cast(u32x4, source8_bf16(O.s, O.k, (mine >> i) & 1u ? t0 + 8 * q + i : 0, 0));
    }
    if (!all) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (!((mine >> i) & 1u)) x[i] = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t keep = ((mine >> (2 * i)) & 1u ? 0xffffu : 0u) | ((mine >> (2 * i + 1)) & 1u ? 0xffff0000u : 0u);
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int k = 0; k < 3; ++k) w[r][k][i] &= keep;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t sel = j & 1 ? 0x07060302u : 0x05040100u;
      u32x4 o;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = __builtin_amdgcn_perm(x[2 * i + 1][j >> 1], x[2 * i][j >> 1], sel);
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int k = 0; k < 3; ++k)
          acc[r][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, o),
                                                              __builtin_bit_cast(bf16x8, w[r][k]), acc[r][j], 0, 0, 0);
    }
  };
  // The wave's steps, 64 looked at together: step i is tokens 32 (i dealt + its place) on.
  const int64_t steps = A.tpad >> 5, dealt = 8 * A.splits, place = split * 8 + wave;
  for (int64_t i0 = 0; i0 * dealt + place < steps; i0 += 64) {
    const int64_t s = (i0 + lane) * dealt + place;
    int2 r = make_int2(-1, -1);
    if (s < steps) r = A.range[s];
    uint64_t some = __ballot(r.x <= a && a <= r.y);
    const uint64_t all = __ballot(r.x == a && a == r.y);
    while (some) {
      const int i = __builtin_ctzll(some);
      some &= some - 1;
      one_step(((i0 + i) * dealt + place) * 32, (all >> i) & 1u);
    }
  }
  const Split P{8, 1, wave, 0};
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    // lane l: rank l % 16, columns j of lanes 4 (l / 16) + 0..3
    reduce_split<8, 4>(acc[r], mem.red, P, [&](int, int j, int l, const f32x4 &s) {
#pragma unroll
      for (int k = 0; k < 4; ++k) mem.out[l & 15][((l >> 4) * 4 + k) * 8 + j] = s[k];
    });
    __syncthreads();
    for (int i = threadIdx.x; i < 2048; i += 512) {
      const int col = O.by_rank ? i & 127 : i >> 4, j = O.by_rank ? i >> 7 : i & 15, rank = (rt0 + r) * 16 + j;
      const int64_t c = outer_col(O, blk, col >> 3) + (col & 7);
      if (rank >= A.rank || c >= O.k) continue;
      const int64_t at = O.by_rank ? (static_cast<int64_t>(a) * A.rank + rank) * O.k + c
                                   : (static_cast<int64_t>(a) * O.k + c) * A.rank + rank;
      if (A.splits > 1)
        A.partial[split * A.all + A.before[which] + at] = mem.out[j][col];
      else
        store1(O.out, A.dtype, at, mem.out[j][col]);
    }
    __syncthreads();
  }
}

// KIND of x; dy is of its tensors' type (BF16).
template <int RT, int KIND, bool BF16>
__global__ void __launch_bounds__(512, 2) back_outer_kernel(OuterArgs A) {
  __shared__ OuterMemory s_mem;
  if (blockIdx.x < A.of[0].blocks)
    outer_sums<RT, BF16 ? FROM_BF16 : FROM_F32>(A, A.of[0], 0, blockIdx.x, s_mem);
  else
    outer_sums<RT, KIND>(A, A.of[1], 1, blockIdx.x - A.of[0].blocks, s_mem);
}

template <int KIND, bool BF16> void launch_outer(const OuterArgs &O, dim3 wgs, hipStream_t stream) {
  if (O.rank <= 16)
    hipLaunchKernelGGL((back_outer_kernel<1, KIND, BF16>), wgs, dim3(512), 0, stream, O);
  else
    hipLaunchKernelGGL((back_outer_kernel<2, KIND, BF16>), wgs, dim3(512), 0, stream, O);
}

// The splits' sums (16 at most), in their order.
__global__ void __launch_bounds__(256) back_join_kernel(OuterArgs A) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= A.all) return;
  float w[16], s = 0.0f;
#pragma unroll
  for (int k = 0; k < 16; ++k) w[k] = A.partial[min(k, A.splits - 1) * A.all + i];
#pragma unroll
  for (int k = 0; k < 16; ++k)
    if (k < A.splits) s += w[k];
  const int which = i >= A.before[1] ? 1 : 0;
  store1(A.of[which].out, A.dtype, i - A.before[which], s);
}

// ---------------------------------------------------------------------------
struct BackPlan {
  int64_t ntile, chunks, tpad, rowpad;
  RowsPlan dx;
  int rpad, tiles, osplits;
  int64_t grads;  // values of both adapters' gradients
  size_t bo, go, geo, po, bto, pto, ato, vto, ppo, vpo, ido, rgo, pao, wo, oo, bytes;
};
// Splits of the tokens for the adapters' gradients: as long as workgroups are fewer than CUs and each wave keeps a step.
int outer_splits(int64_t rows, int64_t cols, int64_t T, int n, int rank) {
  const int64_t wgs = ((rows + 127) / 128 + cols / 128) * n * ((rank + 31) / 32);
  int s = 1;
  while (s < 16 && wgs * s < 256 && s * 256 < T) s *= 2;
  return s;
}
BackPlan plan_back(int fmt, int64_t rows, int64_t cols, int dtype, int64_t T, int n, int rank) {
  BackPlan p{};
  const size_t size = dtype == IQ_DTYPE_F32 ? 4 : 2;
  p.ntile = (T + 15) / 16;
  p.chunks = row_chunks(rows);
  p.dx = plan_rows(T, cols / 256, p.chunks, dtype, dtype == IQ_DTYPE_F32);
  p.bo = ws_up(static_cast<size_t>(kCodebook[fmt]) * 16);
  p.go = p.bo + ws_up(kBoundBytes);
  p.geo = p.go + ws_up(grads_bytes(p.chunks, p.ntile, dtype == IQ_DTYPE_F32));
  p.po = p.geo + ws_up(static_cast<size_t>(p.ntile) * 64);
  p.bto = p.po + ws_up(p.dx.bytes);
  p.bytes = p.bto + kWsAlign;
  if (!rank) return p;
  p.tpad = (T + 31) / 32 * 32;
  p.rowpad = (rows + 255) / 256 * 256;
  p.rpad = (rank + 31) / 32 * 32;
  p.tiles = (rank + 15) / 16;
  p.ato = p.bto + ws_up(static_cast<size_t>(n) * p.tiles * 16 * p.rowpad * size);
  p.pto = p.ato + ws_up(static_cast<size_t>(n) * p.tiles * 16 * cols * size);
  const size_t whole = dtype == IQ_DTYPE_F32 ? ws_up(static_cast<size_t>(p.rpad) * p.tpad * 4) : 0;
  const size_t parts = ws_up(static_cast<size_t>(p.rpad) * p.tpad * 6);
  p.vto = p.pto + whole;
  p.ppo = p.vto + whole;
  p.vpo = p.ppo + parts;
  p.ido = p.vpo + parts;
  p.rgo = p.ido + ws_up(static_cast<size_t>(p.tpad) * 4);
  p.pao = p.rgo + ws_up(static_cast<size_t>(p.tpad) / 4);
  p.wo = p.pao + (dtype == IQ_DTYPE_BF16 ? parts : 0);
  p.oo = p.wo + ws_up(static_cast<size_t>(n) * p.tiles * (cols / 256) * 4);
  p.grads = static_cast<int64_t>(n) * rank * (rows + cols);
  p.osplits = outer_splits(rows, cols, T, n, rank);
  p.bytes = p.oo + (p.osplits > 1 ? ws_up(static_cast<size_t>(p.osplits) * p.grads * 4) : 0) + kWsAlign;
  return p;
}

int check_back(int fmt, int64_t rows, int64_t cols, int dtype, int64_t T, int n, int rank) {
  if (run_bad_fmt(fmt)) return IQ_ERR_FMT;
  if (run_bad_dtype(dtype)) return IQ_ERR_DTYPE;
  if (rows < 0 || T < 0 || cols <= 0 || cols % 256 != 0) return IQ_ERR_SHAPE;
  if (rows > (int64_t(1) << 24) || cols > (int64_t(1) << 24) || T > (int64_t(1) << 24)) return IQ_ERR_SHAPE;
  if (rank < 0 || rank > 1024 || (rank && n < 1)) return IQ_ERR_ARG;
  const int64_t ntile = (T + 15) / 16;
  if (ntile > 4 * 65535 || (rank && n > 65535)) return IQ_ERR_SHAPE;  // the adapters' gradients' grid
  if (T * (cols / 256) >= (int64_t(1) << 26)) return IQ_ERR_SHAPE;    // the tiles of dx
  if (rank && (ntile + 1) * 2 * ((rank + 31) / 32) >= kMaxWG) return IQ_ERR_SHAPE;
  if (rank && (T + 7) / 8 + n * static_cast<int64_t>((rank + 15) / 16) * ((rows + 255) / 256 + cols / 256) + 128 >= kMaxWG)
    return IQ_ERR_SHAPE;
  return IQ_OK;
}

}  // namespace
}  // namespace iq

extern "C" {

int iq_linear_backward_workspace_size(int fmt, int64_t rows, int64_t cols, int dtype, int64_t T, int num_adapters,
                                      int rank, size_t *bytes) {
  const int rc = iq::check_back(fmt, rows, cols, dtype, T, num_adapters, rank);
  if (rc != IQ_OK) return rc;
  if (!bytes) return IQ_ERR_NULL;
  *bytes = rows && T ? iq::plan_back(fmt, rows, cols, dtype, T, num_adapters, rank).bytes : 0;
  return IQ_OK;
}

int iq_linear_backward(int fmt, const uint8_t *packed, int64_t rows, int64_t cols, const float *grid,
                       const void *dy, const void *x, const uint8_t *exponents, int dtype, int64_t T,
                       const void *lora_a, const void *lora_b, const float *lora_scale, const int32_t *lora_ids,
                       int num_adapters, int rank, void *dx, void *da, void *db, void *workspace,
                       size_t workspace_bytes, int32_t *status, hipStream_t stream) {
  using namespace iq;
  int rc = check_back(fmt, rows, cols, dtype, T, num_adapters, rank);
  if (rc != IQ_OK) return rc;
  const bool empty = rows == 0 || T == 0;
  const size_t size = dtype == IQ_DTYPE_F32 ? 4 : 2;
  if (!grid || (rank && (!da || (rows && !db)))) return IQ_ERR_NULL;
  if (!empty && (!packed || !dy || (rank && (!x || !lora_a || !lora_b || !lora_ids)))) return IQ_ERR_NULL;
  if (empty) {
    if (dx && (rc = launch_zero(dx, static_cast<size_t>(T) * cols * size, stream)) != IQ_OK) return rc;
    if (!rank) return IQ_OK;
    if ((rc = launch_zero(da, static_cast<size_t>(num_adapters) * rank * cols * size, stream)) != IQ_OK) return rc;
    return launch_zero(db, static_cast<size_t>(num_adapters) * rank * rows * size, stream);
  }
  if (reinterpret_cast<uintptr_t>(packed) & 1) return IQ_ERR_ARG;
  if (!dx && !rank) return IQ_OK;
  const BackPlan P = plan_back(fmt, rows, cols, dtype, T, num_adapters, rank);
  if ((rc = run_check_ws(P.bytes, workspace, workspace_bytes)) != IQ_OK) return rc;
  char *base = ws_base(workspace);
  _Float16 *tab = reinterpret_cast<_Float16 *>(base);
  const Adapters L{lora_a, lora_b, lora_scale, lora_ids, rank ? num_adapters : 0, rank};
  float *pt = dtype == IQ_DTYPE_F32 ? reinterpret_cast<float *>(base + P.pto) : nullptr;
  float *vt = dtype == IQ_DTYPE_F32 ? reinterpret_cast<float *>(base + P.vto) : nullptr;
  uint16_t *pp = reinterpret_cast<uint16_t *>(base + P.ppo), *vp = reinterpret_cast<uint16_t *>(base + P.vpo);
  int32_t *ids = reinterpret_cast<int32_t *>(base + P.ido);
  int2 *range = reinterpret_cast<int2 *>(base + P.rgo);
  BackPrepArgs A{};
  A.dy = dy;
  A.dtype = dtype;
  A.fmt = fmt;
  A.bytes = block_bytes(fmt);
  A.T = T;
  A.rows = rows;
  A.nb = cols / 256;
  A.nconv = (T + 7) / 8;
  A.packed = packed;
  A.G = Grads{base + P.go, reinterpret_cast<uint32_t *>(base + P.geo), P.ntile};
  A.books = one_codebook(fmt, grid, tab, status);
  A.B = Bound{reinterpret_cast<uint32_t *>(base + P.bo), reinterpret_cast<uint32_t *>(base + P.bo) + kScaleSlots,
              A.books.wg[0], fmt >= IQ1_S};
  A.convert = dx != nullptr;
  A.L = L;
  A.ao = base + P.ato;
  A.bo = base + P.bto;
  A.wild = reinterpret_cast<uint32_t *>(base + P.wo);
  A.tiles = P.tiles;
  A.cols = cols;
  A.rowpad = P.rowpad;
  const int64_t wgs = (dx ? kScaleSlots + A.nconv + A.books.wg[0] : 0) +
                      static_cast<int64_t>(L.n) * P.tiles * ((P.rowpad + cols) / 256);
  if (dtype == IQ_DTYPE_F32)
    hipLaunchKernelGGL(back_prep_kernel<2>, dim3(static_cast<unsigned>(wgs)), dim3(512), 0, stream, A);
  else
    hipLaunchKernelGGL(back_prep_kernel<1>, dim3(static_cast<unsigned>(wgs)), dim3(512), 0, stream, A);
  if (!run_launched()) return IQ_ERR_HIP;
  if (rank) {
    ShrinkArgs S{};
    S.of[0] = Shrink{Source{dy, nullptr, dtype}, rows, A.bo, P.rowpad, pt, pp};
    S.of[1] = Shrink{Source{x, exponents, dtype}, cols, A.ao, cols, vt, vp};
    S.dtype = dtype;
    S.T = T;
    S.tpad = P.tpad;
    S.L = L;
    S.rgroups = (rank + 31) / 32;
    // Slots as long as workgroups are 1,024 at most, as many as are at work at once.  With 512, 1,024, 2,048 and 4,096, us:
    // 4,096 tokens, four adapters of rank 32, together 68, 63, 63, 66, in random order 145, 130, 130, 148; 2,048 tokens,
    // one adapter of rank 16 16, 16, 17, 26, eight in random order 60, 61, 56, 67.
    S.slots = 32;
    while (S.slots > 1 && (P.tpad >> 5) * 2 * S.rgroups * S.slots > 1024) S.slots /= 2;
    S.ids = ids;
    S.range = range;
    S.parts = reinterpret_cast<uint16_t *>(base + P.pao);
    S.status = status;
    const dim3 shrinks(static_cast<unsigned>((P.tpad >> 5) * 2 * S.rgroups * S.slots));
    if (dtype == IQ_DTYPE_F32)  // of either kind
      hipLaunchKernelGGL((back_shrink_kernel<FROM_F32, false>), shrinks, dim3(512), 0, stream, S);
    else if (exponents)
      hipLaunchKernelGGL((back_shrink_kernel<FROM_CHECKPOINT, true>), shrinks, dim3(512), 0, stream, S);
    else
      hipLaunchKernelGGL((back_shrink_kernel<FROM_BF16, true>), shrinks, dim3(512), 0, stream, S);
    if (!run_launched()) return IQ_ERR_HIP;
  }
  if (dx) {
    RowsArgs D{};
    D.packed[0] = D.packed[1] = packed;
    D.nmat = 1;
    D.rows = rows;
    D.nb = cols / 256;
    D.T = T;
    D.tab = tab;
    D.G = A.G;
    D.B = A.B;
    D.out = dx;
    D.partial = reinterpret_cast<float *>(base + P.po);
    D.plan = P.dx;
    D.a = lora_a;
    D.p = pt;
    D.parts = reinterpret_cast<const uint16_t *>(base + P.pao);
    D.wild = reinterpret_cast<const uint32_t *>(base + P.wo);
    D.ids = ids;
    D.rank = rank;
    D.tpad = P.tpad;
    if ((rc = launch_rows(fmt, dtype, D, stream)) != IQ_OK) return rc;
  }
  if (rank) {
    OuterArgs O{};
    O.of[0] = Outer{Source{dy, nullptr, dtype}, rows, (rows + 127) / 128, vt, vp, db, 0};
    O.of[1] = Outer{Source{x, exponents, dtype}, cols, cols / 128, pt, pp, da, 1};
    O.T = T;
    O.tpad = P.tpad;
    O.dtype = dtype;
    O.rank = rank;
    O.rgroups = (rank + 31) / 32;
    O.ids = ids;
    O.range = range;
    O.splits = P.osplits;
    O.partial = reinterpret_cast<float *>(base + P.oo);
    O.before[1] = static_cast<int64_t>(num_adapters) * rank * rows;
    O.all = P.grads;
    const unsigned across = static_cast<unsigned>(O.of[0].blocks + O.of[1].blocks), z = P.osplits;
    const dim3 wgo(across, num_adapters, rank <= 16 ? z : (rank + 31) / 32 * z);
    if (dtype == IQ_DTYPE_F32)
      exponents ? launch_outer<FROM_CHECKPOINT, false>(O, wgo, stream) : launch_outer<FROM_F32, false>(O, wgo, stream);
    else
      exponents ? launch_outer<FROM_CHECKPOINT, true>(O, wgo, stream) : launch_outer<FROM_BF16, true>(O, wgo, stream);
    if (!run_launched()) return IQ_ERR_HIP;
    if (z > 1) {
      hipLaunchKernelGGL(back_join_kernel, dim3(static_cast<unsigned>((P.grads + 255) / 256)), dim3(256), 0, stream, O);
      if (!run_launched()) return IQ_ERR_HIP;
    }
  }
  return IQ_OK;
}

}  // extern "C"
