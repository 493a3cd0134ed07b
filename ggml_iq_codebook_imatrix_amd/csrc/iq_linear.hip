// iq_linear.hip -- iq_linear: tokens through an encoded projection, with the
// low-rank adapters of many requests beside it (include/iq_run.h).
//
// Two launches.  linear_prep_kernel brings the tokens into fp16 operand order,
// converts the codebook, and forms the adapters' rank-wide products v = s A x.
// The second kernel decodes the payload straight into matrix operands, and adds
// B v to its sums before it stores them.

#include "iq_run.hpp"

namespace iq {
namespace {

struct Lora {
  const void *a, *b;
  const float *scale;
  const int32_t *ids;
  int n, rank, chunks;  // chunks of 32 ranks (bf16) or 16 (float32)
  // v in operand order, [tile of 16 tokens][chunk]: bf16 the three bf16 values
  // that add up to it, [3][lane][8]; float32 [lane][4]
  void *v;
};
constexpr int kChunkBytes[2] = {3 * 1024, 1024};  // bf16, float32

struct PrepArgs {
  const void *x;
  int dtype;
  int64_t T, cols, nconv;  // nconv: workgroups that convert (eight tokens each)
  Tokens X;
  Codebooks books;
  Lora L;
  int rtiles;  // tiles of 16 ranks
  int slots;   // workgroups of a token tile and rank tile, for its up to 16 adapters
  int32_t *status;
};

// The adapter of lane l < 16's token in tile tt (-1: none, or no such token).
__device__ __forceinline__ int tile_adapter(const Lora &L, int64_t tt, int64_t T, int lane) {
  const int64_t t = tt * 16 + lane;
  if (lane >= 16 || t >= T) return -1;
  const int a = L.ids[t];
  return a >= 0 && a < L.n ? a : -1;
}

// v for the tokens of tile tt that share the adapter of token `slot`, 16 ranks:
// 16 tokens (A) by the adapter's 16 rows (B), K split over the eight waves; the
// rows of tokens with other adapters are dropped.
__device__ __forceinline__ void lora_shrink(const PrepArgs &P, int64_t tt, int rt, int slot, f32x4 *s_red) {
  const Lora &L = P.L;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, q = lane >> 4;
  const int mine = tile_adapter(L, tt, P.T, lane);
  if (threadIdx.x < 16 && slot == 0 && rt == 0) {
    const int64_t t = tt * 16 + lane;
    if (t < P.T && mine < 0 && L.ids[t] != -1) raise_status(P.status, ST_BADID);
  }
  const int a = __builtin_amdgcn_readlane(mine, slot);
  const uint32_t group = static_cast<uint32_t>(__ballot(mine == a)) & 0xffffu;
  if (a < 0 || (group & ((1u << slot) - 1u))) return;  // an earlier token's workgroup does it
  // rows of other tokens read this one's: fewer lines
  const int64_t t = tt * 16 + (((group >> n) & 1u) ? n : slot);
  const int j = min(rt * 16 + n, L.rank - 1);
  const int64_t xr = t * P.cols + q * 8, ar = (static_cast<int64_t>(a) * L.rank + j) * P.cols + q * 8;
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  const int nb = static_cast<int>(P.cols >> 8), k0 = wave * 32;  // 32 of each 256 columns; U loads in flight
  if (P.dtype == 1) {
    constexpr int U = 8;
    const uint16_t *xp = static_cast<const uint16_t *>(P.x) + xr + k0, *ap = static_cast<const uint16_t *>(L.a) + ar + k0;
    for (int b = 0; b < nb; b += U) {
      bf16x8 xa[U], ab[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = min(b + u, nb - 1) * 256;
        xa[u] = ldu<bf16x8>(xp + at);
        ab[u] = ldu<bf16x8>(ap + at);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (b + u < nb) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xa[u], ab[u], acc, 0, 0, 0);
    }
  } else {
    constexpr int U = 4;
    for (int b = 0; b < nb; b += U) {
      float xa[U][8], ab[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = min(b + u, nb - 1) * 256 + k0;
        load8u(P.x, 0, xr + at, xa[u]);
        load8u(L.a, 0, ar + at, ab[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (b + u < nb)
#pragma unroll
          for (int i = 0; i < 8; ++i) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(xa[u][i], ab[u][i], acc, 0, 0, 0);
    }
  }
  const float scale = L.scale ? L.scale[a] : 1.0f;
  const Split S{8, 1, wave, 0};
  reduce_split<1, 1>(&acc, s_red, S, [&](int, int, int l, const f32x4 &s) {
    const int jj = rt * 16 + (l & 15);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = (l >> 4) * 4 + i;
      if (!((group >> tok) & 1u)) continue;
      float f = jj < L.rank ? s[i] * scale : 0.0f;
      if (P.dtype == 1) {
        uint16_t *v = static_cast<uint16_t *>(L.v) + (tt * L.chunks + (jj >> 5)) * 1536 +
                      (((jj & 31) >> 3) * 16 + tok) * 8 + (jj & 7);
        const bool pad = rt + 1 == P.rtiles && !(rt & 1);  // the upper half of the last 32 ranks is nobody's
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const uint32_t top = __float_as_uint(f) & 0xffff0000u;
          v[k * 512] = static_cast<uint16_t>(top >> 16);
          if (pad) v[k * 512 + 256] = 0;
          f = finite_f(f) ? f - __uint_as_float(top) : 0.0f;  // inf - inf would be NaN
        }
      } else {
        static_cast<float *>(L.v)[(tt * L.chunks + rt) * 256 + (((jj & 15) >> 2) * 16 + tok) * 4 + (jj & 3)] = f;
      }
    }
  });
}

// 4,096 tokens of 5,120: 21 us without adapters (84 MB in and out, 4.0 TB/s: the
// conversion is bound by memory, and its 16-byte pieces), 36 with eight adapters of
// rank 16; 64 tokens of 2,048 with one 3 to 5 us, its loads' latency.
template <int P>
__global__ void __launch_bounds__(512) linear_prep_kernel(PrepArgs A) {
  __shared__ f32x4 s_red[8 * 64];
  int64_t w = blockIdx.x;
  // The shrink first, it takes longest.  Slots last: where one adapter serves a
  // whole tile, only slot 0 has work, and consecutive workgroups go to different
  // XCDs (16 apart all went to one: 8x slower).
  const int64_t tiles = A.X.ntile * A.rtiles;
  if (w < tiles * A.slots) {
    const int first = static_cast<int>(w / tiles);
    w -= first * tiles;
    for (int slot = first; slot < 16; slot += A.slots)
      lora_shrink(A, w / A.rtiles, static_cast<int>(w % A.rtiles), slot, s_red);
    return;
  }
  w -= tiles * A.slots;
  if (w < A.nconv) {
    const int64_t t = w * 8 + (threadIdx.x >> 6);
    if (t < A.T) convert_token<P>(A.x, A.cols, A.X, t, threadIdx.x & 63);
    return;
  }
  w -= A.nconv;
  convert_codebook(A.books, static_cast<int>(w));
}

// acc[r][c] += B v of the adapters that the tiles' tokens name.  Of tile c, wave
// w of nw takes the adapters whose turn t (in order of first use) has
// (t + c) % nw == w; a round takes one adapter of each of the C tiles, and the
// next one's rows of B are fetched before this one multiplies.  32 ranks (bf16) or
// 16 at a time, whose v, of all the tile's tokens, serves every adapter: what rows
// of other tokens give is dropped.  fp32 v is the sum of three bf16 values beside a
// bf16 B (no rounding), and goes through the fp32 cores beside an fp32 B.
template <int P, int C, int R> struct LoraStep {
  bf16x8 w[C][R];     // bf16
  f32x4 wf[C][R];     // float32
  uint32_t group[C];  // tokens of the tile
};

template <int P, int C, int R>
__device__ __forceinline__ void lora_fetch(const Lora &L, int64_t rows, int64_t row0, int ch, const int (&a)[C],
                                           LoraStep<P, C, R> &s) {
  const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (!s.group[c]) continue;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = min(row0 + r * 16 + n, rows - 1), at = (static_cast<int64_t>(a[c]) * rows + row) * L.rank;
      if (P == 1) {
        const int j = ch * 32 + q * 8;
        const uint16_t *b = static_cast<const uint16_t *>(L.b) + at;
        if ((L.rank & 7) == 0) {  // whole eights; past the rank v is zero, and the last eight will do
          s.w[c][r] = ldu<bf16x8>(b + min(j, L.rank - 8));
        } else {
          s.w[c][r] = bf16x8{};
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (j + i < L.rank) s.w[c][r][i] = __builtin_bit_cast(__bf16, b[j + i]);
        }
      } else {
        const int j = ch * 16 + q * 4;
        const float *b = static_cast<const float *>(L.b) + at;
        s.wf[c][r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (j + i < L.rank) s.wf[c][r][i] = b[j + i];
      }
    }
  }
}

template <int P, int C, int R>
__device__ __forceinline__ void lora_expand(const Lora &L, int64_t tt0, int64_t T, int64_t rows, int64_t row0,
                                            int wave, int nw, f32x4 (&acc)[R][C]) {
  const int lane = threadIdx.x & 63, q = lane >> 4;
  int mine[C], turn[C], a[C];
  uint32_t todo[C];
#pragma unroll
  for (int c = 0; c < C; ++c) mine[c] = tile_adapter(L, tt0 + c, T, lane);
  // the wave's next adapter of each tile; 0: none is left
  const auto next_round = [&](uint32_t (&group)[C]) __attribute__((always_inline)) {
    uint32_t any = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      group[c] = 0;
      while (todo[c] && !group[c]) {
        a[c] = __builtin_amdgcn_readlane(mine[c], __builtin_ctz(todo[c]));
        const uint32_t g = static_cast<uint32_t>(__ballot(mine[c] == a[c])) & 0xffffu;
        todo[c] &= ~g;
        if (turn[c]++ % nw == wave) group[c] = g;
      }
      any |= group[c];
    }
    return any;
  };
  for (int ch = 0; ch < L.chunks; ++ch) {
    LoraStep<P, C, R> now, then;
    bf16x8 v[C][3];
    f32x4 vf[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      todo[c] = static_cast<uint32_t>(__ballot(mine[c] >= 0)) & 0xffffu;
      turn[c] = c;
      if (!todo[c]) continue;
      const char *from = static_cast<const char *>(L.v) + ((tt0 + c) * L.chunks + ch) * kChunkBytes[P - 1] + lane * 16;
      if (P == 1) {
#pragma unroll
        for (int k = 0; k < 3; ++k) v[c][k] = *reinterpret_cast<const bf16x8 *>(from + k * 1024);
      } else {
        vf[c] = *reinterpret_cast<const f32x4 *>(from);
      }
    }
    uint32_t more = next_round(now.group);
    if (!more) return;
    lora_fetch<P, C, R>(L, rows, row0, ch, a, now);
    while (more) {
      more = next_round(then.group);
      if (more) lora_fetch<P, C, R>(L, rows, row0, ch, a, then);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (!now.group[c]) continue;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
          if (P == 1) {
#pragma unroll
            for (int k = 0; k < 3; ++k) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[c][k], now.w[c][r], d, 0, 0, 0);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x4f32(vf[c][i], now.wf[c][r][i], d, 0, 0, 0);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if ((now.group[c] >> (q * 4 + k)) & 1u) acc[r][c][k] += d[k];
        }
      }
      now = then;
    }
  }
}

struct LinearArgs {
  const uint8_t *packed;
  int64_t rows, nb, T;
  const _Float16 *tab;
  Tokens X;
  Lora L;
  void *y;
};

// Few tokens, or few tiles: the waves split K (split_blocks), RT row tiles each by
// C token tiles.  Latency bounds it: a wave has one or two blocks, whose payload
// and tokens it waits for once, and then the sums' way through LDS.  5,632 x 2,048,
// IQ2_XS: one token 6.5 us (3.3 MB of payload, 0.5 TB/s), 16 tokens with 16 adapters
// 8.5 us.
template <int F, int P, int C, int RT>
__global__ void __launch_bounds__(512) linear_split_kernel(LinearArgs A) {
  constexpr int G = RT * C < 4 ? RT * C : 4;
  constexpr int kTab = Geo<F>::N, kRed = 8 * G * 64;
  __shared__ uint4 s_mem[kTab > kRed ? kTab : kRed];
  load_table<F>(s_mem, A.tab);
  const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  const Split S = split_of(A.nb);
  const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * S.rw + S.rg) * 16 * RT;
  const int64_t tt0 = static_cast<int64_t>(blockIdx.y) * C;
  const int64_t rowbytes = A.nb * Geo<F>::BYTES, stride = A.X.ntile * P * 4096;
  const _Float16 *x0[C];
  int64_t e0[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int64_t t = min((tt0 + c) * 16 + n, A.T - 1);
    x0[c] = A.X.x16 + (t >> 4) * P * 4096 + (q * 16 + (t & 15)) * 8;
    e0[c] = min((tt0 + c) * 16 + q * 4, A.X.ntile * 16 - 4);
  }
  f32x4 acc[RT][1][C] = {};
  __syncthreads();
  split_blocks<F, P, C, RT, 1>(
      A.nb, S, s_mem, [&](int, int rt) { return A.packed + min(row0 + rt * 16 + n, A.rows - 1) * rowbytes; },
      [&](int64_t b, Operand<P, C> &x) __attribute__((always_inline)) {
        const _Float16 *xp[C];
#pragma unroll
        for (int c = 0; c < C; ++c) xp[c] = x0[c] + b * stride;
        load_operand<P, C>(x, xp);
      },
        acc);
  f32x4 sum[RT][C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int4 e = *reinterpret_cast<const int4 *>(A.X.ex + e0[c]);
#pragma unroll
    for (int r = 0; r < RT; ++r)
      sum[r][c] = f32x4{ldexpf(acc[r][0][c][0], e.x), ldexpf(acc[r][0][c][1], e.y), ldexpf(acc[r][0][c][2], e.z),
                        ldexpf(acc[r][0][c][3], e.w)};
  }
  if (A.L.rank) lora_expand<P, C, RT>(A.L, tt0, A.T, A.rows, row0, S.kg, S.kw, sum);
  reduce_split<RT * C, G>(&sum[0][0], reinterpret_cast<f32x4 *>(s_mem), S, [&](int rg, int tile, int l, const f32x4 &s) {
    const int64_t row = ((static_cast<int64_t>(blockIdx.x) * S.rw + rg) * RT + tile / C) * 16 + (l & 15);
    if (row >= A.rows) return;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t t = (tt0 + tile % C) * 16 + (l >> 4) * 4 + k;
      if (t < A.T) store1(A.y, P == 1, t * A.rows + row, s[k]);
    }
  });
}

// More tokens: the waves are KG groups that take every KG-th block and RG groups
// that take 16 R rows each; the C token tiles of a chunk of KG blocks lie in LDS for
// all of them (64 KiB), the next chunk's on their way in registers.  64 tokens
// through 17,408 x 5,120, IQ1_M, 48 adapters of rank 32: 46 us (0.25 PFLOP/s),
// about 34 without the adapters.  Its decode alone would take a third of that; the
// waves (three a SIMD) wait at each chunk for its tokens and for one another.  One row tile a wave
// (R = 1) in six groups fills 182 CUs, two in four groups 136 CUs (58 us).
template <int F, int P, int C, int R, int KG, int RG>
__global__ void __launch_bounds__(64 * KG * RG, KG * RG / 4) linear_tile_kernel(LinearArgs A) {
  constexpr int NT = 64 * KG * RG, kX = KG * C * P * 512, XU = (kX + NT - 1) / NT, G = 4, kTab = Geo<F>::N;
  __shared__ uint4 s_tab[kTab];
  __shared__ u32x4 s_x[kX];
  static_assert(KG == 1 || kX >= KG * RG * G * 64, "the sums over the waves fit");
  load_table<F>(s_tab, A.tab);
  const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), kg = wave / RG;
  const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * RG + wave % RG) * 16 * R;
  const int64_t tt0 = static_cast<int64_t>(blockIdx.y) * C, rowbytes = A.nb * Geo<F>::BYTES;
  const uint8_t *rp[R];
#pragma unroll
  for (int r = 0; r < R; ++r) rp[r] = A.packed + min(row0 + r * 16 + n, A.rows - 1) * rowbytes;
  u32x4 xr[XU];
  // chunk ch of the token operand: XU units of 16 bytes a thread, [block][tile][part] of 512
  const auto load_x = [&](int64_t ch) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < XU; ++i) {
      const int u = i * NT + static_cast<int>(threadIdx.x), piece = u >> 9;
      if (kX % NT && u >= kX) break;
      const int64_t b = min(ch * KG + piece / (C * P), A.nb - 1);
      const int64_t tile = min(tt0 + piece / P % C, A.X.ntile - 1);
      xr[i] = reinterpret_cast<const u32x4 *>(A.X.x16)[((b * A.X.ntile + tile) * P + piece % P) * 512 + (u & 511)];
    }
  };
  const auto store_x = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < XU; ++i) {
      const int u = i * NT + static_cast<int>(threadIdx.x);
      if (kX % NT && u >= kX) break;
      s_x[u] = xr[i];
    }
  };
  f32x4 acc[R][C];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < C; ++c) acc[r][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t chunks = (A.nb + KG - 1) / KG;
  Words words[R], next[R];
#pragma unroll
  for (int r = 0; r < R; ++r) words[r] = load_words<F>(rp[r] + min(static_cast<int64_t>(kg), A.nb - 1) * Geo<F>::BYTES, q);
  load_x(0);
  store_x();
  __syncthreads();
  for (int64_t ch = 0; ch < chunks; ++ch) {
    if (ch + 1 < chunks) {
#pragma unroll
      for (int r = 0; r < R; ++r)
        next[r] = load_words<F>(rp[r] + min((ch + 1) * KG + kg, A.nb - 1) * Geo<F>::BYTES, q);
      load_x(ch + 1);
    }
    __builtin_amdgcn_sched_barrier(0);  // the loads above go out before the work below, not after it
    if (ch * KG + kg < A.nb) {
      Raw raw[R];
#pragma unroll
      for (int r = 0; r < R; ++r) raw[r] = unpack<F>(words[r], q);
      const _Float16 *xp[C];
#pragma unroll
      for (int c = 0; c < C; ++c) xp[c] = reinterpret_cast<const _Float16 *>(s_x + (kg * C + c) * P * 512 + lane);
      f32x4 part[R][C];
      block_mma<F, P, C, R>(raw, s_tab, xp, part);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < C; ++c) scale_add(acc[r][c], part[r][c], block_scale<F>(raw[r]));
    }
    if (ch + 1 < chunks) {
      __syncthreads();  // the chunk is read
      store_x();
#pragma unroll
      for (int r = 0; r < R; ++r) words[r] = next[r];
      __syncthreads();
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int4 e = *reinterpret_cast<const int4 *>(A.X.ex + min((tt0 + c) * 16 + q * 4, A.X.ntile * 16 - 4));
#pragma unroll
    for (int r = 0; r < R; ++r)
      acc[r][c] = f32x4{ldexpf(acc[r][c][0], e.x), ldexpf(acc[r][c][1], e.y), ldexpf(acc[r][c][2], e.z),
                        ldexpf(acc[r][c][3], e.w)};
  }
  if (A.L.rank) lora_expand<P, C, R>(A.L, tt0, A.T, A.rows, row0, kg, KG, acc);
  const auto put = [&](int64_t r0, int tile, int l, const f32x4 &s) {
    const int64_t row = r0 + (tile / C) * 16 + (l & 15);
    if (row >= A.rows) return;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t t = (tt0 + tile % C) * 16 + (l >> 4) * 4 + k;
      if (t < A.T) store1(A.y, P == 1, t * A.rows + row, s[k]);
    }
  };
  if constexpr (KG == 1) {
#pragma unroll
    for (int i = 0; i < R * C; ++i) put(row0, i, lane, acc[i / C][i % C]);
  } else {  // the KG groups' sums, in their order
    f32x4 *red = reinterpret_cast<f32x4 *>(s_x);
#pragma unroll
    for (int g = 0; g < R * C; g += G) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < G; ++j) red[(wave * G + j) * 64 + lane] = acc[(g + j) / C][(g + j) % C];
      __syncthreads();
      for (int i = threadIdx.x; i < RG * G * 64; i += NT) {
        const int rg = i / (G * 64), rest = i % (G * 64);
        f32x4 s = red[rg * G * 64 + rest];
#pragma unroll
        for (int k = 1; k < KG; ++k) s += red[(k * RG + rg) * G * 64 + rest];
        put((static_cast<int64_t>(blockIdx.x) * RG + rg) * 16 * R, g + rest / 64, rest & 63, s);
      }
    }
  }
}

// Prompts (bf16): eight waves of 16 R rows each by C token tiles.  Registers decide
// the tile, so there are no sums apart from the accumulators: these are kept in
// units of the block's d, and rescaled by the ratio of two blocks' d in between (one
// more rounding of 2^-24 a block, bf16 outputs round by 2^-9).  A block of d = 0
// counts with zero weights instead.  Token operands go from memory to LDS
// directly, half a block ahead.
// 4,096 tokens through 17,408 x 5,120, IQ1_S: 0.74 ms, 0.98 PFLOP/s; the matrix cores
// are busy 44 % of it, LDS 36 %.  What bounds it is the issue of the decode's vector
// instructions (25 a step and row tile, at 5 to 8 cycles with two waves a SIMD)
// beside 2 C matrix instructions of 16 cycles.  R = 4, C = 6 spilled registers (0.77
// at 4,096 columns, against 0.62 with R = 2, C = 10); a third buffer, so that no half
// waits for its tokens, made it 9 % slower, and four waves a SIMD would be bound by
// their LDS reads.
template <int F, int C, int R>
__global__ void __launch_bounds__(512, 2) linear_prompt_kernel(LinearArgs A) {
  constexpr int kHalf = C * 256;  // 16-byte units of half a block: C tiles of 4 KiB
  __shared__ uint4 s_tab[Geo<F>::N];
  __shared__ u32x4 s_x[2][kHalf];
  load_table<F>(s_tab, A.tab);
  const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * 8 + wave) * 16 * R;
  const int64_t tt0 = static_cast<int64_t>(blockIdx.y) * C, rowbytes = A.nb * Geo<F>::BYTES;
  const uint8_t *rp[R];
#pragma unroll
  for (int r = 0; r < R; ++r) rp[r] = A.packed + min(row0 + r * 16 + n, A.rows - 1) * rowbytes;
  // half h of the token operand into buffer h % 2: piece i (1 KiB) by wave i % 8,
  // tile i / 4, its steps' lanes in order
  const auto fetch = [&](int64_t h) __attribute__((always_inline)) {
#pragma unroll
    for (int i0 = 0; i0 < C * 4; i0 += 8) {
      const int i = i0 + wave;
      if (i < C * 4) {
        const int64_t tile = min(tt0 + i / 4, A.X.ntile - 1);
        const u32x4 *from = reinterpret_cast<const u32x4 *>(A.X.x16) + ((h >> 1) * A.X.ntile + tile) * 512 +
                            (h & 1) * 256 + (i & 3) * 64 + lane;
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from,
                                         (__attribute__((address_space(3))) void *)&s_x[h & 1][i * 64], 16, 0, 0);
      }
    }
  };
  f32x4 acc[R][C];
  float unit[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    unit[r] = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[r][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  Words words[R];
#pragma unroll
  for (int r = 0; r < R; ++r) words[r] = load_words<F>(rp[r], q);
  fetch(0);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the barrier does not wait for loads into LDS
  __syncthreads();
  for (int64_t b = 0; b < A.nb; ++b) {
    uint32_t keep[R];
    Raw raw[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      raw[r] = unpack<F>(words[r], q);
      const float d = block_scale<F>(raw[r]);
      keep[r] = d != 0.0f ? ~0u : 0u;
      const float ratio = keep[r] ? unit[r] / d : 1.0f;
      unit[r] = keep[r] ? d : unit[r];
#pragma unroll
      for (int c = 0; c < C; ++c) acc[r][c] *= ratio;
    }
    half8v w[2][R];  // the step in hand and the next, decoded while this one multiplies
#pragma unroll
    for (int r = 0; r < R; ++r) w[0][r] = group_half8<F>(raw[r], 0, s_tab, keep[r]);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int64_t h = 2 * b + half;
      if (h + 1 < 2 * A.nb) fetch(h + 1);
      if (half == 0) {
        const int64_t bn = min(b + 1, A.nb - 1);
#pragma unroll
        for (int r = 0; r < R; ++r) words[r] = load_words<F>(rp[r] + bn * Geo<F>::BYTES, q);
      }
      __builtin_amdgcn_sched_barrier(0);  // the loads above go out before the work below, not after it
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int g = half * 4 + i;
        half8v x[C];
#pragma unroll
        for (int c = 0; c < C; ++c) x[c] = __builtin_bit_cast(half8v, s_x[half][c * 256 + i * 64 + lane]);
        if (g < 7) {
#pragma unroll
          for (int r = 0; r < R; ++r) w[(g + 1) & 1][r] = group_half8<F>(raw[r], g + 1, s_tab, keep[r]);
        }
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int r = 0; r < R; ++r)
            acc[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[c], w[g & 1][r], acc[r][c], 0, 0, 0);
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();  // the next half is there, this one free
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int4 e = *reinterpret_cast<const int4 *>(A.X.ex + min((tt0 + c) * 16 + q * 4, A.X.ntile * 16 - 4));
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const f32x4 s = acc[r][c] * unit[r];
      acc[r][c] = f32x4{ldexpf(s[0], e.x), ldexpf(s[1], e.y), ldexpf(s[2], e.z), ldexpf(s[3], e.w)};
    }
  }
  if (A.L.rank) {
#pragma unroll
    for (int c = 0; c < C; c += 2) {
      f32x4 a[R][2];
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < 2; ++k) a[r][k] = acc[r][c + k];
      lora_expand<1, 2, R>(A.L, tt0 + c, A.T, A.rows, row0, 0, 1, a);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < 2; ++k) acc[r][c + k] = a[r][k];
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t row = row0 + r * 16 + n;
    if (row >= A.rows) continue;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t t = (tt0 + c) * 16 + q * 4 + k;
        if (t < A.T) store1(A.y, 1, t * A.rows + row, acc[r][c][k]);
      }
  }
}

struct LinearPlan {
  TokensPlan x;
  int chunks;
  size_t tab, xo, eo, vo, bytes;
};
LinearPlan plan_linear(int fmt, int64_t cols, int dtype, int64_t T, int rank) {
  LinearPlan p;
  p.x = plan_tokens(T, cols, dtype);
  p.chunks = dtype == IQ_DTYPE_F32 ? (rank + 15) / 16 : (rank + 31) / 32;
  p.tab = 0;
  p.xo = ws_up(static_cast<size_t>(kCodebook[fmt]) * 16);
  p.eo = p.xo + ws_up(p.x.xbytes);
  p.vo = p.eo + ws_up(p.x.ebytes);
  p.bytes = p.vo + ws_up(static_cast<size_t>(p.x.ntile) * p.chunks * kChunkBytes[dtype == IQ_DTYPE_F32]) + kWsAlign;
  return p;
}

int check_linear(int fmt, int64_t rows, int64_t cols, int dtype, int64_t T, int rank) {
  if (run_bad_fmt(fmt)) return IQ_ERR_FMT;
  if (run_bad_dtype(dtype)) return IQ_ERR_DTYPE;
  if (rows < 0 || T < 0 || cols <= 0 || cols % 256 != 0) return IQ_ERR_SHAPE;
  // rows: 512 threads take at least 32 where there are many
  if (rows > (int64_t(1) << 27) || cols > (int64_t(1) << 24) || T > (int64_t(1) << 24)) return IQ_ERR_SHAPE;
  if (rank < 0 || rank > 1024) return IQ_ERR_ARG;
  const int64_t ntile = (T + 15) / 16;
  // the preparing launch: conversion, codebook, adapters
  if ((T + 7) / 8 + 8 + 1024 + ntile * ((rank + 15) / 16) >= kMaxWG) return IQ_ERR_SHAPE;
  if (ntile > 4 * 65535) return IQ_ERR_SHAPE;
  return IQ_OK;
}

template <int F, int P, int C, int RT>
void launch_split(const LinearArgs &A, hipStream_t stream) {
  const int64_t rw = split_rw(A.nb), rows = rw * 16 * RT;
  hipLaunchKernelGGL((linear_split_kernel<F, P, C, RT>),
                     dim3(static_cast<unsigned>((A.rows + rows - 1) / rows),
                          static_cast<unsigned>((A.X.ntile + C - 1) / C)),
                     dim3(static_cast<unsigned>(64 * split_kw(A.nb) * rw)), 0, stream, A);
}

template <int F, int P, int C, int R, int KG, int RG>
void launch_tile(const LinearArgs &A, hipStream_t stream) {
  constexpr int rows = RG * 16 * R;
  hipLaunchKernelGGL((linear_tile_kernel<F, P, C, R, KG, RG>),
                     dim3(static_cast<unsigned>((A.rows + rows - 1) / rows),
                          static_cast<unsigned>((A.X.ntile + C - 1) / C)),
                     dim3(64 * KG * RG), 0, stream, A);
}

template <int F, int C, int R> void launch_prompt(const LinearArgs &A, hipStream_t stream) {
  constexpr int rows = 8 * 16 * R;
  hipLaunchKernelGGL((linear_prompt_kernel<F, C, R>),
                     dim3(static_cast<unsigned>((A.rows + rows - 1) / rows),
                          static_cast<unsigned>((A.X.ntile + C - 1) / C)),
                     dim3(512), 0, stream, A);
}

// What a kernel takes of a large launch: rows and token tiles of a workgroup, one
// workgroup a CU, and the cost of the first round over 256 CUs and of each further
// one (us at 4,096 columns).
struct TileCost {
  int rows, C, first, more;
};
inline int64_t tile_cost(const TileCost &k, int64_t rows, int64_t ntile) {
  const int64_t wgs = (rows + k.rows - 1) / k.rows * ((ntile + k.C - 1) / k.C);
  return k.first + ((wgs + 255) / 256 - 1) * k.more;
}

template <int F, int P> void launch_linear(const LinearArgs &A, hipStream_t stream) {
  const int64_t ntile = A.X.ntile, rtiles = (A.rows + 15) / 16, pairs = rtiles * ntile;
  if (ntile == 1) {
    // Four row tiles a wave share its tokens and its workgroup's beginning and end
    // (2,048 columns, 1 token: 8,192 rows 9.1 us with one and 10.6 with four, 12,288
    // 11.3 and 10.7, 40,960 24.3 and 17.7).
    if (rtiles / split_rw(A.nb) <= 640)
      launch_split<F, P, 1, 1>(A, stream);
    else
      launch_split<F, P, 1, 4>(A, stream);
    return;
  }
  // Measured at 4,096 columns, bf16 (float32): 512 tile pairs 16.5 us with one row
  // tile a wave and 18.4 with two (26.1, 27.7), 1,024 pairs 22.5 and 21.5 (34.0,
  // 28.1).  2,048 pairs take 31 us with two and 38 in tiles (4,096: 59 and 70); two
  // token tiles would leave half of a tile empty.
  if (pairs <= 512) return launch_split<F, P, 2, 1>(A, stream);
  if (ntile == 2 || pairs <= 2048 * P) return launch_split<F, P, 2, 2>(A, stream);
  const TileCost costs[2][6] = {
      {{64, 4, 37, 21}, {128, 4, 47, 31}, {96, 4, 40, 28}, {128, 8, 56, 46}, {256, 8, 80, 74}, {256, 10, 92, 90}},
      {{128, 4, 70, 47}, {256, 4, 90, 76}}};
  int best = 0;
  for (int i = 1; i < (P == 1 ? 6 : 2); ++i)
    if (tile_cost(costs[P - 1][i], A.rows, ntile) < tile_cost(costs[P - 1][best], A.rows, ntile)) best = i;
  if (best == 0) return launch_tile<F, P, 4, 1, 2 / P, 4 * P>(A, stream);
  if (best == 1) return launch_tile<F, P, 4, 2, 2 / P, 4 * P>(A, stream);
  if constexpr (P == 1) {
    if (best == 2) return launch_tile<F, P, 4, 1, 2, 6>(A, stream);
    if (best == 3) return launch_prompt<F, 8, 1>(A, stream);
    if (best == 4) return launch_prompt<F, 8, 2>(A, stream);
    launch_prompt<F, 10, 2>(A, stream);
  }
}

}  // namespace
}  // namespace iq

extern "C" {

int iq_linear_workspace_size(int fmt, int64_t rows, int64_t cols, int dtype, int64_t T, int rank, size_t *bytes) {
  const int rc = iq::check_linear(fmt, rows, cols, dtype, T, rank);
  if (rc != IQ_OK) return rc;
  if (!bytes) return IQ_ERR_NULL;
  *bytes = rows && T ? iq::plan_linear(fmt, cols, dtype, T, rank).bytes : 0;
  return IQ_OK;
}

int iq_linear(int fmt, const uint8_t *packed, int64_t rows, int64_t cols, const float *grid, const void *x,
              int dtype, int64_t T, const void *lora_a, const void *lora_b, const float *lora_scale,
              const int32_t *lora_ids, int num_adapters, int rank, void *y, void *workspace,
              size_t workspace_bytes, int32_t *status, hipStream_t stream) {
  using namespace iq;
  int rc = check_linear(fmt, rows, cols, dtype, T, rank);
  if (rc != IQ_OK) return rc;
  const bool empty = rows == 0 || T == 0;
  if (!grid || (!empty && (!packed || !x || !y || (rank && (!lora_a || !lora_b || !lora_ids))))) return IQ_ERR_NULL;
  if (rank && num_adapters < 1) return IQ_ERR_ARG;
  if (empty) return IQ_OK;
  if (reinterpret_cast<uintptr_t>(packed) & 1) return IQ_ERR_ARG;
  const LinearPlan P = plan_linear(fmt, cols, dtype, T, rank);
  if ((rc = run_check_ws(P.bytes, workspace, workspace_bytes)) != IQ_OK) return rc;
  char *base = ws_base(workspace);
  _Float16 *tab = reinterpret_cast<_Float16 *>(base + P.tab);
  const Tokens X{reinterpret_cast<_Float16 *>(base + P.xo), reinterpret_cast<int32_t *>(base + P.eo), P.x.ntile};
  const Lora L{lora_a, lora_b, lora_scale, lora_ids, num_adapters, rank, P.chunks, base + P.vo};
  PrepArgs A{};
  A.x = x;
  A.dtype = dtype;
  A.T = T;
  A.cols = cols;
  A.nconv = (T + 7) / 8;
  A.X = X;
  A.books = one_codebook(fmt, grid, tab, status);
  A.L = L;
  A.rtiles = (rank + 15) / 16;
  A.slots = 16;  // as many as are at work at once; more only wait (4,096 sorted tokens: 42 us, so 35)
  while (A.slots > 1 && P.x.ntile * A.rtiles * A.slots > 512) A.slots /= 2;
  A.status = status;
  const dim3 wgs(static_cast<unsigned>(A.nconv + A.books.wg[0] + P.x.ntile * A.rtiles * A.slots));
  if (dtype == IQ_DTYPE_F32)
    hipLaunchKernelGGL(linear_prep_kernel<2>, wgs, dim3(512), 0, stream, A);
  else
    hipLaunchKernelGGL(linear_prep_kernel<1>, wgs, dim3(512), 0, stream, A);
  if (!run_launched()) return IQ_ERR_HIP;
  const LinearArgs M{packed, rows, cols / 256, T, tab, X, L, y};
#define CALL(F) dtype == IQ_DTYPE_F32 ? launch_linear<F, 2>(M, stream) : launch_linear<F, 1>(M, stream)
  IQ_BY_FMT(fmt, CALL)
#undef CALL
  return run_launched() ? IQ_OK : IQ_ERR_HIP;
}

}  // extern "C"
