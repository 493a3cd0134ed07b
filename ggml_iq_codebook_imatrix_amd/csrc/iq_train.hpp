// iq_train.hpp -- what the calls of include/iq_train.h share: checkpoints as
// tokens, the bound on a payload's weights, gradients in operand order, and the
// product of gradients with encoded weights over the weights' rows.
#pragma once

#include "iq_run.hpp"
#include "iq_train.h"

namespace iq {

// Gradients for products over rows: g [chunk of 64 rows][tile of 16 tokens][step of 32 rows][lane][8], rows in their
// order, lane 16 q + n with token n and rows 8 q on.  bf16 gradients of a caller are fp16 under a power of two a token
// (grad_power; exact, in steps of 2^-39 of a token's largest), others fp32 as they are, whose lanes' first four rows come
// before all lanes' other four: a lane's loads of 16 bytes are 1 KiB in a row for the wave.  most [tokens]: the fp32 bits
// of the largest finite magnitude.  Rows past the last of a weight are zeros, tokens past the last are left unwritten.
struct Grads {
  void *g;
  uint32_t *most;
  int64_t ntile;
};
// The power of two that brings a token's gradients under 2^15 (wide: as a factor, which has to be a number).
__host__ __device__ inline int grad_power(uint32_t most, bool wide) {
  const int n = 141 - (static_cast<int>(most >> 23) > 1 ? static_cast<int>(most >> 23) : 1);
  return wide && n > 126 ? 126 : n;
}
__host__ __device__ inline int64_t row_chunks(int64_t rows) { return (rows + 63) / 64; }
inline size_t grads_bytes(int64_t chunks, int64_t ntile, bool wide) {
  return static_cast<size_t>(chunks) * ntile * (wide ? 4096 : 2048);
}

// What bounds a payload's weights, found by a preparing launch: the largest finite
// block scale (fp16 bits) of each of kScaleSlots workgroups' shares, and the largest
// finite magnitude (fp32 bits) of each 512 codebook entries.
constexpr int kScaleSlots = 64, kGridSlots = 4;
struct Bound {
  uint32_t *scale, *grid;
  int ngrid;
  int iq1;
};
constexpr size_t kBoundBytes = (kScaleSlots + kGridSlots) * 4;

// Tokens to bring into operand order: as they are, or a checkpoint.
struct Source {
  const void *x;
  const uint8_t *ex;  // a checkpoint's exponents; null: x is of `dtype`
  int dtype;
};

// Tokens of the forward product: of a checkpoint, one part serves (its values have
// seven bits).
inline int source_parts(const Source &s) { return s.ex || s.dtype == IQ_DTYPE_BF16 ? 1 : 2; }

// dx of gradients G with one or two encoded weights of the same size (see iq_rows.hip).  The workgroups' tiles of dx:
// the first `full` whole, of the others the rows split, whose sums a second launch adds.
struct RowsPlan {
  int tiles;  // of 16 tokens, in a workgroup's tile, which is a block of columns wide
  int64_t full, rest;
  int splits;
  size_t bytes;  // at least those of the rest's partial sums; never less for more tokens
};
RowsPlan plan_rows(int64_t T, int64_t nb, int64_t chunks, int dtype, bool wide);
struct RowsArgs {
  const uint8_t *packed[2];
  int nmat;
  int64_t rows, nb, T;
  const _Float16 *tab;
  Grads G;
  Bound B;
  void *out;
  float *partial;  // [tile of the rest][split][16 tiles or all tokens, if fewer][256 columns]
  RowsPlan plan;
  // adapters (rank 0: none): A, p of the tokens (f32: [rank][tpad]; bf16: three values that add up to it, [tile of 16
  // tokens][32 ranks][3][lane][8]), their adapters (-1: none),
  // and where A is not finite [adapter][tile of 16 ranks][256 columns]
  const void *a;
  const float *p;
  const uint16_t *parts;
  const uint32_t *wild;
  const int32_t *ids;
  int rank;
  int64_t tpad;
};
inline int block_bytes(int fmt) {
  constexpr int bytes[5] = {Geo<IQ2_XXS>::BYTES, Geo<IQ2_XS>::BYTES, Geo<IQ2_S>::BYTES, Geo<IQ1_S>::BYTES,
                            Geo<IQ1_M>::BYTES};
  return bytes[fmt];
}
int launch_zero(void *p, size_t bytes, hipStream_t stream);  // bytes: a multiple of two
int launch_rows(int fmt, int dtype, const RowsArgs &A, hipStream_t stream);

#ifdef __HIPCC__

__device__ __forceinline__ float load1(const void *x, int dtype, int64_t i) {
  return dtype == 1 ? bf16_to_f32(static_cast<const uint16_t *>(x)[i]) : static_cast<const float *>(x)[i];
}

// Eight consecutive values to any address.
__device__ __forceinline__ void store8u(void *y, int dtype, int64_t i, const float v[8]) {
  if (dtype == 1) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = f32_to_bf16(v[2 * j]) | (static_cast<uint32_t>(f32_to_bf16(v[2 * j + 1])) << 16);
    const uint4 o = make_uint4(w[0], w[1], w[2], w[3]);
    __builtin_memcpy(static_cast<uint16_t *>(y) + i, &o, 16);
  } else {
    __builtin_memcpy(static_cast<float *>(y) + i, v, 32);
  }
}

// The larger of `most` and a value's magnitude, as fp32 bits; infinities and NaN are passed over.
__device__ __forceinline__ uint32_t max_bits(uint32_t most, float v) {
  const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
  return b < 0x7f800000u ? max(most, b) : most;
}

// Eight rows of one token's gradients (fp32), chunk0 chunks into G; row a multiple of eight.
__device__ __forceinline__ void put_grads(const Grads &G, int64_t chunk0, int64_t t, int64_t row, const float (&v)[8]) {
  const int in = static_cast<int>(row & 63);
  float *to = static_cast<float *>(G.g) + ((chunk0 + (row >> 6)) * G.ntile + (t >> 4)) * 1024 + (in >> 5) * 512 +
              (((in & 31) >> 3) * 16 + (t & 15)) * 4;
  *reinterpret_cast<f32x4 *>(to) = f32x4{v[0], v[1], v[2], v[3]};
  *reinterpret_cast<f32x4 *>(to + 256) = f32x4{v[4], v[5], v[6], v[7]};
}

// Eight codes of one block times 2^n; -128 to NaN.  A code plus 128 is a byte, which converts in one instruction.
__device__ __forceinline__ void decode_codes(uint2 w, int n, float v[8]) {
  const uint32_t u[2] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u};
  const float unit = ldexpf(1.0f, n);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = (static_cast<float>((u[j >> 2] >> (8 * (j & 3))) & 255u) - 128.0f) * unit;
  const auto zero_byte = [](uint32_t x) { return (x - 0x01010101u) & ~x & 0x80808080u; };
  if (zero_byte(u[0]) | zero_byte(u[1])) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (!((u[j >> 2] >> (8 * (j & 3))) & 255u)) v[j] = __uint_as_float(0x7fc00000u);
  }
}

// As convert_token, of a checkpoint: the largest block exponent takes the place of
// the largest magnitude's, so that codes become at most 127 * 2^8.
__device__ __forceinline__ void convert_checkpoint(const int8_t *codes, const uint8_t *ex, int64_t cols,
                                                   const Tokens &X, int64_t t, int lane) {
  const int64_t blocks = cols >> 5;
  const uint8_t *er = ex + t * blocks;
  uint32_t most = 1;
  for (int64_t b = lane; b < blocks; b += 64) most = max(most, static_cast<uint32_t>(er[b]));
  const int n = 141 - static_cast<int>(wave_max_u32(most));
  constexpr int U = 4;
  for (int64_t k = 0; k < cols; k += 512 * U) {
    uint2 w[U];
    int e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t col = min(k + u * 512 + lane * 8, cols - 8);
      w[u] = ldu<uint2>(codes + t * cols + col);
      e[u] = er[col >> 5];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t col = k + u * 512 + lane * 8;
      if (col >= cols) break;
      const int g = static_cast<int>(col & 255) >> 3;
      float v[8];
      decode_codes(w[u], e[u] - 133 + n, v);
      half8v hi;
#pragma unroll
      for (int h = 0; h < 8; ++h) hi[h] = static_cast<_Float16>(v[kept_at(h)]);
      *reinterpret_cast<half8v *>(X.x16 + ((col >> 8) * X.ntile + (t >> 4)) * 4096 +
                                  ((g & 7) * 64 + (g >> 3) * 16 + (t & 15)) * 8) = hi;
    }
  }
  if (lane == 0) X.ex[t] = -n;
}

// The largest exponent field of a row's finite magnitudes (at least 1), by one wave.
__device__ __forceinline__ uint32_t row_exponent(const void *x, int dtype, int64_t n, int64_t t, int lane) {
  uint32_t e = 1;
  const int64_t base = t * n, whole = n & ~int64_t(7);
  for (int64_t k = lane * 8; k < whole; k += 512) {
    float v[8];
    load8u(x, dtype, base + k, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) e = max_exponent(e, v[j]);
  }
  if (whole + lane < n) e = max_exponent(e, load1(x, dtype, base + whole + lane));
  return wave_max_u32(e);
}

// Where an array in LDS begins, for the two loads below.
#define IQ_LDS_ADDRESS(array) \
  static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char *)(array)))
// 64 lanes' 16 bytes each, from base + off on, to 1 KiB of LDS at `to` (base and `to` the same in all lanes).  The
// compiler takes every later read of LDS for one of these bytes and waits for them, which is a memory's latency lost in
// each round of a buffer; written out, they are waited for where the buffers change (wait_loads), and by nothing before.
// m0 leaves as an output, so that the compiler takes none it has set for one that is still there.
__device__ __forceinline__ void load_to_lds(const char *base, uint32_t off, uint32_t to) {
  uint32_t m0;
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               : "={m0}"(m0)
               : "v"(off), "s"(base), "s"(to)
               : "memory");
}
// The same of 4 bytes each, to 256 bytes of LDS.
__device__ __forceinline__ void load_words_to_lds(const char *base, uint32_t off, uint32_t to) {
  uint32_t m0;
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
               : "={m0}"(m0)
               : "v"(off), "s"(base), "s"(to)
               : "memory");
}
// All loads but the wave's last N (in the order of their issue).
template <int N> __device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }

// A wave's maximum into LDS, the workgroup's into *out (NW waves).
template <int NW> __device__ __forceinline__ void workgroup_max(uint32_t v, uint32_t *red, uint32_t *out) {
  const uint32_t m = wave_max_u32(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    uint32_t r = red[0];
    for (int w = 1; w < NW; ++w) r = max(r, red[w]);
    *out = r;
  }
}

// Workgroup s of kScaleSlots (512 threads): the largest finite block scale of its
// share of `blocks` blocks of `count` payloads.
__device__ __forceinline__ void bound_scales(int fmt, int bytes, const uint8_t *const (&packed)[2], int count,
                                             int64_t blocks, const Bound &B, int s, uint32_t *red) {
  uint32_t most = 0;
  for (int m = 0; m < count; ++m)
    for (int64_t b = s * 512 + static_cast<int>(threadIdx.x); b < blocks; b += kScaleSlots * 512) {
      const uint8_t *blk = packed[m] + b * bytes;
      uint32_t d;
      if (fmt == IQ1_M) {
        const uint2 w = ldu<uint2>(blk + 48);
        d = ((w.x >> 12) & 15u) | ((w.x >> 28) << 4) | (((w.y >> 12) & 15u) << 8) | ((w.y >> 28) << 12);
      } else {
        d = *reinterpret_cast<const uint16_t *>(blk);
      }
      d &= 0x7fffu;
      if (d < 0x7c00u) most = max(most, d);
    }
  workgroup_max<8>(most, red, B.scale + s);
}

// With the workgroup that converts 512 codebook entries.
__device__ __forceinline__ void bound_codebook(const Codebooks &C, const Bound &B, int wg, uint32_t *red) {
  uint32_t most = 0;
  const int i = wg * 512 + static_cast<int>(threadIdx.x);
  if (i < C.n[0]) {
    float g[8];
    load8u(C.grid[0], 0, static_cast<int64_t>(i) * 8, g);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (finite_f(g[j])) most = max(most, __float_as_uint(g[j]) & 0x7fffffffu);
  }
  workgroup_max<8>(most, red, B.grid + wg);
}

// An e with |d| < 2^e for every finite block scale (with IQ2's 2^-3) of the payloads.
__device__ __forceinline__ int scale_exponent(const Bound &B) {
  const uint32_t d = wave_max_u32(B.scale[threadIdx.x & 63]);
  const float f = f16_bits_to_f32(static_cast<uint16_t>(d)) * (B.iq1 ? 1.0f : 0.125f);
  return f > 0.0f ? static_cast<int>(__float_as_uint(f) >> 23) - 126 : 0;
}

// The power of two to take off m v so that the largest a codebook can form stays under 2^15: 0 for all that fp16 holds
// with a bit to spare, which the layouts' own are far below.
__device__ __forceinline__ int codebook_shift(const Bound &B) {
  const int lane = threadIdx.x & 63;
  const float g = __uint_as_float(wave_max_u32(lane < B.ngrid ? B.grid[lane] : 0u));
  const float most = B.iq1 ? 15.0f * (g + 0.125f) : 31.0f * g;
  return min(max(static_cast<int>(__float_as_uint(most) >> 23) - 126 - 15, 0), 10);
}

// The fields of group g, from a block in LDS, `half` bytes (0 or 2) behind an address that is a multiple of four.
struct Fields {
  uint32_t k, ls, mask, h, d16;
};
template <int F> __device__ __forceinline__ Fields read_fields(const uint8_t *blk, int g, uint32_t half) {
  const auto u16 = [&](int at) -> uint32_t { return *reinterpret_cast<const uint16_t *>(blk + at); };
  Fields f;
  f.mask = f.h = 0;
  if (F == IQ1_M) {
    // the scale and the shifts as words: with narrow reads, five more, the product of two weights of 17,408 x 5,120 and
    // 4,096 tokens took 2,680 us instead of 2,620 (the other layouts' fields as words changed nothing)
    const uint32_t *w = reinterpret_cast<const uint32_t *>(blk - half + 48);
    const uint32_t w0 = __builtin_amdgcn_alignbyte(w[1], w[0], half), w1 = __builtin_amdgcn_alignbyte(w[2], w[1], half);
    f.d16 = ((w0 >> 12) & 15u) | ((w0 >> 28) << 4) | (((w1 >> 12) & 15u) << 8) | ((w1 >> 28) << 12);
    const uint32_t nib = (blk[32 + (g >> 1)] >> (4 * (g & 1))) & 15u;
    f.k = blk[g] | ((nib & 7u) << 8);
    f.h = nib >> 3;
    f.ls = ((g & 16 ? w1 : w0) >> (16 * ((g >> 3) & 1) + 3 * ((g >> 1) & 3))) & 7u;
    return f;
  }
  f.d16 = u16(0);
  if (F == IQ2_XXS) {
    const int at = 2 + 8 * (g >> 2);
    f.k = blk[at + (g & 3)];
    const uint32_t word = u16(at + 4) | (u16(at + 6) << 16);
    f.mask = (word >> (7 * (g & 3))) & 127u;
    f.ls = word >> 28;
  } else if (F == IQ2_XS) {
    const uint32_t v = u16(2 + 2 * g);
    f.k = v & 511u;
    f.mask = v >> 9;
    f.ls = (blk[66 + (g >> 2)] >> (4 * ((g >> 1) & 1))) & 15u;
  } else if (F == IQ2_S) {
    f.k = blk[2 + g] | (((blk[66 + (g >> 2)] >> (2 * (g & 3))) & 3u) << 8);
    f.mask = blk[34 + g];
    f.ls = (blk[74 + (g >> 2)] >> (4 * ((g >> 1) & 1))) & 15u;
  } else {
    const uint32_t w = u16(34 + 2 * (g >> 2));
    f.k = blk[2 + g] | (((w >> (3 * (g & 3))) & 7u) << 8);
    f.ls = (w >> 12) & 7u;
    f.h = w >> 15;
  }
  return f;
}

// m v of a group, e its codebook entry, times `shrink` (a power of two): w[p] holds values p (low half) and p + 4.
template <int F>
__device__ __forceinline__ void row_weights(const Fields &f, const uint4 &e, half2v shrink, uint32_t (&w)[4]) {
  const uint32_t o[4] = {e.x, e.y, e.z, e.w}, sum = f.ls * 0x20002u + 0x64016401u;  // as in multiplier2
  const half2v m2 = __builtin_elementwise_fma(__builtin_bit_cast(half2v, sum), shrink, shrink * static_cast<_Float16>(-1024.0f));
  if (Geo<F>::IQ1) {
    const half2v up = m2 * static_cast<_Float16>(0.125f);
    const half2v c2 = __builtin_bit_cast(half2v, __builtin_bit_cast(uint32_t, up) ^ (f.h * 0x80008000u));
#pragma unroll
    for (int p = 0; p < 4; ++p)
      w[p] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(half2v, o[p]), m2, c2));
  } else {
    uint32_t t = sign_places<F>(f.mask);
#pragma unroll
    for (int p = 3; p >= 0; --p) {
      const half2v v = __builtin_bit_cast(half2v, o[p]) * m2;
      w[p] = __builtin_bit_cast(uint32_t, v) ^ (t & 0x80008000u);
      asm("v_add_u32 %0, %0, %0" : "+v"(t));
    }
  }
}

#endif  // __HIPCC__

}  // namespace iq
