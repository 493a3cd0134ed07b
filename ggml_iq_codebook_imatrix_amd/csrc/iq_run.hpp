// iq_run.hpp -- what iq_linear (iq_linear.hip) and iq_moe (iq_moe.hip) share:
// payload fields to fp16 matrix operands, tokens in operand order, and the
// products of one 256-column block.  Declared in include/iq_run.h.
//
// A weight is d * m * v: d the block's fp16 scale, m the group's odd multiplier,
// v its signed codebook value.  The products run on the fp16 matrix cores:
// m * v is formed in packed fp16 (exact for the layouts' codebooks: at most 11
// bits), d is applied in fp32 to each 256-column block's sum, and the token's
// power-of-two scale to the whole sum.
//
// Operand layout (v_mfma_f32_16x16x32_f16): the weights are B, lane l holding
// eight consecutive k of row n = l % 16; the tokens are A, lane l holding the
// same k of token m = l % 16; D has lane l hold row n = l % 16 and tokens
// 4 (l / 16) + 0..3, so a block's d, known to the lane that decodes row n,
// scales that lane's own sums.  The order of k is free as long as both operands
// use it: lane quarter q = l / 16 takes the block's 64 columns from 64 q on,
// eight at a step, so that a lane's share of the payload is contiguous (two or
// three wide loads a block) and a step's eight values are one codebook entry.
// Within the eight, value j and value j + 4 share a register (kept_at): the signs
// of the four pairs are then one bit apart, and bringing them to the sign places
// is an addition (x + x), which issues at twice the rate of a shift.
#pragma once

#include "iq_common.hpp"
#include "iq_internal.hpp"
#include "iq_run.h"

namespace iq {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));  // arrays of it stay in registers, of uint4 they did not

constexpr int ST_ROUNDED = IQ_STATUS_ROUNDED;
constexpr int kCodebook[5] = {256, 512, 1024, 2048, 2048};
// A dimension of a grid holds fewer than 2^32 threads: this many workgroups of 512.
constexpr int64_t kMaxWG = (int64_t(1) << 23) - 1;

inline bool run_launched() { return hipGetLastError() == hipSuccess; }
inline bool run_bad_fmt(int f) { return f < 0 || f > 4; }
inline bool run_bad_dtype(int d) { return d != IQ_DTYPE_F32 && d != IQ_DTYPE_BF16; }
inline int run_check_ws(size_t need, const void *ws, size_t have) {
  if (!ws) return IQ_ERR_NULL;
  return have < need ? IQ_ERR_WORKSPACE : IQ_OK;
}

// Tokens in fp16: x16 [block][tile of 16 tokens][part][step 0..7][lane][8], the
// A operand of a step as 1 KiB of consecutive memory; ex [tokens]: the power of
// two that undoes a token's scaling.  Rows past the last token are left unwritten;
// kernels that take whole tiles read them, and since a row of A gives a row of D, they
// reach only outputs that are not stored.
struct Tokens {
  _Float16 *x16;
  int32_t *ex;
  int64_t ntile;  // tiles of 16 tokens
};
struct TokensPlan {
  int64_t ntile;
  int parts;
  size_t xbytes, ebytes;
};
inline TokensPlan plan_tokens(int64_t T, int64_t cols, int dtype) {
  TokensPlan p;
  p.ntile = (T + 15) / 16;
  p.parts = dtype == IQ_DTYPE_F32 ? 2 : 1;
  p.xbytes = static_cast<size_t>(cols / 256) * p.ntile * p.parts * 8192;
  p.ebytes = static_cast<size_t>(p.ntile) * 64;
  return p;
}

// Codebooks to convert: up to two, 512 entries a workgroup of 512 threads.
struct Codebooks {
  const float *grid[2];
  _Float16 *tab[2];
  int n[2], iq1[2], wg[2];
  int32_t *status;
};
inline Codebooks one_codebook(int fmt, const float *grid, _Float16 *tab, int32_t *status) {
  Codebooks c{};
  c.grid[0] = grid;
  c.tab[0] = tab;
  c.n[0] = kCodebook[fmt];
  c.iq1[0] = fmt >= IQ1_S;
  c.wg[0] = (kCodebook[fmt] + 511) / 512;
  c.status = status;
  return c;
}

#define IQ_BY_FMT(fmt, CALL)            \
  switch (fmt) {                        \
    case IQ2_XXS: CALL(IQ2_XXS); break; \
    case IQ2_XS: CALL(IQ2_XS); break;   \
    case IQ2_S: CALL(IQ2_S); break;     \
    case IQ1_S: CALL(IQ1_S); break;     \
    default: CALL(IQ1_M); break;        \
  }

#ifdef __HIPCC__

template <class V> __device__ __forceinline__ V ldu(const void *p) {  // any alignment
  V v;
  __builtin_memcpy(&v, p, sizeof(V));
  return v;
}

__device__ __forceinline__ void store1(void *y, int dtype, int64_t i, float v) {
  if (dtype == 1)
    static_cast<uint16_t *>(y)[i] = f32_to_bf16(v);
  else
    static_cast<float *>(y)[i] = v;
}

// Eight consecutive values from any address.
__device__ __forceinline__ void load8u(const void *base, int dtype, int64_t idx, float v[8]) {
  if (dtype == 1) {
    const uint4 u = ldu<uint4>(static_cast<const uint16_t *>(base) + idx);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const float4 a = ldu<float4>(static_cast<const float *>(base) + idx);
    const float4 b = ldu<float4>(static_cast<const float *>(base) + idx + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

// ---------------------------------------------------------------------------
// Payload fields
// ---------------------------------------------------------------------------
// One lane's share of a block: the fields of groups 8q .. 8q + 7.
struct Raw {
  uint32_t a[4];
  uint32_t s;
  uint32_t d16;
};

// The words that hold them, as loaded.  Payload addresses are even, and blocks of
// 66, 74, 82 and 50 bytes put every other one across 4-byte words.  Measured on
// one CU, 16 bytes from each of 16 rows four times: 35 cycles at 4-byte aligned
// addresses, 125 at others (2 and 4 bytes 37 at any, 8 bytes 33 and 64).  So
// whole aligned words are loaded, and the fields moved into place by a byte
// permutation when the block's turn comes; d, which lies before the first
// quarter's fields, comes with that quarter's words.
struct Words {
  uint32_t w[9];
  uint32_t sel;  // the permutation: bytes 2.. or 4.. of a pair of words
};

// Payload comes from global memory, which the compiler cannot see of an address that was rounded or chosen: told so, it
// does not make flat loads, which a barrier waits for as for LDS.
template <class V, int ALIGN> __device__ __forceinline__ V ld_global(uintptr_t p) {
  struct __attribute__((packed, aligned(ALIGN))) At {
    V v;
  };
  return reinterpret_cast<const __attribute__((address_space(1))) At *>(p)->v;
}
template <class V> __device__ __forceinline__ V ldw(uintptr_t p) { return ld_global<V, 4>(p); }  // 4-byte aligned
struct Words3 {
  uint32_t x, y, z;
};
__device__ __forceinline__ Words3 ldw3(uintptr_t p) {
  return Words3{ldw<uint32_t>(p), ldw<uint32_t>(p + 4), ldw<uint32_t>(p + 8)};
}

template <int F> __device__ __forceinline__ Words load_words(const uint8_t *blk, int q) {
  Words r;
  const uintptr_t a = reinterpret_cast<uintptr_t>(blk) & ~uintptr_t(3);
  r.sel = (reinterpret_cast<uintptr_t>(blk) & 2) ? 0x07060504u : 0x05040302u;
  if (F == IQ2_XXS || F == IQ2_XS) {
    const u32x4 v = ldw<u32x4>(a + 16 * q);
    r.w[0] = v[0]; r.w[1] = v[1]; r.w[2] = v[2]; r.w[3] = v[3];
    if (F == IQ2_XXS) {
      r.w[4] = ldw<uint32_t>(a + 16 * q + 16);
    } else {  // the last fields and the scales; the fifth word of other quarters is their neighbour's first
      const Words3 t = ldw3(a + 64);
      r.w[4] = t.x; r.w[5] = t.y; r.w[6] = t.z;
    }
  } else if (F == IQ2_S) {
    const Words3 k = ldw3(a + 8 * q), m = ldw3(a + 32 + 8 * q);
    const uintptr_t t = reinterpret_cast<uintptr_t>(blk) + 66 + 2 * q;
    const Words3 e = ldw3(t & ~uintptr_t(3));
    r.w[0] = k.x; r.w[1] = k.y; r.w[2] = k.z;
    r.w[3] = m.x; r.w[4] = m.y; r.w[5] = m.z;
    r.w[6] = e.x; r.w[8] = e.z;
    r.w[7] = (t & 2) ? 0x07060302u : 0x05040100u;
  } else if (F == IQ1_S) {
    const Words3 k = ldw3(a + 8 * q);
    r.w[0] = k.x; r.w[1] = k.y; r.w[2] = k.z;
    r.w[3] = ld_global<uint32_t, 2>(reinterpret_cast<uintptr_t>(blk) + 34 + 4 * q);
  } else {
    const uintptr_t b = reinterpret_cast<uintptr_t>(blk);
    const u32x2 k = ld_global<u32x2, 2>(b + 8 * q), w = ld_global<u32x2, 2>(b + 48);
    r.w[0] = k[0]; r.w[1] = k[1]; r.w[2] = ld_global<uint32_t, 2>(b + 32 + 4 * q);
    r.w[3] = w[0]; r.w[4] = w[1];
  }
  return r;
}

// All lanes of the wave take part (words are passed between the quarters).
template <int F> __device__ __forceinline__ Raw unpack(const Words &v, int q) {
  Raw r;
  const int lane = threadIdx.x & 63;
  r.a[2] = r.a[3] = r.s = 0;
  if (F == IQ1_M) {
    r.a[0] = v.w[0]; r.a[1] = v.w[1]; r.a[2] = v.w[2];
    r.s = ((q & 2) ? v.w[4] : v.w[3]) >> ((q & 1) * 16);  // scale word q
    r.d16 = ((v.w[3] >> 12) & 15u) | ((v.w[3] >> 28) << 4) | (((v.w[4] >> 12) & 15u) << 8) | ((v.w[4] >> 28) << 12);
    return r;
  }
  const auto pair = [&](uint32_t lo, uint32_t hi) { return __builtin_amdgcn_perm(hi, lo, v.sel); };
  // d: the two bytes before the fields, in the first quarter's first word
  const uint32_t first = v.sel == 0x07060504u ? v.w[0] >> 16 : v.w[0] & 0xffffu;
  r.d16 = static_cast<uint32_t>(__shfl(static_cast<int>(first), lane & 15, 64));
  r.a[0] = pair(v.w[0], v.w[1]);
  r.a[1] = pair(v.w[1], v.w[2]);
  if (F == IQ2_XXS || F == IQ2_XS) {
    uint32_t fifth = v.w[4];
    if (F == IQ2_XS) {
      const uint32_t other = static_cast<uint32_t>(__shfl(static_cast<int>(v.w[0]), lane + 16, 64));
      fifth = q == 3 ? v.w[4] : other;
      // the scales' bytes 2q and 2q + 1 lie 2 + 2q bytes into the words, or 4 + 2q
      const uint32_t lo = pair(v.w[4], v.w[5]), hi = pair(v.w[5], v.w[6]);
      r.s = ((q & 2) ? hi : lo) >> ((q & 1) * 16);
    }
    r.a[2] = pair(v.w[2], v.w[3]);
    r.a[3] = pair(v.w[3], fifth);
  } else if (F == IQ2_S) {
    r.a[2] = pair(v.w[3], v.w[4]);
    r.a[3] = pair(v.w[4], v.w[5]);
    r.s = __builtin_amdgcn_perm(v.w[8], v.w[6], v.w[7]);
  } else {
    r.a[2] = v.w[3];
  }
  return r;
}

template <int F> __device__ __forceinline__ float block_scale(const Raw &r) {
  const float d = f16_bits_to_f32(static_cast<uint16_t>(r.d16));
  return Geo<F>::IQ1 ? d : d * 0.125f;  // exact: a power of two
}

// Which of a group's eight values the operands' element h holds.
__device__ constexpr int kept_at(int h) { return (h >> 1) + 4 * (h & 1); }

// The fields of one group: codebook entry, multiplier, signs (IQ2) or shift (IQ1).
struct GroupFields {
  uint32_t k, ls, mask, h;
};
template <int F> __device__ __forceinline__ GroupFields group_fields(const Raw &r, int i) {
  GroupFields g{};
  if (F == IQ2_XXS) {
    const uint32_t word = r.a[2 * (i >> 2) + 1];
    g.k = (r.a[2 * (i >> 2)] >> (8 * (i & 3))) & 255u;
    g.mask = (word >> (7 * (i & 3))) & 127u;
    g.ls = word >> 28;
  } else if (F == IQ2_XS) {
    const uint32_t v = r.a[i >> 1] >> (16 * (i & 1));
    g.k = v & 511u;
    g.mask = (v >> 9) & 127u;
    g.ls = (r.s >> (4 * (i >> 1))) & 15u;
  } else if (F == IQ2_S) {
    g.k = ((r.a[i >> 2] >> (8 * (i & 3))) & 255u) | (((r.s >> (2 * i)) & 3u) << 8);
    g.mask = (r.a[2 + (i >> 2)] >> (8 * (i & 3))) & 255u;
    g.ls = (r.s >> (16 + 4 * (i >> 1))) & 15u;
  } else if (F == IQ1_S) {
    const uint32_t w = r.a[2] >> (16 * (i >> 2));
    g.k = ((r.a[i >> 2] >> (8 * (i & 3))) & 255u) | (((w >> (3 * (i & 3))) & 7u) << 8);
    g.ls = (w >> 12) & 7u;
    g.h = (w >> 15) & 1u;
  } else {
    const uint32_t nib = r.a[2] >> (4 * i);
    g.k = ((r.a[i >> 2] >> (8 * (i & 3))) & 255u) | ((nib & 7u) << 8);
    g.h = (nib >> 3) & 1u;
    g.ls = (r.s >> (3 * (i >> 1))) & 7u;
  }
  return g;
}

// 2 ls + 1 twice in fp16: added to 1,024 in its last bits, and 1,024 taken off (exact).
__device__ __forceinline__ half2v multiplier2(uint32_t ls) {
  const uint32_t sum = ls * 0x20002u + 0x64016401u;
  return __builtin_bit_cast(half2v, sum) - half2v{static_cast<_Float16>(1024.0f), static_cast<_Float16>(1024.0f)};
}

// The signs of IQ2's eight values where doubling brings pair after pair: those of
// values 3 and 7 in bits 15 and 31, those of p and p + 4 after 3 - p doublings.  The
// eighth sign is the parity of the seven (IQ2_S holds it).
template <int F> __device__ __forceinline__ uint32_t sign_places(uint32_t mask) {
  uint32_t twice = mask << 1;
  if (Geo<F>::PARITY) twice |= __builtin_popcount(twice) << 8;
  return twice * 0x800800u;  // the signs in bits 12.. and 24..; a product of 24 bits, one of 32 has a quarter of the rate
}

// m * v of a group as eight fp16 values (e: its codebook entry in fp16); zeros
// where keep is 0 instead of all ones.
template <int F>
__device__ __forceinline__ half8v weights_half8(const GroupFields &g, const uint4 &e, uint32_t keep) {
  const half2v m2 = __builtin_bit_cast(half2v, __builtin_bit_cast(uint32_t, multiplier2(g.ls)) & keep);
  uint32_t o[4] = {e.x, e.y, e.z, e.w};
  if (Geo<F>::IQ1) {
    const half2v up = m2 * static_cast<_Float16>(0.125f);
    const half2v c2 = __builtin_bit_cast(half2v, __builtin_bit_cast(uint32_t, up) ^ (g.h * 0x80008000u));
#pragma unroll
    for (int p = 0; p < 4; ++p)  // m g + m delta, rounded once
      o[p] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(half2v, o[p]), m2, c2));
  } else {
    uint32_t t = sign_places<F>(g.mask);
#pragma unroll
    for (int p = 3; p >= 0; --p) {
      const half2v v = __builtin_bit_cast(half2v, o[p]) * m2;
      o[p] = __builtin_bit_cast(uint32_t, v) ^ (t & 0x80008000u);
      asm("v_add_u32 %0, %0, %0" : "+v"(t));  // t + t in C becomes a shift, at half the rate
    }
  }
  return __builtin_bit_cast(half8v, make_uint4(o[0], o[1], o[2], o[3]));
}

// The same of group 8q + i (tab: the codebook).
template <int F>
__device__ __forceinline__ half8v group_half8(const Raw &r, int i, const uint4 *tab, uint32_t keep = ~0u) {
  const GroupFields g = group_fields<F>(r, i);
  return weights_half8<F>(g, tab[g.k], keep);
}

template <int F> __device__ __forceinline__ void load_table(uint4 *s_tab, const _Float16 *tab) {
  for (int i = threadIdx.x; i < Geo<F>::N; i += blockDim.x) s_tab[i] = reinterpret_cast<const uint4 *>(tab)[i];
}

// part[r][c] = one block of R row tiles by C token tiles; xp[c]: the lane's
// share of the block's token operand (P parts: fp32 tokens are the sum of two).
template <int F, int P, int C, int R>
__device__ __forceinline__ void block_mma(const Raw (&raw)[R], const uint4 *tab, const _Float16 *const (&xp)[C],
                                          f32x4 (&part)[R][C]) {
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < C; ++c) part[r][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    half8v x[C][P];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int p = 0; p < P; ++p) x[c][p] = *reinterpret_cast<const half8v *>(xp[c] + p * 4096 + i * 512);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const half8v w = group_half8<F>(raw[r], i, tab);
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int p = 0; p < P; ++p)
          part[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[c][p], w, part[r][c], 0, 0, 0);
    }
  }
}

// acc += d * part
__device__ __forceinline__ void scale_add(f32x4 &acc, const f32x4 &part, float d) {
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] = fmaf(d, part[k], acc[k]);
}

template <int CTRL> __device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(static_cast<int>(v), static_cast<int>(v), CTRL, 0xf,
                                                                  0xf, false)));
}
// maximum over the wave, the same in every lane: prefixes within rows of 16, then across the rows
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = dpp_max<0x111>(v);
  v = dpp_max<0x112>(v);
  v = dpp_max<0x114>(v);
  v = dpp_max<0x118>(v);
  v = dpp_max<0x142>(v);
  v = dpp_max<0x143>(v);
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}

// ---------------------------------------------------------------------------
// Tokens to fp16
// ---------------------------------------------------------------------------
// The exponent field of the largest finite magnitude seen so far (at least 1).
__device__ __forceinline__ uint32_t max_exponent(uint32_t e, float v) {
  const uint32_t u = (__float_as_uint(v) >> 23) & 255u;
  return max(e, u == 255u ? 1u : u);
}
// 2^n with n = 141 - e brings that magnitude under 2^15; infinities and NaN pass
__device__ __forceinline__ void to_parts(float v, int n, _Float16 &hi, _Float16 &lo) {
  const float f = ldexpf(v, n);
  hi = static_cast<_Float16>(f);
  lo = finite_f(f) ? static_cast<_Float16>(f - static_cast<float>(hi)) : static_cast<_Float16>(0.0f);
}

// One wave converts one token: its largest exponent, then its values, which it
// holds in registers (or reads again: past 6,144 bf16 or 2,048 fp32 columns).  The
// tile's other tokens are neighbouring waves', so that the 16-byte pieces of a
// line are written at about the same time.
template <int P>
__device__ __forceinline__ void convert_token(const void *x, int64_t cols, const Tokens &X, int64_t t, int lane) {
  constexpr int U = P == 1 ? 12 : 4;  // loads in flight, 512 columns each
  u32x4 raw[U][P];
  const char *row = static_cast<const char *>(x) + t * cols * (2 * P);
  const auto load = [&](int64_t k) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k + u * 512 >= cols) break;
      const int64_t col = k + u * 512 + lane * 8;
      const char *from = row + (col < cols ? col : 0) * (2 * P);  // past the row: its first values again
#pragma unroll
      for (int i = 0; i < P; ++i) raw[u][i] = ldu<u32x4>(from + 16 * i);
    }
  };
  const auto value = [&](int u, int j) __attribute__((always_inline)) {
    if (P == 2) return __uint_as_float(raw[u][j >> 2][j & 3]);
    const uint32_t w = raw[u][0][j >> 1];
    return __uint_as_float(j & 1 ? w & 0xffff0000u : w << 16);
  };
  uint32_t e = 1;
  for (int64_t k = 0; k < cols; k += 512 * U) {
    load(k);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k + u * 512 >= cols) break;
#pragma unroll
      for (int j = 0; j < 8; ++j) e = max_exponent(e, value(u, j));
    }
  }
  const int n = 141 - static_cast<int>(wave_max_u32(e));
  for (int64_t k = 0; k < cols; k += 512 * U) {
    if (cols > 512 * U) load(k);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t col = k + u * 512 + lane * 8;
      if (k + u * 512 >= cols) break;
      if (col >= cols) continue;
      const int g = static_cast<int>(col & 255) >> 3;  // group of the block: quarter g / 8, step g % 8
      half8v hi, lo;
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        _Float16 a, b;
        to_parts(value(u, kept_at(h)), n, a, b);
        hi[h] = a;
        lo[h] = b;
      }
      _Float16 *p = X.x16 + ((col >> 8) * X.ntile + (t >> 4)) * P * 4096 +
                    ((g & 7) * 64 + (g >> 3) * 16 + (t & 15)) * 8;
      *reinterpret_cast<half8v *>(p) = hi;
      if (P == 2) *reinterpret_cast<half8v *>(p + 4096) = lo;
    }
  }
  if (lane == 0) X.ex[t] = -n;
}

// One codebook entry per thread.  Every product with a multiplier is exact in
// fp16 if that with the largest is: products of odd numbers are odd, so the
// largest has the most bits.
__device__ __forceinline__ void convert_codebook(const Codebooks &B, int wg) {
  const int which = wg >= B.wg[0] ? 1 : 0;
  const int i = (which ? wg - B.wg[0] : wg) * 512 + static_cast<int>(threadIdx.x);
  if (i >= B.n[which]) return;
  float g[8];
  load8u(B.grid[which], 0, static_cast<int64_t>(i) * 8, g);
  half8v o;
  bool inexact = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const auto check = [&](float f) { inexact |= static_cast<float>(static_cast<_Float16>(f)) != f; };
    o[j] = static_cast<_Float16>(g[kept_at(j)]);
    check(g[j]);
    if (B.iq1[which]) {
      check(15.0f * (g[j] + 0.125f));
      check(15.0f * (g[j] - 0.125f));
    } else {
      check(31.0f * g[j]);
    }
  }
  reinterpret_cast<half8v *>(B.tab[which])[i] = o;
  if (inexact) raise_status(B.status, ST_ROUNDED);
}

// ---------------------------------------------------------------------------
// Waves that split K.  A workgroup is kw x rw waves: wave (kg, rg) takes every
// kw-th block of its row group's RT tiles of 16 rows.  The blocks of a row are
// read by the workgroup at the same time, so that its lines, which hold nearly
// two blocks, are fetched once (one wave walking along its rows found them gone
// from L1 at every other block, and was bound by the requests); and a wave's
// token operand, one block, stays in registers for all of its row tiles.
// ---------------------------------------------------------------------------
struct Split {
  int kw, rw, kg, rg;
};
inline int split_kw(int64_t nb) { return nb < 8 ? static_cast<int>(nb) : 8; }
inline int split_rw(int64_t nb) { return 8 / split_kw(nb); }
__device__ __forceinline__ Split split_of(int64_t nb) {
  Split s;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  s.kw = nb < 8 ? static_cast<int>(nb) : 8;
  s.rw = static_cast<int>(blockDim.x >> 6) / s.kw;
  s.kg = wave % s.kw;
  s.rg = wave / s.kw;
  return s;
}

template <int P, int C> struct Operand {
  half8v v[8][C][P];
};
// xp[c]: the lane's share of the block
template <int P, int C>
__device__ __forceinline__ void load_operand(Operand<P, C> &x, const _Float16 *const (&xp)[C]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int p = 0; p < P; ++p) x.v[i][c][p] = *reinterpret_cast<const half8v *>(xp[c] + p * 4096 + i * 512);
}

// acc[rt][m][c] += the wave's blocks of M matrices.  rowp(m, rt): the lane's row;
// loadx(b, x): the operand of block b.
template <int F, int P, int C, int RT, int M, class RowP, class LoadX>
__device__ __forceinline__ void split_blocks(int64_t nb, const Split &S, const uint4 *tab, RowP rowp, LoadX loadx,
                                             f32x4 (&acc)[RT][M][C]) {
  const int q = (threadIdx.x & 63) >> 4;
  Operand<P, C> x;
  Words words[M];
#pragma unroll
  for (int m = 0; m < M; ++m) words[m] = load_words<F>(rowp(m, 0) + static_cast<int64_t>(S.kg) * Geo<F>::BYTES, q);
  for (int64_t b = S.kg; b < nb; b += S.kw) {
    loadx(b, x);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      Words next[M];  // the next row tile, or the first of the next block
      const int64_t bn = rt + 1 < RT ? b : min(b + S.kw, nb - 1);
#pragma unroll
      for (int m = 0; m < M; ++m) next[m] = load_words<F>(rowp(m, rt + 1 < RT ? rt + 1 : 0) + bn * Geo<F>::BYTES, q);
      __builtin_amdgcn_sched_barrier(0);  // one row tile's work at a time: more costs registers, and with them waves
      f32x4 part[M][C];
      Raw raw[M];
#pragma unroll
      for (int m = 0; m < M; ++m) {
        raw[m] = unpack<F>(words[m], q);
#pragma unroll
        for (int c = 0; c < C; ++c) part[m][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int m = 0; m < M; ++m) {
          const half8v w = group_half8<F>(raw[m], i, tab);
#pragma unroll
          for (int c = 0; c < C; ++c)
#pragma unroll
            for (int p = 0; p < P; ++p)
              part[m][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x.v[i][c][p], w, part[m][c], 0, 0, 0);
        }
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const float d = block_scale<F>(raw[m]);
#pragma unroll
        for (int c = 0; c < C; ++c) scale_add(acc[rt][m][c], part[m][c], d);
        words[m] = next[m];
      }
    }
  }
}

// Sums over the kw waves of each row group through LDS, in their order, G tiles
// of 16 x 16 at a time; then f(rg, tile, lane, sum).  red: 8 * G * 64 f32x4.
template <int N, int G, class Fn>
__device__ __forceinline__ void reduce_split(const f32x4 *acc, f32x4 *red, const Split &S, Fn f) {
  const int lane = static_cast<int>(threadIdx.x) & 63;
#pragma unroll
  for (int g = 0; g < N; g += G) {
    __syncthreads();  // what the memory held before is read
#pragma unroll
    for (int j = 0; j < G; ++j) red[((S.rg * S.kw + S.kg) * G + j) * 64 + lane] = acc[g + j];
    __syncthreads();
    for (int i = threadIdx.x; i < S.rw * G * 64; i += blockDim.x) {
      const int rg = i / (G * 64), rest = i % (G * 64);
      const f32x4 *p = red + rg * S.kw * G * 64 + rest;
      f32x4 s = p[0];
      for (int k = 1; k < S.kw; ++k) s += p[k * G * 64];
      f(rg, g + rest / 64, rest & 63, s);
    }
  }
}

#endif  // __HIPCC__

}  // namespace iq
