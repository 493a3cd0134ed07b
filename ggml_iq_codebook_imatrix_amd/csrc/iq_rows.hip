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

#include "iq_train.hpp"

namespace iq {
namespace {

// acc[j][c] += p A of the adapters that the wave's tokens (tiles tt .. tt + C - 1) name, columns col + j of the lane's
// eight.  32 ranks at a time: a lane has eight ranks of its eight columns, which byte permutations make operands of
// (bf16; p is the sum of three bf16 values, without a rounding), or four ranks at a time on the fp32 cores.  What
// rows of tokens with other adapters give is dropped.
template <int P, int C>
__device__ __forceinline__ void add_adapters(const RowsArgs &A, int64_t tt, int64_t col, f32x4 (&acc)[8][C]) {
  const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  const int64_t cols = A.nb * 256, mytok = tt * 16 + lane;
  const int mine = lane < 16 * C && mytok < A.T ? A.ids[mytok] : -1;
  uint64_t todo = __ballot(mine >= 0);
  while (todo) {
    const int a = __builtin_amdgcn_readlane(mine, __builtin_ctzll(todo));
    const uint64_t group = __ballot(mine == a);
    todo &= ~group;
    for (int r0 = 0; r0 < A.rank; r0 += P == 1 ? 32 : 4) {
      if constexpr (P == 1) {
        const uint16_t *from = static_cast<const uint16_t *>(A.a) + static_cast<int64_t>(a) * A.rank * cols + col;
        u32x4 w[8];  // ranks r0 + 8 q + i; past the last p is zero
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = ldu<u32x4>(from + min(r0 + 8 * q + i, A.rank - 1) * cols);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          if (!((group >> (16 * c)) & 0xffffu)) continue;
          bf16x8 v[3];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float f = r0 + 8 * q + i < A.rank ? A.p[(r0 + 8 * q + i) * A.tpad + (tt + c) * 16 + n] : 0.0f;
#pragma unroll
            for (int k = 0; k < 3; ++k) {
              const uint32_t top = __float_as_uint(f) & 0xffff0000u;
              v[k][i] = __builtin_bit_cast(__bf16, static_cast<uint16_t>(top >> 16));
              f = finite_f(f) ? f - __uint_as_float(top) : 0.0f;
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t sel = j & 1 ? 0x07060302u : 0x05040100u;
            u32x4 o;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = __builtin_amdgcn_perm(w[2 * i + 1][j >> 1], w[2 * i][j >> 1], sel);
            f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < 3; ++k)
              d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[k], __builtin_bit_cast(bf16x8, o), d, 0, 0, 0);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if ((group >> (16 * c + 4 * q + k)) & 1u) acc[j][c][k] += d[k];
          }
        }
      } else {
        float w[8];
        load8u(A.a, 0, (static_cast<int64_t>(a) * A.rank + min(r0 + q, A.rank - 1)) * cols + col, w);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          if (!((group >> (16 * c)) & 0xffffu)) continue;
          const float v = r0 + q < A.rank ? A.p[(r0 + q) * A.tpad + (tt + c) * 16 + n] : 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const f32x4 d = __builtin_amdgcn_mfma_f32_16x16x4f32(v, w[j], f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if ((group >> (16 * c + 4 * q + k)) & 1u) acc[j][c][k] += d[k];
          }
        }
      }
    }
  }
}

// Waves: 4 token groups (of C tiles) by H halves of a block's columns.  LORA: with adapters.
template <int F, int P, int C, int H, bool LORA>
__global__ void __launch_bounds__(256 * H, H) rows_kernel(RowsArgs A) {
  constexpr int NW = 4 * H, NT = 64 * NW, TA = 4 * C;
  constexpr int W = (Geo<F>::BYTES + 5) / 4, NR = (64 * W + NT - 1) / NT;  // words of a row's block, a thread's share
  __shared__ uint4 s_tab[Geo<F>::N];
  __shared__ u32x4 s_a[2][TA * P * 2 * 64];   // [tile][part][step][lane]
  __shared__ u32x4 s_b[2][H * 8 * P * 2 * 64];  // [half][column j][part][step][lane]
  __shared__ uint32_t s_raw[2][64 * W];
  load_table<F>(s_tab, A.tab);
  const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wt = wave / H, wh = wave % H;
  const int64_t cb = blockIdx.x / (2 / H), cols = A.nb * 256, rowbytes = A.nb * Geo<F>::BYTES;
  const int half0 = H == 2 ? 0 : static_cast<int>(blockIdx.x & 1);  // the first half that the workgroup takes
  const int64_t tt0 = static_cast<int64_t>(blockIdx.y) * TA;
  const int64_t per = (A.rows + 63) / 64, chunks = per * A.nmat;
  const int64_t share = (chunks + A.splits - 1) / A.splits, ch0 = blockIdx.z * share, ch1 = min(ch0 + share, chunks);
  const int ew = weight_exponent(A.B);
  const float unit = ldexpf(1.0f, 15 - ew - (Geo<F>::IQ1 ? 0 : 3));
  const uint8_t *const p0 = A.packed[0] + cb * Geo<F>::BYTES, *const p1 = A.packed[A.nmat - 1] + cb * Geo<F>::BYTES;

  // Chunk ch's blocks, whole aligned words; rows past the last read the last's.
  uint32_t raw[NR];
  const auto load_raw = [&](int64_t ch) __attribute__((always_inline)) {
    const bool second = ch >= per;
    const uint8_t *base = second ? p1 : p0;
    const int64_t row0 = (second ? ch - per : ch) * 64;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int u = i * NT + static_cast<int>(threadIdx.x);
      if (64 * W % NT && u >= 64 * W) break;
      const int r = u / W, w = u % W;
      const uintptr_t at = reinterpret_cast<uintptr_t>(base + min(row0 + r, A.rows - 1) * rowbytes);
      const int last = (static_cast<int>(at & 2) + Geo<F>::BYTES - 1) >> 2;
      raw[i] = ldw<uint32_t>((at & ~uintptr_t(3)) + 4 * min(w, last));
    }
  };
  const auto store_raw = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int u = i * NT + static_cast<int>(threadIdx.x);
      if (64 * W % NT && u >= 64 * W) break;
      s_raw[buf][u] = raw[i];
    }
  };
  const auto fetch = [&](int64_t ch, int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i0 = 0; i0 < TA * P * 2; i0 += NW) {
      const int i = i0 + wave;
      const int64_t tile = min(tt0 + i / (2 * P), A.G.ntile - 1);
      const u32x4 *from = reinterpret_cast<const u32x4 *>(A.G.g16) + (ch * A.G.ntile + tile) * (P * 128) +
                          (i % (2 * P)) * 64 + lane;
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from,
                                       (__attribute__((address_space(3))) void *)&s_a[buf][i * 64], 16, 0, 0);
    }
  };
  // The thread's group and four rows of each chunk.
  const int group = (half0 + wave % H) * 16 + n, quad = (wave / H) * 4 + q;
  const auto decode = [&](int64_t ch, int buf) __attribute__((always_inline)) {
    const bool second = ch >= per;
    const uintptr_t base = reinterpret_cast<uintptr_t>(second ? p1 : p0);
    const int64_t row0 = (second ? ch - per : ch) * 64;
    uint32_t hi[4][4], lo[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t r = min(row0 + quad * 4 + j, A.rows - 1);
      const uint32_t off = static_cast<uint32_t>(base + r * rowbytes) & 2u;
      const uint8_t *blk = reinterpret_cast<const uint8_t *>(&s_raw[buf][(quad * 4 + j) * W]) + off;
      whole_weights<F, P>(read_fields<F>(blk, group), unit, s_tab, hi[j], lo[j]);
    }
    // operand [wave % H][column][part][quad / 8], lane 16 ((quad % 8) / 2) + n, half quad % 2
    uint2 *to = reinterpret_cast<uint2 *>(s_b[buf]) +
                (((wave % H) * 8 * P * 2 + quad / 8) * 64 + (quad % 8) / 2 * 16 + n) * 2 + quad % 2;
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
      for (int k = 0; k < 2; ++k) {  // column p + 4 k
        const uint32_t sel = k ? 0x07060302u : 0x05040100u;
#pragma unroll
        for (int part = 0; part < P; ++part) {
          const uint32_t(&v)[4][4] = part ? lo : hi;
          to[((p + 4 * k) * P + part) * 256] = make_uint2(__builtin_amdgcn_perm(v[1][p], v[0][p], sel),
                                                          __builtin_amdgcn_perm(v[3][p], v[2][p], sel));
        }
      }
  };

  f32x4 acc[8][C], part[P == 2 ? 8 : 1][C];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int c = 0; c < C; ++c) acc[j][c] = part[j % (P == 2 ? 8 : 1)][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (ch0 < ch1) {
    load_raw(ch0);
    fetch(ch0, 0);
    store_raw(0);
    load_raw(min(ch0 + 1, ch1 - 1));
    __syncthreads();
    decode(ch0, 0);
    store_raw(1);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the barrier does not wait for loads into LDS
    __syncthreads();
  }
  for (int64_t ch = ch0; ch < ch1; ++ch) {
    const int cur = static_cast<int>(ch - ch0) & 1;
    if (ch + 1 < ch1) {
      fetch(ch + 1, cur ^ 1);
      load_raw(min(ch + 2, ch1 - 1));
      __builtin_amdgcn_sched_barrier(0);  // the loads above go out before the work below
      decode(ch + 1, cur ^ 1);
    }
#pragma unroll
    for (int step = 0; step < 2; ++step) {
      half8v a[C][P];
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int p = 0; p < P; ++p)
          a[c][p] = __builtin_bit_cast(half8v, s_a[cur][(((wt * C + c) * P + p) * 2 + step) * 64 + lane]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        half8v b[P];
#pragma unroll
        for (int p = 0; p < P; ++p)
          b[p] = __builtin_bit_cast(half8v, s_b[cur][(((wh * 8 + j) * P + p) * 2 + step) * 64 + lane]);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          f32x4 &to = P == 2 ? part[j % (P == 2 ? 8 : 1)][c] : acc[j][c];
          to = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[c][0], b[0], to, 0, 0, 0);
          if (P == 2) {
            to = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[c][P - 1], b[0], to, 0, 0, 0);
            to = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[c][0], b[P - 1], to, 0, 0, 0);
          }
        }
      }
    }
    if (P == 2 && (((ch - ch0) & 3) == 3 || ch + 1 == ch1)) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int c = 0; c < C; ++c) {
          f32x4 &p = part[j % (P == 2 ? 8 : 1)][c];
          acc[j][c] += p;
          p = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
    }
    if (ch + 1 < ch1) {
      store_raw(cur);  // read by the decode before the last barrier
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
    }
  }
  // tokens 4 q + k of tile c, columns 8 n + j of the wave's half
  const int64_t col = cb * 256 + (half0 + wh) * 128 + 8 * n, tw = tt0 + wt * C;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int4 e4 = *reinterpret_cast<const int4 *>(A.G.ex + min((tw + c) * 16 + q * 4, A.G.ntile * 16 - 4));
    const int e[4] = {e4.x, e4.y, e4.z, e4.w};
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[j][c][k] = ldexpf(acc[j][c][k], e[k] + ew - 15);
  }
  if (LORA && blockIdx.z == 0) add_adapters<P, C>(A, tw, col, acc);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int64_t t0 = (tw + c) * 16 + q * 4;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (t0 + k >= A.T) continue;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = acc[j][c][k];
      if (A.splits > 1)
        store8u(A.partial + (blockIdx.z * A.T + t0 + k) * cols, 0, col, v);
      else
        store8u(A.out, P == 1, (t0 + k) * cols + col, v);
    }
  }
}

// The splits' sums, in their order.
template <int P> __global__ void __launch_bounds__(256) rows_join_kernel(RowsArgs A) {
  const int64_t n = A.T * A.nb * 256, i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (i >= n) return;
  float v[8];
  load8u(A.partial, 0, i, v);
  for (int s = 1; s < A.splits; ++s) {
    float w[8];
    load8u(A.partial, 0, s * n + i, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += w[j];
  }
  store8u(A.out, P == 1, i, v);
}

// An empty sum's result (a fill by the runtime is no kernel, and would enter a captured graph as another node).
__global__ void __launch_bounds__(256) zero_kernel(uint16_t *p, size_t n) {
  for (size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<size_t>(gridDim.x) * 256)
    p[i] = 0;
}

template <int F, int P, int C, int H, bool LORA> void launch_tile(const RowsArgs &A, hipStream_t stream) {
  hipLaunchKernelGGL((rows_kernel<F, P, C, H, LORA>),
                     dim3(static_cast<unsigned>(A.nb * (2 / H)), static_cast<unsigned>((A.G.ntile + 4 * C - 1) / (4 * C)),
                          static_cast<unsigned>(A.splits)),
                     dim3(256 * H), 0, stream, A);
}

template <int F, bool LORA> void launch_fmt(int dtype, const RowsArgs &A, hipStream_t stream) {
  constexpr bool big = Geo<F>::N > 1024;  // 32 KiB of codebook
  if (dtype == IQ_DTYPE_F32) return launch_tile<F, 2, big ? 1 : 2, 1, LORA>(A, stream);
  launch_tile<F, 1, big ? 3 : 4, 2, LORA>(A, stream);
}

}  // namespace

int rows_splits(int64_t T, int64_t cols, int64_t chunks, int dtype) {
  const int64_t wgs = (cols / 128) * ((T + 127) / 128);
  int64_t s = 512 / (wgs < 1 ? 1 : wgs);
  if (s > chunks / 4) s = chunks / 4;
  (void)dtype;
  return static_cast<int>(s < 1 ? 1 : s > 64 ? 64 : s);
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
  if (A.splits > 1) {
    const int64_t units = A.T * A.nb * 32;
    const dim3 wgs(static_cast<unsigned>((units + 255) / 256));
    if (dtype == IQ_DTYPE_F32)
      hipLaunchKernelGGL(rows_join_kernel<2>, wgs, dim3(256), 0, stream, A);
    else
      hipLaunchKernelGGL(rows_join_kernel<1>, wgs, dim3(256), 0, stream, A);
    if (!run_launched()) return IQ_ERR_HIP;
  }
  return IQ_OK;
}

}  // namespace iq
