// iq_checkpoint.hip -- iq_checkpoint and iq_restore: activations in 8 bits
// (include/iq_train.h).
//
// Bound by memory: a thread takes eight columns, four neighbouring ones a block
// of 32, whose largest magnitude goes through two lane exchanges.  A tensor
// whose rows are whole blocks is one long row.  8,192 x 17,408 in bf16: 97 us to
// keep (432 MB, 4.4 TB/s) and 72 to restore (5.9 TB/s), f32 161 and 145 (4.5 and 5.0),
// with six tensors in turn, more than the caches hold, where a copy reaches 5.1 (a
// restore's codes are fresh from the keeping); the same tensor each time takes as
// long.  37 x 1,001 in f32 6 and 5, a launch's latency.

#include "iq_train.hpp"

namespace iq {
namespace {

constexpr int kUnits = 4;                // units of eight columns a thread, all in flight together
constexpr int kRowCols = 256 * 8 * kUnits;  // columns a workgroup takes

struct CheckpointArgs {
  const void *x;
  void *y;
  int dtype;
  int64_t cols, blocks;  // columns and blocks of a row
  uint32_t wpr;          // workgroups a row
  int8_t *codes;
  uint8_t *ex;
  int32_t *status;
};

// The row and the first column of the thread's unit u.
__device__ __forceinline__ void unit_of(const CheckpointArgs &A, int u, int64_t &row, int64_t &col) {
  row = blockIdx.x / A.wpr;
  col = static_cast<int64_t>(blockIdx.x % A.wpr) * kRowCols + (u * 256 + static_cast<int>(threadIdx.x)) * 8;
}

__global__ void __launch_bounds__(256) checkpoint_kernel(CheckpointArgs A) {
  float v[kUnits][8];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    int64_t row, col;
    unit_of(A, u, row, col);
    const int64_t at = row * A.cols + col;
    if (col + 8 <= A.cols) {
      load8u(A.x, A.dtype, at, v[u]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[u][j] = col + j < A.cols ? load1(A.x, A.dtype, at + j) : 0.0f;
    }
  }
  bool bad = false;
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    int64_t row, col;
    unit_of(A, u, row, col);
    uint32_t most = 0;  // magnitudes order as their bits do
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t b = __float_as_uint(v[u][j]) & 0x7fffffffu;
      if (b < 0x7f800000u) most = max(most, b);
    }
    most = max(most, static_cast<uint32_t>(__shfl_xor(static_cast<int>(most), 1, 64)));
    most = max(most, static_cast<uint32_t>(__shfl_xor(static_cast<int>(most), 2, 64)));
    int e = max(static_cast<int>(most >> 23), 1);
    if (e < 254 && rintf(ldexpf(__uint_as_float(most), 133 - e)) > 127.0f) ++e;
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool finite = finite_f(v[u][j]);
      bad |= !finite;
      const float r = fminf(fmaxf(rintf(ldexpf(v[u][j], 133 - e)), -127.0f), 127.0f);
      const int code = finite ? static_cast<int>(r) : -128;
      w[j >> 2] |= (static_cast<uint32_t>(code) & 255u) << (8 * (j & 3));
    }
    const int64_t at = row * A.cols + col;
    if (col + 8 <= A.cols) {
      const uint2 o = make_uint2(w[0], w[1]);
      __builtin_memcpy(A.codes + at, &o, 8);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col + j < A.cols) A.codes[at + j] = static_cast<int8_t>(w[j >> 2] >> (8 * (j & 3)));
    }
    if (col < A.cols && (col & 31) == 0) A.ex[row * A.blocks + (col >> 5)] = static_cast<uint8_t>(e);
  }
  if (bad) raise_status(A.status, ST_NONFINITE);
}

__global__ void __launch_bounds__(256) restore_kernel(CheckpointArgs A) {
  uint2 w[kUnits];
  int e[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    int64_t row, col;
    unit_of(A, u, row, col);
    const int64_t at = row * A.cols + col;
    w[u] = make_uint2(0, 0);
    if (col + 8 <= A.cols) {
      w[u] = ldu<uint2>(A.codes + at);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col + j < A.cols)
          (j < 4 ? w[u].x : w[u].y) |= (static_cast<uint32_t>(A.codes[at + j]) & 255u) << (8 * (j & 3));
    }
    e[u] = col < A.cols ? A.ex[row * A.blocks + (col >> 5)] : 0;
  }
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    int64_t row, col;
    unit_of(A, u, row, col);
    const int64_t at = row * A.cols + col;
    float v[8];
    decode_codes(w[u], e[u] - 133, v);
    if (col + 8 <= A.cols) {
      store8u(A.y, A.dtype, at, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col + j < A.cols) store1(A.y, A.dtype, at + j, v[j]);
    }
  }
}

int check_checkpoint(int dtype, int64_t T, int64_t cols) {
  if (run_bad_dtype(dtype)) return IQ_ERR_DTYPE;
  if (T < 0 || cols < 0 || cols > (int64_t(1) << 24) || T > (int64_t(1) << 24)) return IQ_ERR_SHAPE;
  // workgroups: of rows one by one, or of all columns in one row
  if (T * ((cols + kRowCols - 1) / kRowCols) >= 2 * kMaxWG) return IQ_ERR_SHAPE;
  return IQ_OK;
}

// Rows of whole blocks as one row.
dim3 plan_rows(CheckpointArgs &A, int64_t T, int64_t cols) {
  if (cols % 32 == 0) {
    cols *= T;
    T = 1;
  }
  A.cols = cols;
  A.blocks = (cols + 31) / 32;
  A.wpr = static_cast<uint32_t>((cols + kRowCols - 1) / kRowCols);
  return dim3(static_cast<unsigned>(T * A.wpr));
}

}  // namespace
}  // namespace iq

extern "C" {

int iq_checkpoint(const void *x, int dtype, int64_t T, int64_t cols, int8_t *codes, uint8_t *exponents,
                  int32_t *status, hipStream_t stream) {
  using namespace iq;
  const int rc = check_checkpoint(dtype, T, cols);
  if (rc != IQ_OK) return rc;
  if (T == 0 || cols == 0) return IQ_OK;
  if (!x || !codes || !exponents) return IQ_ERR_NULL;
  CheckpointArgs A{};
  A.x = x;
  A.dtype = dtype;
  A.codes = codes;
  A.ex = exponents;
  A.status = status;
  const dim3 wgs = plan_rows(A, T, cols);
  hipLaunchKernelGGL(checkpoint_kernel, wgs, dim3(256), 0, stream, A);
  return run_launched() ? IQ_OK : IQ_ERR_HIP;
}

int iq_restore(const int8_t *codes, const uint8_t *exponents, int64_t T, int64_t cols, void *y, int dtype,
               hipStream_t stream) {
  using namespace iq;
  const int rc = check_checkpoint(dtype, T, cols);
  if (rc != IQ_OK) return rc;
  if (T == 0 || cols == 0) return IQ_OK;
  if (!y || !codes || !exponents) return IQ_ERR_NULL;
  CheckpointArgs A{};
  A.y = y;
  A.dtype = dtype;
  A.codes = const_cast<int8_t *>(codes);
  A.ex = const_cast<uint8_t *>(exponents);
  const dim3 wgs = plan_rows(A, T, cols);
  hipLaunchKernelGGL(restore_kernel, wgs, dim3(256), 0, stream, A);
  return run_launched() ? IQ_OK : IQ_ERR_HIP;
}

}  // extern "C"
