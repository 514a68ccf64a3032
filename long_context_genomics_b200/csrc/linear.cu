// linear.cu -- the products of the linear layers (ag_linear_fwd, ag_linear_bwd)
// on the CUDA cores, and the column sums of the bias gradient.
//
//   y = act(x W^T + b) + residual;  dx = (dy W) act'(preact);  dW = dy^T x;
//   db = sum over rows of dy.
#include "ag_internal.h"
#include "linear_epilogue.cuh"

namespace ag {
namespace {

// C[m, n] = sum_k A(m, k) B(n, k) with element (m, k) of A at m * am + k * ak
// and (n, k) of B at n * bn + k * bk: 64 x 64 tiles, 4 x 4 per thread, float32
// sums in a fixed order.
constexpr int kT = 64, kTK = 16;

__global__ void __launch_bounds__(256)
    linear_simt_kernel(const uint16_t *__restrict__ A, int64_t am, int64_t ak,
                       const uint16_t *__restrict__ B, int64_t bn, int64_t bk, int64_t M,
                       int64_t N, int64_t K, int64_t tiles_n, const LinearEpilogue e) {
  __shared__ float a_s[kTK][kT + 1], b_s[kTK][kT + 1];
  const int64_t m0 = (blockIdx.x / tiles_n) * kT, n0 = (blockIdx.x % tiles_n) * kT;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < K; k0 += kTK) {
    for (int i = threadIdx.x; i < kT * kTK; i += 256) {
      const int r = ak == 1 ? i / kTK : i % kT, c = ak == 1 ? i % kTK : i / kT;
      float v[1] = {0.f};
      if (m0 + r < M && k0 + c < K) load_values<1>(A, (m0 + r) * am + (k0 + c) * ak, e.dtype, v);
      a_s[c][r] = v[0];
      const int r2 = bk == 1 ? i / kTK : i % kT, c2 = bk == 1 ? i % kTK : i / kT;
      float w[1] = {0.f};
      if (n0 + r2 < N && k0 + c2 < K) load_values<1>(B, (n0 + r2) * bn + (k0 + c2) * bk, e.dtype, w);
      b_s[c2][r2] = w[0];
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kTK; ++c) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = a_s[c][ty + 16 * i], b[i] = b_s[c][tx + 16 * i];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m < M && n < N) {
        float v[1] = {acc[i][j]};
        const float b[1] = {e.bias ? e.bias[n] : 0.f};
        linear_finish<1>(e, v, b, m, n);
      }
    }
}

// db[n] = sum_m dy[m, n]: 32 columns per block, 8 lanes over the rows.
__global__ void __launch_bounds__(256)
    column_sum_kernel(const uint16_t *__restrict__ dy, int64_t ld, int64_t M, int64_t N,
                      int dtype, float *__restrict__ db) {
  __shared__ float part[8][32];
  const int c = threadIdx.x % 32, r = threadIdx.x / 32;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 32 + c;
  double s = 0.0;
  if (n < N)
    for (int64_t m = r; m < M; m += 8) {
      float v[1];
      load_values<1>(dy, m * ld + n, dtype, v);
      s += v[0];
    }
  part[r][c] = static_cast<float>(s);
  __syncthreads();
  if (r == 0 && n < N) {
    float t = 0.f;
    for (int i = 0; i < 8; ++i) t += part[i][c];
    db[n] = t;
  }
}

cudaError_t product(const void *A, int64_t am, int64_t ak, const void *B, int64_t bn, int64_t bk,
                    int64_t M, int64_t N, int64_t K, const LinearEpilogue &e, cudaStream_t s) {
  const int64_t tm = (M + kT - 1) / kT, tn = (N + kT - 1) / kT;
  if (tm * tn > 0x7FFFFFFF) return cudaErrorInvalidValue;
  linear_simt_kernel<<<static_cast<unsigned>(tm * tn), 256, 0, s>>>(
      static_cast<const uint16_t *>(A), am, ak, static_cast<const uint16_t *>(B), bn, bk, M, N, K,
      tn, e);
  return cudaGetLastError();
}

}  // namespace

cudaError_t linear_fwd_workspace(const LinearFwd &a, int64_t *bytes) {
  (void)a;
  *bytes = 0;
  return cudaSuccess;
}

cudaError_t launch_linear_fwd(const LinearFwd &a) {
  return product(a.x, a.ldx, 1, a.W, a.ldw, 1, a.M, a.N, a.K, a.epi, a.stream);
}

cudaError_t linear_bwd_workspace(const LinearBwd &a, int64_t *bytes) {
  (void)a;
  *bytes = 0;
  return cudaSuccess;
}

cudaError_t launch_linear_bwd(const LinearBwd &a) {
  cudaError_t e = cudaSuccess;
  if (a.dx.out && a.M > 0)
    e = product(a.dy, a.lddy, 1, a.W, 1, a.ldw, a.M, a.K, a.N, a.dx, a.stream);
  if (e != cudaSuccess) return e;
  if (a.dW.out) e = product(a.dy, 1, a.lddy, a.x, 1, a.ldx, a.N, a.K, a.M, a.dW, a.stream);
  if (e != cudaSuccess) return e;
  if (a.db) {
    column_sum_kernel<<<static_cast<unsigned>((a.N + 31) / 32), 256, 0, a.stream>>>(
        static_cast<const uint16_t *>(a.dy), a.lddy, a.M, a.N, a.dx.dtype, a.db);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace ag
