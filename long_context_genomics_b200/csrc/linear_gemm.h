// linear_gemm.h -- the tensor-core product behind the linear layers, between
// linear.cu (which plans it) and linear_sm100.cu.
#pragma once

#include "ag_internal.h"

namespace ag {

// A 16-bit matrix in memory: `rows` rows of `cols` dense elements, ld apart;
// p 16-byte aligned and ld a multiple of 8 (what TMA reads).
struct Operand {
  const void *p;
  int64_t rows, cols, ld;
};

struct GemmPlan {
  int bn;      // columns of a tile: 256 or 128
  int splits;  // parts of the summed dimension
};

// C[m, n] = sum_k A(m, k) B(n, k), m < M, n < N, k < K.  A lies as [M][K], or
// with a_mn as [K][M]; B as [N][K], or with b_mn as [K][N] (a_mn only with
// b_mn).
struct Gemm {
  Operand A, B;
  bool a_mn, b_mn;
  int64_t M, N, K;
  GemmPlan plan;
  float *partial;  // plan.splits > 1: [splits][M][partial_ld(N)] float32
  LinearEpilogue epi;
  int num_sms;
  unsigned *err;
  EncodeTiledFn encode;
  cudaStream_t stream;
};
inline int64_t partial_ld(int64_t N) { return (N + 7) / 8 * 8; }
cudaError_t launch_gemm(const Gemm &g);

}  // namespace ag
