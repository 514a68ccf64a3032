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
  int bn;       // columns of a tile: 256 or 128
  int splits;   // parts of the summed dimension
  double time;  // estimated, in SM cycles
};

// Which items (tiles x parts) of a product a cluster takes, one a round: in the
// first `extra` rounds only the clusters from `from` on take one each, in later
// rounds all of them.  So the second of two products in one launch goes first to
// the clusters that have one item fewer of the first.
struct Turns {
  int from, extra;
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
// The gradients of a linear layer in one launch: dW (a_mn, b_mn; its items go
// first), then dx (b_mn, one part) by `turns`; both with tiles of one width.
// `done` is false, and nothing is launched, where TMA can address dx's arrays but
// not dW's (which is rare enough to take two launches).
cudaError_t launch_gemm_pair(const Gemm &dW, const Gemm &dx, Turns turns, bool *done);

}  // namespace ag
