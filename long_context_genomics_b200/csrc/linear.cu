// linear.cu -- ag_linear_fwd and ag_linear_bwd: how their products are run.
//
//   y = act(x W^T + b) + residual;  dx = (dy W) act'(preact);  dW = dy^T x;
//   db = sum over rows of dy.
//
// The products go to the tensor cores (linear_sm100.cu), planned here; beside
// them are the kernels that join split sums, copy operands whose rows TMA cannot
// read, and sum dy's columns.
#include "ag_internal.h"
#include "linear_epilogue.cuh"
#include "linear_gemm.h"

namespace ag {
namespace {

// --------------------------------------------------------------------------
// The plan of a product on `clusters` 2-SM clusters: the tile width and the
// parts of the summed dimension with the least estimated time, in cycles.
GemmPlan plan_gemm(int64_t M, int64_t N, int64_t K, int clusters) {
  const int64_t k_tiles = (K + 63) / 64;
  GemmPlan best{256, 1};
  double least = 0;
  for (int bn = 256; bn >= 128; bn -= 128) {
    const int64_t tiles = ((M + 255) / 256) * ((N + bn - 1) / bn);
    for (int splits = 1; splits <= 32 && splits <= k_tiles; ++splits) {
      const int64_t waves = (tiles * splits + clusters - 1) / clusters;
      const int64_t deep = (k_tiles + splits - 1) / splits;
      double t = static_cast<double>(waves) * (deep * (bn == 256 ? 530 : 300) + 500) +
                 (bn == 256 ? 4000 : 2500);
      // The join: a second launch, and every partial sum written and read.
      if (splits > 1) t += 4000 + static_cast<double>(splits) * M * partial_ld(N) * 8 / 4000;
      if (least == 0 || t < least) least = t, best = {bn, splits};
    }
  }
  return best;
}

// --------------------------------------------------------------------------
// C from its partial sums: V columns of a row per thread, the parts added in
// order.
template <int V>
__global__ void __launch_bounds__(256)
    linear_join_kernel(const float *__restrict__ partial, int splits, int64_t M, int64_t N,
                       int64_t ld, const LinearEpilogue e) {
  const int64_t per_row = (N + V - 1) / V;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= M * per_row) return;
  const int64_t row = i / per_row, col = i % per_row * V;
  float v[V], bias[V];
#pragma unroll
  for (int c = 0; c < V; ++c) v[c] = 0.f, bias[c] = e.bias ? e.bias[col + c] : 0.f;
  for (int s = 0; s < splits; ++s) {
    float w[V];
    load_values<V>(partial, (s * M + row) * ld + col, AG_F32, w);
#pragma unroll
    for (int c = 0; c < V; ++c) v[c] += w[c];
  }
  linear_finish<V>(e, v, bias, row, col);
}

// A copy of a 16-bit matrix with rows that TMA can read.
__global__ void __launch_bounds__(256)
    pack_rows_kernel(const uint16_t *__restrict__ from, int64_t ld_from, uint16_t *__restrict__ to,
                     int64_t ld_to, int64_t rows, int64_t cols) {
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
    for (int64_t c = threadIdx.x; c < cols; c += 256) to[r * ld_to + c] = from[r * ld_from + c];
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

// --------------------------------------------------------------------------
// The workspace is laid out by the same code that uses it: with base NULL only
// its size comes out.
struct Workspace {
  char *base;
  int64_t used = 0;
  void *take(int64_t bytes) {
    void *p = base ? base + used : nullptr;
    used += (bytes + 255) / 256 * 256;
    return p;
  }
};

bool tma_readable(const void *p, int64_t ld) { return aligned(p, 16) && ld % 8 == 0; }

// The operand as TMA can read it, in place or as a copy in the workspace.
struct Packed {
  Operand op;
  bool copy;
};
Packed place(const void *p, int64_t rows, int64_t cols, int64_t ld, Workspace &ws) {
  if (tma_readable(p, ld)) return {{p, rows, cols, ld}, false};
  const int64_t ld_to = (cols + 7) / 8 * 8;
  return {{ws.take(rows * ld_to * 2), rows, cols, ld_to}, true};
}
cudaError_t fill(const Packed &k, const void *p, int64_t ld, int num_sms, cudaStream_t s) {
  if (!k.copy) return cudaSuccess;
  const int64_t blocks = k.op.rows < 16 * num_sms ? k.op.rows : 16 * num_sms;
  pack_rows_kernel<<<static_cast<unsigned>(blocks), 256, 0, s>>>(
      static_cast<const uint16_t *>(p), ld, static_cast<uint16_t *>(const_cast<void *>(k.op.p)),
      k.op.ld, k.op.rows, k.op.cols);
  return cudaGetLastError();
}

int64_t partial_bytes(const GemmPlan &plan, int64_t M, int64_t N) {
  return plan.splits > 1 ? plan.splits * M * partial_ld(N) * 4 : 0;
}

cudaError_t run(Gemm &g) {
  cudaError_t e = launch_gemm(g);
  if (e != cudaSuccess || g.plan.splits == 1) return e;
  const int v = g.epi.vec8 ? 8 : 1;
  const int64_t blocks = (g.M * ((g.N + v - 1) / v) + 255) / 256;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  if (v == 8)
    linear_join_kernel<8><<<static_cast<unsigned>(blocks), 256, 0, g.stream>>>(
        g.partial, g.plan.splits, g.M, g.N, partial_ld(g.N), g.epi);
  else
    linear_join_kernel<1><<<static_cast<unsigned>(blocks), 256, 0, g.stream>>>(
        g.partial, g.plan.splits, g.M, g.N, partial_ld(g.N), g.epi);
  return cudaGetLastError();
}

struct FwdLayout {
  Packed x, W;
  GemmPlan plan;
  float *partial;
};
FwdLayout fwd_layout(const LinearFwd &a, Workspace &ws) {
  FwdLayout l;
  l.plan = plan_gemm(a.M, a.N, a.K, a.num_sms / 2);
  l.x = place(a.x, a.M, a.K, a.ldx, ws);
  l.W = place(a.W, a.N, a.K, a.ldw, ws);
  l.partial = static_cast<float *>(ws.take(partial_bytes(l.plan, a.M, a.N)));
  return l;
}

struct BwdLayout {
  Packed dy, x, W;
  GemmPlan dx_plan, dW_plan;
  float *partial;  // of dx, then of dW
};
BwdLayout bwd_layout(const LinearBwd &a, Workspace &ws) {
  BwdLayout l{};
  int64_t partial = 0;
  if (a.dx.out || a.dW.out) l.dy = place(a.dy, a.M, a.N, a.lddy, ws);
  if (a.dx.out) {
    l.dx_plan = plan_gemm(a.M, a.K, a.N, a.num_sms / 2);
    l.W = place(a.W, a.N, a.K, a.ldw, ws);
    partial = partial_bytes(l.dx_plan, a.M, a.K);
  }
  if (a.dW.out) {
    l.dW_plan = plan_gemm(a.N, a.K, a.M, a.num_sms / 2);
    l.x = place(a.x, a.M, a.K, a.ldx, ws);
    const int64_t b = partial_bytes(l.dW_plan, a.N, a.K);
    partial = b > partial ? b : partial;
  }
  l.partial = static_cast<float *>(ws.take(partial));
  return l;
}

}  // namespace

cudaError_t linear_fwd_workspace(const LinearFwd &a, int64_t *bytes) {
  Workspace ws{nullptr};
  fwd_layout(a, ws);
  *bytes = ws.used;
  return cudaSuccess;
}

cudaError_t launch_linear_fwd(const LinearFwd &a) {
  Workspace ws{static_cast<char *>(a.workspace)};
  const FwdLayout l = fwd_layout(a, ws);
  cudaError_t e = fill(l.x, a.x, a.ldx, a.num_sms, a.stream);
  if (e == cudaSuccess) e = fill(l.W, a.W, a.ldw, a.num_sms, a.stream);
  if (e != cudaSuccess) return e;
  Gemm g{l.x.op, l.W.op, false, false, a.M, a.N, a.K, l.plan, l.partial, a.epi,
         a.num_sms, a.err, a.encode, a.stream};
  return run(g);
}

cudaError_t linear_bwd_workspace(const LinearBwd &a, int64_t *bytes) {
  Workspace ws{nullptr};
  bwd_layout(a, ws);
  *bytes = ws.used;
  return cudaSuccess;
}

cudaError_t launch_linear_bwd(const LinearBwd &a) {
  Workspace ws{static_cast<char *>(a.workspace)};
  const BwdLayout l = bwd_layout(a, ws);
  cudaError_t e = fill(l.dy, a.dy, a.lddy, a.num_sms, a.stream);
  if (e == cudaSuccess) e = fill(l.W, a.W, a.ldw, a.num_sms, a.stream);
  if (e == cudaSuccess) e = fill(l.x, a.x, a.ldx, a.num_sms, a.stream);
  if (e == cudaSuccess && a.dx.out) {
    Gemm g{l.dy.op, l.W.op, false, true, a.M, a.K, a.N, l.dx_plan, l.partial, a.dx,
           a.num_sms, a.err, a.encode, a.stream};
    e = run(g);
  }
  if (e == cudaSuccess && a.dW.out) {
    Gemm g{l.dy.op, l.x.op, true, true, a.N, a.K, a.M, l.dW_plan, l.partial, a.dW,
           a.num_sms, a.err, a.encode, a.stream};
    e = run(g);
  }
  if (e == cudaSuccess && a.db) {
    column_sum_kernel<<<static_cast<unsigned>((a.N + 31) / 32), 256, 0, a.stream>>>(
        static_cast<const uint16_t *>(a.dy), a.lddy, a.M, a.N, a.dx.dtype, a.db);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace ag
