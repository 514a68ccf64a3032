// linear.cu -- ag_linear_fwd and ag_linear_bwd: how their products are run.
//
//   y = act(x W^T + b) + residual;  dx = (dy W) act'(preact);  dW = dy^T x;
//   db = sum over rows of dy.
//
// The products go to the tensor cores (linear_sm100.cu), planned here; beside
// them are the kernels that join split sums, copy operands whose rows TMA cannot
// read, sum dy's columns, and multiply a few rows without the tensor cores.
#include "ag_internal.h"
#include "launch.cuh"
#include "linear_epilogue.cuh"
#include "linear_gemm.h"

namespace ag {
namespace {

// --------------------------------------------------------------------------
// The plan of a product on `clusters` 2-SM clusters: the tile width and the
// parts of the summed dimension with the least estimated time, in SM cycles.
// Fitted to measurements of 20 shapes (8 x 8 to 16384 x 4096 x 1024; splits 1
// to 24, both widths): 64 terms of a tile take 620 cycles at width 256 and 430
// at 128 (twice the columns per row of A that is read), a kernel 10500 or 8700
// beside its sums, and joining splits a launch and the traffic of the partial
// sums.  Some of both sides, us: 1024 x 1024 x 1024 width 256 11.0, 128 8.4;
// 4096 x 4096 x 1024 28.7, 35.3; 1152 x 1024 x 8192 in 1, 3, 7 parts 43.8,
// 24.4, 27.1; 300 x 136 x 4096 in 1, 8, 24 parts 17.5, 10.3, 11.
double item_time(int bn, int64_t deep) { return deep * (bn == 256 ? 620 : 430) + 300; }
double join_time(int splits, int64_t M, int64_t N) {
  return splits > 1 ? 6000 + static_cast<double>(splits) * M * partial_ld(N) * 8 / 4000 : 0;
}
GemmPlan plan_gemm(int64_t M, int64_t N, int64_t K, int clusters) {
  const int64_t k_tiles = (K + 63) / 64;
  GemmPlan best{256, 1, 0};
  for (int bn = 256; bn >= 128; bn -= 128) {
    const int64_t tiles = ((M + 255) / 256) * ((N + bn - 1) / bn);
    for (int splits = 1; splits <= 32 && splits <= k_tiles; ++splits) {
      const int64_t waves = (tiles * splits + clusters - 1) / clusters;
      const int64_t deep = (k_tiles + splits - 1) / splits;
      const double t =
          waves * item_time(bn, deep) + (bn == 256 ? 10500 : 8700) + join_time(splits, M, N);
      if (best.time == 0 || t < best.time) best = {bn, splits, t};
    }
  }
  return best;
}

// Both gradients of a layer in one launch (dW [N, K] over M rows in parts, then
// dx [M, K] over N): the parts and turns with the least estimated time.  What is
// idle in one product's last round then works on the other, and a launch with
// its first loads and last stores is saved.  us in two launches and in one:
// 8192 x 1152 x 1024 43.9, 36.0; 4096 x 1024 x 4096 with a GELU's slope 72.3, 61.1;
// 1024 x 1024 x 1024 17.6, 10.3; 64 x 512 x 512 11.5, 6.6; 65536 x 128 x 128 29.8,
// 28.9; 16384 x 4096 x 1024 200, 189; 777 x 501 x 1003 (plain epilogues) 21.7, 13.4;
// 1000 x 3000 x 600, whose dx could be split when alone, 24.4, 26.1.
struct PairPlan {
  int bn, splits;
  Turns turns;
  double time;
};
PairPlan plan_pair(int64_t M, int64_t N, int64_t K, int clusters) {
  const int64_t m_tiles = (M + 63) / 64, n_tiles = (N + 63) / 64;
  PairPlan best{256, 1, {0, 0}, 0};
  for (int bn = 256; bn >= 128; bn -= 128) {
    const int64_t columns = (K + bn - 1) / bn, dx_items = (M + 255) / 256 * columns,
                  dW_tiles = (N + 255) / 256 * columns;
    const double dx_item = item_time(bn, n_tiles);
    for (int splits = 1; splits <= 32 && splits <= m_tiles; ++splits) {
      const double dW_item = item_time(bn, (m_tiles + splits - 1) / splits);
      const int64_t rounds = dW_tiles * splits / clusters;
      const int from = static_cast<int>(dW_tiles * splits % clusters), few = clusters - from;
      // The clusters without an item in dW's last round can be so many rounds of
      // dx ahead.
      const int64_t ahead = from > 0 ? static_cast<int64_t>(dW_item / dx_item) + 1 : 0,
                    all_dx = (dx_items + few - 1) / few, most = ahead < all_dx ? ahead : all_dx;
      for (int extra = 0; extra <= most && extra <= 64; ++extra) {
        const int64_t left = dx_items - static_cast<int64_t>(extra) * few;
        const int64_t more = left > 0 ? (left + clusters - 1) / clusters : 0;
        const double long_way = (rounds + (from > 0)) * dW_item + more * dx_item,
                     short_way = rounds * dW_item + (extra + more) * dx_item;
        const double t = (long_way > short_way ? long_way : short_way) +
                         (bn == 256 ? 10500 : 8700) + join_time(splits, N, K);
        if (best.time == 0 || t < best.time) best = {bn, splits, {from, extra}, t};
      }
    }
  }
  return best;
}

// --------------------------------------------------------------------------
// db from the partial sums of dy's columns [parts][N] (column_sum_kernel): 32
// columns a block, its warps over the parts, all in a fixed order.
struct ColumnParts {
  const float *partial;
  int parts;
  int64_t N;
  float *db;
  __host__ unsigned blocks() const { return db ? static_cast<unsigned>((N + 31) / 32) : 0; }
};
__device__ __forceinline__ void join_columns(const ColumnParts &c, unsigned block) {
  __shared__ float sums[8][32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t n = static_cast<int64_t>(block) * 32 + lane;
  float s = 0.f;
  if (n < c.N)
    for (int i = warp; i < c.parts; i += 8) s += c.partial[i * c.N + n];
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && n < c.N) {
#pragma unroll
    for (int w = 1; w < 8; ++w) s += sums[w][lane];
    c.db[n] = s;
  }
}

// C from its partial sums: V columns of a row per thread, the parts added in
// order.  The blocks behind the first `blocks` join db's parts, where there are
// some (one launch less: 2 us of a layer's gradients).
template <int V>
__global__ void __launch_bounds__(256)
    linear_join_kernel(const float *__restrict__ partial, int splits, int64_t M, int64_t N,
                       int64_t ld, const LinearEpilogue e, unsigned blocks, const ColumnParts c) {
  begin_after_previous();
  if (blockIdx.x >= blocks) {
    join_columns(c, blockIdx.x - blocks);
    return;
  }
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

// Copies of 16-bit matrices with rows that TMA can read, all in one launch.  A
// thread takes 8 columns: single loads, all on their way at once, and one
// 16-byte store (the copy's rows are padded to 8 columns, with zeros).
struct Copies {
  struct One {
    const uint16_t *from;
    uint16_t *to;
    int64_t ld_from, ld_to, rows, cols;
  } m[3];
  int n;
};
__global__ void __launch_bounds__(256) pack_rows_kernel(const Copies c) {
  begin_after_previous();
  const Copies::One m = c.m[blockIdx.y];
  const int64_t per_row = m.ld_to / 8, groups = m.rows * per_row;
  for (int64_t g = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; g < groups;
       g += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t r = g / per_row, k = (g - r * per_row) * 8;
    const uint16_t *from = m.from + r * m.ld_from + k;
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = k + i < m.cols ? from[i] : 0;
    *reinterpret_cast<uint4 *>(m.to + r * m.ld_to + k) =
        make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
  }
}

// db[n] = sum_m dy[m, n].  A block takes 32 V columns and a part of the rows:
// lanes over the columns (V each), warps over the rows.  With one part it writes
// db, otherwise partial sums [part][N] that column_join_kernel adds in order.
template <int V>
__global__ void __launch_bounds__(256)
    column_sum_kernel(const uint16_t *__restrict__ dy, int64_t ld, int64_t M, int64_t N, int dtype,
                      int parts, float *__restrict__ out) {
  __shared__ float part[8][32 * V];
  begin_after_previous();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t col = (static_cast<int64_t>(blockIdx.x) * 32 + lane) * V;
  const int64_t from = M * blockIdx.y / parts, to = M * (blockIdx.y + 1) / parts;
  float s[V];
#pragma unroll
  for (int i = 0; i < V; ++i) s[i] = 0.f;
  if (col < N) {
#pragma unroll 4
    for (int64_t m = from + warp; m < to; m += 8) {
      float v[V];
      load_values<V>(dy, m * ld + col, dtype, v);
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] += v[i];
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) part[warp][i * 32 + lane] = s[i];
  __syncthreads();
  if (static_cast<int>(threadIdx.x) < 32 * V) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += part[w][threadIdx.x];
    const int64_t n = (static_cast<int64_t>(blockIdx.x) * 32 + lane) * V + warp;
    if (n < N) out[blockIdx.y * N + n] = t;
  }
}
__global__ void __launch_bounds__(256) column_join_kernel(const ColumnParts c) {
  begin_after_previous();
  join_columns(c, blockIdx.x);
}

// Whether TMA can read a matrix in place.
bool tma_readable(const void *p, int64_t ld) { return aligned(p, 16) && ld % 8 == 0; }

// --------------------------------------------------------------------------
// Up to 8 rows of x: the weights' one pass through the SMs sets the time, and a
// tile of 256 rows would be almost empty.  A warp takes kRowsW rows of W at a
// time, its lanes 8 consecutive terms each (V == 1: one, for rows that 16-byte
// loads cannot read), and the warps of a block first share out the summed
// dimension, so that even a small W has all its loads in flight at once.  Each
// block writes its outputs itself: no workspace and one launch.  us at 1, 4 and 8
// rows and the tensor cores' at 4 and 8: 1024 x 1536 2.9, 3.4, 5.5 and 8.3, 8.6;
// 4096 x 1024 4.7, 6.5, 10.5 and 7.5, 7.5; 1024 x 4096 3.7, 4.7, 8.0 and 9.4, 9.3;
// 128 x 1024 2.5, 3.2, 5.0 and 8.1, 8.3; 501 x 1003 2.7, 3.5, 4.7 and 10.0, 10.3;
// 16384 x 1024 10.4, 19.4, 29.3 and 12.6, 12.1.
constexpr int kSkinnyRows = 8;
constexpr int kRowsW = 4;

template <int MT, int V>
__global__ void __launch_bounds__(256)
    linear_skinny_kernel(const uint16_t *__restrict__ x, int64_t ldx,
                         const uint16_t *__restrict__ W, int64_t ldw, int M, int64_t N, int64_t K,
                         int warps_k, const LinearEpilogue e) {
  __shared__ float part[8][kRowsW * MT];
  begin_after_previous();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int wk = warp % warps_k, group = warp / warps_k;
  const int64_t n0 = (static_cast<int64_t>(blockIdx.x) * (8 / warps_k) + group) * kRowsW;
  float acc[kRowsW][MT];
#pragma unroll
  for (int r = 0; r < kRowsW; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[r][m] = 0.f;
  if (n0 < N) {
    // Rows past the last repeat it; what they give is not written.
    const uint16_t *w_row[kRowsW], *x_row[MT];
#pragma unroll
    for (int r = 0; r < kRowsW; ++r) w_row[r] = W + min(n0 + r, N - 1) * ldw;
#pragma unroll
    for (int m = 0; m < MT; ++m) x_row[m] = x + static_cast<int64_t>(min(m, M - 1)) * ldx;
#pragma unroll 2
    for (int64_t k = (static_cast<int64_t>(wk) * 32 + lane) * V; k < K; k += warps_k * 32 * V) {
      float w[kRowsW][V];
#pragma unroll
      for (int r = 0; r < kRowsW; ++r) load_values<V>(w_row[r], k, e.dtype, w[r]);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float v[V];
        load_values<V>(x_row[m], k, e.dtype, v);
#pragma unroll
        for (int r = 0; r < kRowsW; ++r)
#pragma unroll
          for (int i = 0; i < V; ++i) acc[r][m] = fmaf(w[r][i], v[i], acc[r][m]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRowsW; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float s = acc[r][m];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == 0) part[warp][r * MT + m] = s;
    }
  __syncthreads();
  if (wk == 0 && lane < kRowsW * MT) {
    float v[1] = {0.f};
    for (int i = 0; i < warps_k; ++i) v[0] += part[warp + i][lane];
    const int64_t n = n0 + lane / MT;
    const int m = lane % MT;
    if (n < N && m < M) {
      const float bias[1] = {e.bias ? e.bias[n] : 0.f};
      linear_finish<1>(e, v, bias, m, n);
    }
  }
}

// How the kernel divides a product: warps over the summed dimension, blocks, and
// the steps of a warp along it.
struct SkinnyShape {
  bool vec;
  int warps_k;
  int64_t blocks, steps;
};
SkinnyShape skinny_shape(const LinearFwd &a) {
  SkinnyShape s;
  s.vec = a.K % 8 == 0 && a.ldx % 8 == 0 && a.ldw % 8 == 0 && aligned(a.x, 16) && aligned(a.W, 16);
  const int64_t deep = 32 * (s.vec ? 8 : 1);
  s.warps_k = 1;
  while (s.warps_k < 8 && s.warps_k * deep < a.K) s.warps_k *= 2;
  const int64_t rows = static_cast<int64_t>(8 / s.warps_k) * kRowsW;
  s.blocks = (a.N + rows - 1) / rows;
  s.steps = (a.K + s.warps_k * deep - 1) / (s.warps_k * deep);
  return s;
}

// Whether a product of few rows goes through the skinny kernel: one row always,
// up to 8 where that is estimated to take no longer than the tensor cores (with
// their copies of rows that TMA cannot read).  Estimated in SM cycles from the
// rounds of blocks (3 of 1 or 2 rows of x to an SM, 2 of more) and their steps,
// of which those of single loads are a tenth; fitted to 43 weights of 64 x 65536
// to 65536 x 512 at 2 to 8 rows: the choice takes 0.8 % more than the better of
// both on average, the skinny kernel for all of them 14 %.
bool takes_skinny(const LinearFwd &a) {
  if (a.M > kSkinnyRows || a.M <= 1) return a.M <= 1;
  struct Cost {
    int per_sm, start, round, step;
  };
  const Cost c = a.M == 2  ? Cost{3, 2850, 2470, 1615}
                 : a.M <= 4 ? Cost{2, 2280, 3135, 1805}
                            : Cost{2, 3800, 3800, 3800};
  const SkinnyShape s = skinny_shape(a);
  const int64_t at_once = static_cast<int64_t>(c.per_sm) * a.num_sms;
  const double rounds = static_cast<double>((s.blocks + at_once - 1) / at_once);
  const double time = c.start + rounds * (c.round + c.step * (s.vec ? 1.0 : 0.1) * s.steps);
  // (No plan takes less than one tile's products, or one step of them and a join;
  // so the smallest calls need none.)
  const double whole = 8700 + item_time(128, (a.K + 63) / 64),
               split = 8700 + item_time(128, 1) + join_time(2, 1, 1);
  if (time <= (whole < split ? whole : split)) return true;
  const bool copies = !tma_readable(a.x, a.ldx) || !tma_readable(a.W, a.ldw);
  return time <= plan_gemm(a.M, a.N, a.K, a.num_sms / 2).time + (copies ? 5000 : 0);
}

template <int MT>
cudaError_t launch_skinny(const LinearFwd &a) {
  const SkinnyShape s = skinny_shape(a);
  auto *kernel = s.vec ? linear_skinny_kernel<MT, 8> : linear_skinny_kernel<MT, 1>;
  return launch_after_previous(kernel, static_cast<unsigned>(s.blocks), 256, 0, a.stream,
                               static_cast<const uint16_t *>(a.x), a.ldx,
                               static_cast<const uint16_t *>(a.W), a.ldw, static_cast<int>(a.M),
                               a.N, a.K, s.warps_k, a.epi);
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
// Notes the copy that an operand needs, and makes those noted.
void note(Copies &c, const Packed &k, const void *p, int64_t ld) {
  if (!k.copy) return;
  c.m[c.n++] = {static_cast<const uint16_t *>(p),
                static_cast<uint16_t *>(const_cast<void *>(k.op.p)), ld, k.op.ld, k.op.rows,
                k.op.cols};
}
cudaError_t make(const Copies &c, int num_sms, cudaStream_t s) {
  if (c.n == 0) return cudaSuccess;
  int64_t blocks = 0;
  for (int i = 0; i < c.n; ++i) {
    const int64_t b = (c.m[i].rows * (c.m[i].ld_to / 8) + 255) / 256;
    blocks = b > blocks ? b : blocks;
  }
  if (blocks > 16 * num_sms) blocks = 16 * num_sms;
  return launch_after_previous(pack_rows_kernel, dim3(static_cast<unsigned>(blocks), c.n), 256, 0, s,
                               c);
}

int64_t partial_bytes(const GemmPlan &plan, int64_t M, int64_t N) {
  return plan.splits > 1 ? plan.splits * M * partial_ld(N) * 4 : 0;
}

// The joining of a product's parts, and of db's.
cudaError_t join(const Gemm &g, const ColumnParts &c) {
  if (g.plan.splits == 1) return cudaSuccess;
  const int v = g.epi.vec8 ? 8 : 1;
  const unsigned blocks =  // at most 2^38 / 256
      static_cast<unsigned>((g.M * ((g.N + v - 1) / v) + 255) / 256);
  return launch_after_previous(v == 8 ? linear_join_kernel<8> : linear_join_kernel<1>,
                               blocks + c.blocks(), 256, 0, g.stream, g.partial, g.plan.splits, g.M,
                               g.N, partial_ld(g.N), g.epi, blocks, c);
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

// In how many parts of its rows dy is summed: enough blocks for every SM, at
// least 64 rows each.
int column_parts(int64_t M, int64_t N, bool vec, int num_sms) {
  const int64_t blocks = (N + (vec ? 255 : 31)) / (vec ? 256 : 32);
  int64_t parts = (4 * num_sms + blocks - 1) / blocks;
  if (parts > (M + 63) / 64) parts = (M + 63) / 64;
  return static_cast<int>(parts < 1 ? 1 : parts);
}

struct BwdLayout {
  Packed dy, x, W;
  GemmPlan dx_plan, dW_plan;
  PairPlan pair;
  bool paired;
  float *partial;     // of dx, then of dW
  float *db_partial;
  int db_parts;
  bool db_vec;
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
  // In one launch where that is estimated to be faster (plan_pair).  Of 110 shapes
  // measured both ways (8 to 16384 rows, 64 to 8192 columns) that takes 0.9 % more
  // than the better one on average.  On the wrong side by most, us in two launches
  // and in one: 1000 x 3000 x 600 24.4, 26.1 (taken in one); 1264 x 5824 x 240 28.9,
  // 23.5 and 120 x 3840 x 1048 25.1, 21.0 (taken in two).
  if (a.dx.out && a.dW.out) {
    l.pair = plan_pair(a.M, a.N, a.K, a.num_sms / 2);
    l.paired = l.pair.time < l.dx_plan.time + l.dW_plan.time;
    const int64_t b = l.paired ? partial_bytes({l.pair.bn, l.pair.splits, 0}, a.N, a.K) : 0;
    partial = b > partial ? b : partial;
  }
  if (a.db) {
    l.db_vec = a.N % 8 == 0 && tma_readable(a.dy, a.lddy);
    l.db_parts = column_parts(a.M, a.N, l.db_vec, a.num_sms);
    l.db_partial = static_cast<float *>(ws.take(l.db_parts > 1 ? l.db_parts * a.N * 4 : 0));
  }
  l.partial = static_cast<float *>(ws.take(partial));
  return l;
}

}  // namespace

cudaError_t linear_fwd_workspace(const LinearFwd &a, int64_t *bytes) {
  Workspace ws{nullptr};
  if (!takes_skinny(a)) fwd_layout(a, ws);
  *bytes = ws.used;
  return cudaSuccess;
}

cudaError_t launch_linear_fwd(const LinearFwd &a) {
  if (takes_skinny(a))
    return a.M == 1   ? launch_skinny<1>(a)
           : a.M == 2 ? launch_skinny<2>(a)
           : a.M <= 4 ? launch_skinny<4>(a)
                      : launch_skinny<8>(a);
  Workspace ws{static_cast<char *>(a.workspace)};
  const FwdLayout l = fwd_layout(a, ws);
  Copies copies{};
  note(copies, l.x, a.x, a.ldx);
  note(copies, l.W, a.W, a.ldw);
  cudaError_t e = make(copies, a.num_sms, a.stream);
  if (e != cudaSuccess) return e;
  const Gemm g{l.x.op, l.W.op, false, false, a.M, a.N, a.K, l.plan, l.partial, a.epi,
         a.num_sms, a.err, a.encode, a.stream};
  e = launch_gemm(g);
  return e == cudaSuccess ? join(g, ColumnParts{}) : e;
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
  Copies copies{};
  note(copies, l.dy, a.dy, a.lddy);
  note(copies, l.W, a.W, a.ldw);
  note(copies, l.x, a.x, a.ldx);
  cudaError_t e = make(copies, a.num_sms, a.stream);
  Gemm dx{l.dy.op, l.W.op, false, true, a.M, a.K, a.N, l.dx_plan, l.partial, a.dx,
          a.num_sms, a.err, a.encode, a.stream};
  Gemm dW{l.dy.op, l.x.op, true, true, a.N, a.K, a.M, l.dW_plan, l.partial, a.dW,
          a.num_sms, a.err, a.encode, a.stream};
  bool done = false;
  if (e == cudaSuccess && l.paired) {
    Gemm one = dx, two = dW;
    one.plan = {l.pair.bn, 1, 0}, two.plan = {l.pair.bn, l.pair.splits, 0};
    e = launch_gemm_pair(two, one, l.pair.turns, &done);
    if (done) dW.plan = two.plan;
  }
  if (e == cudaSuccess && a.dx.out && !done) {
    e = launch_gemm(dx);
    if (e == cudaSuccess) e = join(dx, ColumnParts{});
  }
  if (e == cudaSuccess && a.dW.out && !done) e = launch_gemm(dW);
  // db's parts behind the products, which leave dy in L2 (in front of them 0.6 to
  // 1.6 us slower with cold operands), and joined in one launch with dW's.
  ColumnParts c{};
  if (e == cudaSuccess && a.db) {
    const int cols = l.db_vec ? 256 : 32;
    const dim3 grid(static_cast<unsigned>((a.N + cols - 1) / cols), l.db_parts);
    e = launch_after_previous(l.db_vec ? column_sum_kernel<8> : column_sum_kernel<1>, grid, 256, 0,
                              a.stream, static_cast<const uint16_t *>(a.dy), a.lddy, a.M, a.N,
                              a.dx.dtype, l.db_parts, l.db_parts > 1 ? l.db_partial : a.db);
    if (l.db_parts > 1) c = {l.db_partial, l.db_parts, a.N, a.db};
  }
  if (e != cudaSuccess) return e;
  if (a.dW.out && dW.plan.splits > 1) return join(dW, c);
  return c.db ? launch_after_previous(column_join_kernel, c.blocks(), 256, 0, a.stream, c) : e;
}

}  // namespace ag
