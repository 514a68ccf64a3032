// grad_clip.cu -- the global 2-norm of many gradient tensors and their scaling
// in place (ag_grad_clip).
//
//   norm = sqrt(sum g^2),  c = min(1, max_norm / (norm + eps)),  g = c g
//
// Bound by memory: one read for the norm, and where c < 1 another read and a
// write.  The tensors are cut into chunks; a fixed grid of blocks takes them
// in turn, so a partial sum belongs to a block and the order of every
// addition is fixed.  Squares and sums are in 64 bits: a float32 square of a
// large gradient overflows and of a small one vanishes; the conversions and the
// 64-bit products keep up with memory.  Measured: 98 million float32 values in
// 126 tensors 70 us for the norm alone (5.6 TB/s) and 223 us with the scaling
// (5.3 TB/s over its three passes; 392 MB do not stay in L2 between them); 14
// tensors of 98 thousand bf16 values 7.5 us, which is two launches (one cluster
// of 8 blocks doing both in one launch took 7.4 us, and 10 us from 131 thousand
// float32 values on, against 8.5).
#include <cmath>

#include "ag_internal.h"
#include "launch.cuh"
#include "linear_epilogue.cuh"

namespace ag {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 16384;         // elements
// Tensors per launch: the list travels as a kernel argument.  A list of 32
// (0.7 KB) takes the launching thread 5.9 us for the two kernels, one of 512
// (10.8 KB) 13.9 us.
constexpr int kFewTensors = 32, kMaxTensors = 512;
constexpr int kBlocksPerSm = 4;

template <int MOST>
struct TensorList {
  void *ptr[MOST];
  int64_t count[MOST];
  uint32_t first[MOST + 1];           // first chunk of each tensor
  uint8_t dtype[MOST];
  int n;
};

struct Chunk {
  void *base;
  int64_t at;
  int len, dtype;
};
template <int MOST>
__device__ __forceinline__ Chunk chunk_of(const TensorList<MOST> &list, uint32_t c) {
  int lo = 0, hi = list.n;            // first[lo] <= c < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (list.first[mid] <= c) lo = mid;
    else hi = mid;
  }
  Chunk k;
  k.base = list.ptr[lo];
  k.at = static_cast<int64_t>(c - list.first[lo]) * kChunk;
  const int64_t left = list.count[lo] - k.at;
  k.len = static_cast<int>(left < kChunk ? left : kChunk);
  k.dtype = list.dtype[lo];
  return k;
}

// Elements of the chunk before the first whose address is 16-byte aligned.
__device__ __forceinline__ int head_of(const Chunk &k) {
  const int size = k.dtype == AG_F32 ? 4 : 2;
  const uintptr_t p = reinterpret_cast<uintptr_t>(k.base) + static_cast<uintptr_t>(k.at) * size;
  const int h = static_cast<int>((16 - (p & 15)) & 15) / size;
  return h < k.len ? h : k.len;
}

__device__ __forceinline__ double block_sum(double s) {
  __shared__ double part[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  __syncthreads();
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = s;
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) t += part[i];
  return t;
}

template <int MOST>
__global__ void __launch_bounds__(kThreads)
    square_sum_kernel(const __grid_constant__ TensorList<MOST> list, double *partial) {
  begin_after_previous();
  double s = 0.0;
  for (uint32_t c = blockIdx.x; c < list.first[list.n]; c += gridDim.x) {
    const Chunk k = chunk_of(list, c);
    const int head = head_of(k), body = (k.len - head) / 8;
    for (int i = threadIdx.x; i < body; i += kThreads) {
      float v[8];
      load_values<8>(k.base, k.at + head + 8 * static_cast<int64_t>(i), k.dtype, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) s = fma(static_cast<double>(v[j]), static_cast<double>(v[j]), s);
    }
    const int rest = k.len - 8 * body;  // the head and the tail, one by one
    if (static_cast<int>(threadIdx.x) < rest) {
      const int i = static_cast<int>(threadIdx.x) < head ? threadIdx.x : threadIdx.x + 8 * body;
      float v[1];
      load_values<1>(k.base, k.at + i, k.dtype, v);
      s = fma(static_cast<double>(v[0]), static_cast<double>(v[0]), s);
    }
  }
  s = block_sum(s);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// The sum of `slots` partials, the same in every block and thread.
__device__ __forceinline__ double total_of(const double *partial, int slots) {
  double s = 0.0;
  for (int i = threadIdx.x; i < slots; i += kThreads) s += partial[i];
  return block_sum(s);
}

__global__ void __launch_bounds__(kThreads)
    total_kernel(const double *partial, int slots, double *total) {
  begin_after_previous();
  const double t = total_of(partial, slots);
  if (threadIdx.x == 0) *total = t;
}

template <int MOST>
__global__ void __launch_bounds__(kThreads)
    scale_kernel(const __grid_constant__ TensorList<MOST> list, const double *partial, int slots,
                 float max_norm, float eps, float *norm_out) {
  begin_after_previous();
  const double norm = sqrt(total_of(partial, slots));
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = static_cast<float>(norm);
  if (max_norm == INFINITY || norm == 0.0) return;  // (zeros stay zeros, also with eps == 0)
  const double ratio = static_cast<double>(max_norm) / (norm + static_cast<double>(eps));
  // Written so that a NaN stays a NaN.
  const float c = ratio >= 1.0 ? 1.f : static_cast<float>(ratio);
  if (c == 1.f) return;
  // A factor below the normal numbers of 32 bits (gradients near their largest)
  // would keep only some of its digits: it is applied in two steps.
  const bool tiny = ratio < 0x1p-126;
  const float once = tiny ? static_cast<float>(ratio * 0x1p120) : c, again = tiny ? 0x1p-120f : 1.f;
  // From the end: what the first pass read last is still in L2.
  const uint32_t chunks = list.first[list.n];
  for (uint32_t q = blockIdx.x; q < chunks; q += gridDim.x) {
    const Chunk k = chunk_of(list, chunks - 1 - q);
    const int head = head_of(k), body = (k.len - head) / 8;
    for (int i = threadIdx.x; i < body; i += kThreads) {
      float v[8];
      const int64_t at = k.at + head + 8 * static_cast<int64_t>(i);
      load_values<8>(k.base, at, k.dtype, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = v[j] * once * again;
      store_values<8>(k.base, at, k.dtype, v);
    }
    const int rest = k.len - 8 * body;
    if (static_cast<int>(threadIdx.x) < rest) {
      const int i = static_cast<int>(threadIdx.x) < head ? threadIdx.x : threadIdx.x + 8 * body;
      float v[1];
      load_values<1>(k.base, k.at + i, k.dtype, v);
      v[0] = v[0] * once * again;
      store_values<1>(k.base, k.at + i, k.dtype, v);
    }
  }
}

// Takes tensors [from, n) that are not empty into `list` up to its capacity;
// returns the index of the next one that is not empty.  The entry point's limits (2^42 elements, 2^20
// tensors) keep the chunks of a launch below 2^29.
template <int MOST>
int64_t fill(TensorList<MOST> &list, void *const *grads, const int64_t *counts, const int *dtypes,
             int64_t from, int64_t n) {
  list.n = 0;
  list.first[0] = 0;
  int64_t chunks = 0;
  int64_t i = from;
  for (; i < n; ++i) {
    if (counts[i] == 0) continue;
    if (list.n == MOST) break;
    list.ptr[list.n] = grads[i];
    list.count[list.n] = counts[i];
    list.dtype[list.n] = static_cast<uint8_t>(dtypes[i]);
    chunks += (counts[i] + kChunk - 1) / kChunk;
    list.first[++list.n] = static_cast<uint32_t>(chunks);
  }
  return i;
}

}  // namespace

// One partial per block and launch, and the total of several launches.
int64_t grad_clip_workspace(int64_t n, int num_sms) {
  const int64_t launches = n <= kMaxTensors ? 1 : (n + kMaxTensors - 1) / kMaxTensors;
  return (launches * num_sms * kBlocksPerSm + 1) * static_cast<int64_t>(sizeof(double));
}

namespace {

template <int MOST>
cudaError_t clip(void *const *grads, const int64_t *counts, const int *dtypes, int64_t n,
                 float max_norm, float eps, float *norm_out, double *workspace, int most,
                 cudaStream_t stream) {
  TensorList<MOST> list;
  int slots = 0, launches = 0;
  for (int64_t i = 0; i < n;) {
    i = fill(list, grads, counts, dtypes, i, n);
    if (list.n == 0) break;  // (nothing but empty tensors)
    const unsigned chunks = list.first[list.n];
    const int blocks = chunks < static_cast<unsigned>(most) ? static_cast<int>(chunks) : most;
    const cudaError_t e = launch_after_previous(square_sum_kernel<MOST>, blocks, kThreads, 0, stream,
                                                list, workspace + slots);
    if (e != cudaSuccess) return e;
    slots += blocks;
    ++launches;
  }
  const double *sums = workspace;
  if (launches > 1) {
    double *total = workspace + slots;
    const cudaError_t e =
        launch_after_previous(total_kernel, 1, kThreads, 0, stream, workspace, slots, total);
    if (e != cudaSuccess) return e;
    sums = total;
    slots = 1;
  }
  int64_t i = 0;
  bool first = true;
  do {
    if (launches != 1) i = fill(list, grads, counts, dtypes, i, n);
    else i = n;  // the list still holds them all
    const unsigned chunks = list.first[list.n];
    int blocks = chunks < static_cast<unsigned>(most) ? static_cast<int>(chunks) : most;
    if (blocks == 0 || std::isinf(max_norm)) blocks = 1;
    const cudaError_t e =
        launch_after_previous(scale_kernel<MOST>, blocks, kThreads, 0, stream, list, sums, slots,
                              max_norm, eps, first ? norm_out : nullptr);
    if (e != cudaSuccess) return e;
    first = false;
  } while (i < n && !std::isinf(max_norm));
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_grad_clip(void *const *grads, const int64_t *counts, const int *dtypes,
                             int64_t n, float max_norm, float eps, float *norm_out,
                             double *workspace, int num_sms, cudaStream_t stream) {
  const int most = num_sms * kBlocksPerSm;
  return n <= kFewTensors ? clip<kFewTensors>(grads, counts, dtypes, n, max_norm, eps, norm_out,
                                              workspace, most, stream)
                          : clip<kMaxTensors>(grads, counts, dtypes, n, max_norm, eps, norm_out,
                                              workspace, most, stream);
}

}  // namespace ag
