// qk_norm_rope.cu -- per-head norm of queries and keys with the rotation by
// position, from the projections' layout [B, L, H, D] to the attention's
// [B, H, L, D], and its gradients (ag_qk_norm_rope_fwd, ag_qk_norm_rope_bwd).
//
//   n = (x - mean) r,  v = n w + b,  out = R(position) v
//   g = R^T dout,  dw = sum g n,  db = sum g,  d = g w,
//   dx = r (d - n mean(d n) - mean d)
//
// Bound by memory: every element is read once and written once (the backward
// reads x and dout and writes dx).  A block takes kPos positions with all
// their heads, so each position's angles are formed once for all heads.
#include "ag_internal.h"
#include "linear_epilogue.cuh"

namespace ag {
namespace {

constexpr int kPos = 4;        // positions per block and turn
constexpr int kThreads = 256;  // 8 warps
constexpr int kWarps = kThreads / 32;

// cos and sin of position * frequency.  The product and its reduction to one
// turn are in 64 bits (two-part 2 pi), so the phase of a far position is as
// exact as the frequency; the reduced angle then goes through float32.
__device__ __forceinline__ float2 turn(long long pos, double freq) {
  const double a = static_cast<double>(pos) * freq;
  const double n = rint(a * 0.15915494309189535);
  double r = fma(n, -6.283185307179586, a);
  r = fma(n, -2.4492935982947064e-16, r);
  float s, c;
  sincospif(static_cast<float>(r * 0.3183098861837907), &s, &c);
  return make_float2(c, s);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float load_one(const void *p, int64_t at, int dtype) {
  float v[1];
  load_values<1>(p, at, dtype, v);
  return v[0];
}
__device__ __forceinline__ void store_one(void *p, int64_t at, int dtype, float x) {
  const float v[1] = {x};
  store_values<1>(p, at, dtype, v);
}

// The pair member of element i and whether i is the second of its pair.
struct Pair {
  int other, angle;
  bool second;
};
__device__ __forceinline__ Pair pair_of(int i, int R, int rope) {
  Pair p;
  if (rope == AG_ROPE_HALVES) {
    const int h = R >> 1;
    p.second = i >= h;
    p.other = p.second ? i - h : i + h;
    p.angle = p.second ? i - h : i;
  } else {
    p.second = i & 1;
    p.other = i ^ 1;
    p.angle = i >> 1;
  }
  return p;
}

// mean and 1 / sqrt(mean square + eps) of a row held in shared memory.
__device__ __forceinline__ void row_stats(const float *row, int D, int norm, float eps, int lane,
                                          float &mean, float &r) {
  mean = 0.f, r = 1.f;
  if (norm == AG_NORM_NONE) return;
  if (norm == AG_NORM_LAYER) {
    float s = 0.f;
    for (int i = lane; i < D; i += 32) s += row[i];
    mean = warp_sum(s) / D;
  }
  float q = 0.f;
  for (int i = lane; i < D; i += 32) q = fmaf(row[i] - mean, row[i] - mean, q);
  r = 1.f / sqrtf(warp_sum(q) / D + eps);
}

// One warp per (position, head) row, any D and any strides.
__global__ void __launch_bounds__(kThreads) qk_fwd_kernel(const QkArgs a) {
  extern __shared__ float smem[];
  const int half = a.R >> 1, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  float2 *cs = reinterpret_cast<float2 *>(smem);
  float *row = smem + 2 * kPos * half + warp * a.D;
  const int64_t p0 = static_cast<int64_t>(blockIdx.x) * kPos;
  const int np = static_cast<int>(min(static_cast<int64_t>(kPos), a.positions_total - p0));
  for (int i = threadIdx.x; i < np * half; i += kThreads) {
    const int64_t b = (p0 + i / half) / a.L, l = (p0 + i / half) % a.L;
    cs[i] = turn(a.positions ? a.positions[b * a.pos_sb + l] : l, a.inv_freq[i % half]);
  }
  __syncthreads();
  const int heads = a.side[0].H + a.side[1].H;
  for (int t = warp; t < np * heads; t += kWarps) {
    const int which = t % heads >= a.side[0].H;
    const QkSide &s = a.side[which];
    const int h = t % heads - (which ? a.side[0].H : 0), p = t / heads;
    const int64_t b = (p0 + p) / a.L, l = (p0 + p) % a.L;
    const int64_t at = b * s.sb + l * s.sl + h * s.sh;
    for (int i = lane; i < a.D; i += 32) row[i] = load_one(s.x, at + i, a.x_dtype);
    float mean, r;
    row_stats(row, a.D, a.norm, a.eps, lane, mean, r);
    for (int i = lane; i < a.D; i += 32) {
      float v = (row[i] - mean) * r;
      if (s.w) v *= s.w[i];
      if (s.b) v += s.b[i];
      row[i] = v;
    }
    __syncwarp();
    const int64_t to = ((b * s.H + h) * a.L + l) * a.D;
    for (int i = lane; i < a.D; i += 32) {
      float v = row[i];
      if (i < a.R) {
        const Pair q = pair_of(i, a.R, a.rope);
        const float2 c = cs[p * half + q.angle];
        v = fmaf(v, c.x, q.second ? row[q.other] * c.y : -row[q.other] * c.y);
      }
      store_one(s.out, to + i, a.o_dtype, v);
    }
    __syncwarp();
  }
}

// Backward: the same rows.  Each warp adds its rows' parameter gradients to
// its own part of shared memory (element i always by lane i % 32: no atomics),
// the block then adds its warps' in order and writes one partial per block;
// qk_params_kernel adds those.
__global__ void __launch_bounds__(kThreads) qk_bwd_kernel(const QkArgs a, int warps) {
  extern __shared__ float smem[];
  const int half = a.R >> 1, warp = threadIdx.x / 32, lane = threadIdx.x % 32, D = a.D;
  float2 *cs = reinterpret_cast<float2 *>(smem);
  float *row = smem + 2 * kPos * half + warp * 2 * D, *grad = row + D;
  float *sums = smem + 2 * kPos * half + warps * 2 * D;  // [warps][2 sides][w, b][D]
  float *own = sums + warp * 4 * D;
  for (int i = lane; i < 4 * D; i += 32) own[i] = 0.f;
  const int heads = a.side[0].H + a.side[1].H;
  for (int64_t p0 = static_cast<int64_t>(blockIdx.x) * kPos; p0 < a.positions_total;
       p0 += static_cast<int64_t>(gridDim.x) * kPos) {
    const int np = static_cast<int>(min(static_cast<int64_t>(kPos), a.positions_total - p0));
    __syncthreads();
    for (int i = threadIdx.x; i < np * half; i += blockDim.x) {
      const int64_t b = (p0 + i / half) / a.L, l = (p0 + i / half) % a.L;
      cs[i] = turn(a.positions ? a.positions[b * a.pos_sb + l] : l, a.inv_freq[i % half]);
    }
    __syncthreads();
    for (int t = warp; t < np * heads; t += warps) {
      const int which = t % heads >= a.side[0].H;
      const QkSide &s = a.side[which];
      const int h = t % heads - (which ? a.side[0].H : 0), p = t / heads;
      const int64_t b = (p0 + p) / a.L, l = (p0 + p) % a.L;
      const int64_t at = b * s.sb + l * s.sl + h * s.sh;
      const int64_t from = ((b * s.H + h) * a.L + l) * D;
      for (int i = lane; i < D; i += 32) {
        row[i] = load_one(s.x, at + i, a.x_dtype);
        grad[i] = load_one(s.g, from + i, a.o_dtype);
      }
      float mean, r;
      row_stats(row, D, a.norm, a.eps, lane, mean, r);
      __syncwarp();
      float along = 0.f, total = 0.f;
      for (int i = lane; i < D; i += 32) {
        float g = grad[i];
        if (i < a.R) {
          const Pair q = pair_of(i, a.R, a.rope);
          const float2 c = cs[p * half + q.angle];
          g = fmaf(g, c.x, q.second ? -grad[q.other] * c.y : grad[q.other] * c.y);
        }
        const float n = (row[i] - mean) * r;
        own[which * 2 * D + i] += g * n;
        own[which * 2 * D + D + i] += g;
        const float d = s.w ? g * s.w[i] : g;
        along = fmaf(d, n, along);
        total += d;
      }
      along = a.norm == AG_NORM_NONE ? 0.f : warp_sum(along) / D;
      total = a.norm == AG_NORM_LAYER ? warp_sum(total) / D : 0.f;
      const int64_t to = b * s.dxb + l * s.dxl + h * s.dxh;
      for (int i = lane; i < D; i += 32) {
        float g = grad[i];
        if (i < a.R) {
          const Pair q = pair_of(i, a.R, a.rope);
          const float2 c = cs[p * half + q.angle];
          g = fmaf(g, c.x, q.second ? -grad[q.other] * c.y : grad[q.other] * c.y);
        }
        const float n = (row[i] - mean) * r, d = s.w ? g * s.w[i] : g;
        store_one(s.dx, to + i, a.x_dtype, r * (d - n * along - total));
      }
      __syncwarp();
    }
  }
  __syncthreads();
  if (a.partial)
    for (int i = threadIdx.x; i < 4 * D; i += blockDim.x) {
      float t = 0.f;
      for (int w = 0; w < warps; ++w) t += sums[w * 4 * D + i];
      a.partial[static_cast<int64_t>(blockIdx.x) * 4 * D + i] = t;
    }
}

// The parameter gradients: sums of the blocks' partials [blocks][4][D], 32
// columns per block, 8 lanes over the partials, in 64 bits and a fixed order.
__global__ void __launch_bounds__(256)
    qk_params_kernel(const float *partial, int blocks, int D, float *qw, float *qb, float *kw,
                     float *kb) {
  __shared__ double part[8][32];
  const int c = threadIdx.x % 32, r = threadIdx.x / 32, n = blockIdx.x * 32 + c;
  double t = 0.0;
  if (n < 4 * D)
    for (int i = r; i < blocks; i += 8) t += partial[static_cast<int64_t>(i) * 4 * D + n];
  part[r][c] = t;
  __syncthreads();
  if (r != 0 || n >= 4 * D) return;
  for (int i = 1; i < 8; ++i) t += part[i][c];
  float *to = n < 2 * D ? (n < D ? qw : qb) : (n < 3 * D ? kw : kb);
  if (to) to[n % D] = static_cast<float>(t);
}

int bwd_warps(int D) { return D <= 512 ? 8 : 4; }
int bwd_blocks(int64_t total, int num_sms) {
  const int64_t turns = (total + kPos - 1) / kPos;
  return static_cast<int>(turns < 4 * num_sms ? turns : 4 * num_sms);
}

cudaError_t allow_smem(const void *kernel, size_t bytes) {
  return bytes <= 48 * 1024 ? cudaSuccess
                            : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(bytes));
}

}  // namespace

int64_t qk_bwd_workspace(int64_t positions_total, int64_t D, int num_sms) {
  return static_cast<int64_t>(bwd_blocks(positions_total, num_sms)) * 4 * D * 4;
}

cudaError_t launch_qk_fwd(const QkArgs &a, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  const size_t smem = (static_cast<size_t>(kPos) * a.R + kWarps * static_cast<size_t>(a.D)) * 4;
  cudaError_t e = allow_smem(reinterpret_cast<const void *>(qk_fwd_kernel), smem);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (a.positions_total + kPos - 1) / kPos;
  qk_fwd_kernel<<<static_cast<unsigned>(blocks), kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_qk_bwd(const QkArgs &a, int num_sms, cudaStream_t stream) {
  const int warps = bwd_warps(a.D), blocks = bwd_blocks(a.positions_total, num_sms);
  const size_t smem = (static_cast<size_t>(kPos) * a.R + warps * 6 * static_cast<size_t>(a.D)) * 4;
  cudaError_t e = allow_smem(reinterpret_cast<const void *>(qk_bwd_kernel), smem);
  if (e != cudaSuccess) return e;
  qk_bwd_kernel<<<blocks, warps * 32, smem, stream>>>(a, warps);
  e = cudaGetLastError();
  if (e != cudaSuccess || !a.partial) return e;
  qk_params_kernel<<<(4 * a.D + 31) / 32, 256, 0, stream>>>(
      a.partial, blocks, a.D, a.side[0].dw, a.side[0].db, a.side[1].dw, a.side[1].db);
  return cudaGetLastError();
}

}  // namespace ag
