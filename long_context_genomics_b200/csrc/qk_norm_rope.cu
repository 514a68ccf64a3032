// qk_norm_rope.cu -- per-head norm of queries and keys with the rotation by
// position, from the projections' layout [B, L, H, D] to the attention's
// [B, H, L, D], and its gradients (ag_qk_norm_rope_fwd, ag_qk_norm_rope_bwd).
//
//   n = (x - mean) r,  v = n w + b,  out = R(position) v
//   g = R^T dout,  dw = sum g n,  db = sum g,  d = g w,
//   dx = r (d - n mean(d n) - mean d)
//
// Bound by memory: every element is read once and written once (the backward
// reads x and dout and writes dx).
//
// Rows kernels (heads of a multiple of 8 up to 256 elements, at addresses that
// 4 elements' loads can take): a warp takes one position with all its heads, so
// that the position's angles are formed once for them, and no other warp waits
// for it.  A row lies in D / 8 lanes, eight elements each in two quads; where
// halves are rotated, a lane's quads are 4 elements of the first half and their
// partners in the second, so no lane needs another's values but for the norm's
// sums.  All of a position's rows are loaded before any is worked on (the
// forward takes four, the backward two row steps at a time): that many bytes in
// flight is what the memory's rate asks for.
//
// General kernels: one warp per row through shared memory, any size or stride.
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

// --------------------------------------------------------------------------
// Rows kernels.

// A lane's eight elements of a row, two quads at a and b, as loaded (WIDE:
// float32) and as numbers.  Loading and widening are apart so that nothing
// waits for a load before all of them have been issued.
template <bool WIDE>
struct Raw;
template <>
struct Raw<true> {
  float4 a, b;
};
template <>
struct Raw<false> {
  uint2 a, b;
};
struct Eight {
  float v[8];
};

template <bool WIDE>
__device__ __forceinline__ Raw<WIDE> load8(const void *p, int64_t row, int a, int b) {
  if constexpr (WIDE) {
    const float *q = static_cast<const float *>(p) + row;
    return {*reinterpret_cast<const float4 *>(q + a), *reinterpret_cast<const float4 *>(q + b)};
  } else {
    const uint16_t *q = static_cast<const uint16_t *>(p) + row;
    return {*reinterpret_cast<const uint2 *>(q + a), *reinterpret_cast<const uint2 *>(q + b)};
  }
}
__device__ __forceinline__ float2 widen2(uint32_t w, bool bf16) {
  if (bf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <bool WIDE>
__device__ __forceinline__ Eight widen(const Raw<WIDE> &r, bool bf16) {
  if constexpr (WIDE) {
    return {{r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w}};
  } else {
    const float2 p = widen2(r.a.x, bf16), q = widen2(r.a.y, bf16), s = widen2(r.b.x, bf16),
                 t = widen2(r.b.y, bf16);
    return {{p.x, p.y, q.x, q.y, s.x, s.y, t.x, t.y}};
  }
}
__device__ __forceinline__ uint32_t narrow2(float x, float y, bool bf16) {
  if (bf16) return pack_bf16x2(x, y);
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t *>(&h);
}
template <bool WIDE>
__device__ __forceinline__ void store8(void *p, int64_t row, int a, int b, const Eight &e, bool bf16) {
  const float *v = e.v;
  if constexpr (WIDE) {
    float *q = static_cast<float *>(p) + row;
    *reinterpret_cast<float4 *>(q + a) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(q + b) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint16_t *q = static_cast<uint16_t *>(p) + row;
    *reinterpret_cast<uint2 *>(q + a) =
        make_uint2(narrow2(v[0], v[1], bf16), narrow2(v[2], v[3], bf16));
    *reinterpret_cast<uint2 *>(q + b) =
        make_uint2(narrow2(v[4], v[5], bf16), narrow2(v[6], v[7], bf16));
  }
}
// Sum over the LPR lanes of a row.
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ Eight param8(const float *p, int a, int b, float otherwise) {
  Eight e;
#pragma unroll
  for (int i = 0; i < 8; ++i) e.v[i] = p ? __ldg(p + (i < 4 ? a + i : b + i - 4)) : otherwise;
  return e;
}

// Where a lane's quads lie, and whether they turn.
struct Lane {
  int a, b;
  bool in, turns;
};
template <int LPR>
__device__ __forceinline__ Lane lane_of(int lane, int D, int R, int rope) {
  const int l = lane % LPR;
  Lane t;
  t.in = 8 * l < D;
  t.turns = 8 * l < R;
  if (rope == AG_ROPE_HALVES && t.turns)
    t.a = 4 * l, t.b = R / 2 + 4 * l;
  else
    t.a = 8 * l, t.b = 8 * l + 4;
  return t;
}
// The lane's four pairs turned by the position's angles; sign -1: back.
__device__ __forceinline__ void turn_pairs(Eight &e, const float4 *cs, int rope, float sign) {
  const float4 p = cs[0], q = cs[1];  // (cos, sin) of four angles
  const float c[4] = {p.x, p.z, q.x, q.z};
  const float s[4] = {sign * p.y, sign * p.w, sign * q.y, sign * q.w};
  const bool halves = rope == AG_ROPE_HALVES;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = halves ? e.v[i] : e.v[2 * i], y = halves ? e.v[i + 4] : e.v[2 * i + 1];
    const float u = fmaf(x, c[i], -y * s[i]), w = fmaf(y, c[i], x * s[i]);
    if (halves) e.v[i] = u, e.v[i + 4] = w;
    else e.v[2 * i] = u, e.v[2 * i + 1] = w;
  }
}

// The position's angles into the warp's own shared memory.
__device__ __forceinline__ void warp_angles(const QkArgs &a, float2 *cs, int64_t b, int64_t l,
                                            int lane) {
  __syncwarp();
  const long long pos = a.positions ? a.positions[b * a.pos_sb + l] : l;
  for (int i = lane; i < a.R / 2; i += 32) cs[i] = turn(pos, a.inv_freq[i]);
  __syncwarp();
}

// n = (x - mean) r in place; r.
template <int LPR>
__device__ __forceinline__ float normalise(Eight &e, const QkArgs &a, float inv_d, bool in) {
  if (a.norm == AG_NORM_NONE) return 1.f;
  float mean = 0.f;
  if (a.norm == AG_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += e.v[i];
    mean = row_sum<LPR>(s) * inv_d;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    e.v[i] = in ? e.v[i] - mean : 0.f;
    q = fmaf(e.v[i], e.v[i], q);
  }
  const float r = 1.f / sqrtf(fmaf(row_sum<LPR>(q), inv_d, a.eps));
#pragma unroll
  for (int i = 0; i < 8; ++i) e.v[i] *= r;
  return r;
}

template <int LPR, bool X32, bool O32>
__global__ void __launch_bounds__(kThreads, 3) qk_fwd_rows_kernel(const QkArgs a) {
  extern __shared__ float smem[];
  constexpr int kAtOnce = 32 / LPR, kSteps = 4;  // rows per step; steps loaded together
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  float2 *cs = reinterpret_cast<float2 *>(smem) + warp * (a.R / 2);
  const Lane t = lane_of<LPR>(lane, a.D, a.R, a.rope);
  const float inv_d = 1.f / a.D;
  const bool x_bf16 = a.x_dtype == AG_BF16, o_bf16 = a.o_dtype == AG_BF16;
  const uint32_t L = static_cast<uint32_t>(a.L), total = static_cast<uint32_t>(a.positions_total);
  for (uint32_t pos = blockIdx.x * kWarps + warp; pos < total; pos += gridDim.x * kWarps) {
    const uint32_t b32 = pos / L;
    const int64_t b = b32, l = pos - b32 * L;
    if (a.R) warp_angles(a, cs, b, l, lane);
    const float4 *angles = reinterpret_cast<const float4 *>(cs) + 2 * (lane % LPR);
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      const QkSide &s = a.side[which];
      const int64_t from = b * s.sb + l * s.sl, to = (b * s.H * a.L + l) * a.D;
      const Eight w = t.in ? param8(s.w, t.a, t.b, 1.f) : Eight{}, bias = t.in ? param8(s.b, t.a, t.b, 0.f) : Eight{};
#pragma unroll 1
      for (int h0 = 0; h0 < s.H; h0 += kAtOnce * kSteps) {
        Raw<X32> raw[kSteps];
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
          const int h = h0 + u * kAtOnce + lane / LPR;
          raw[u] = Raw<X32>{};
          if (t.in && h < s.H) raw[u] = load8<X32>(s.x, from + h * s.sh, t.a, t.b);
        }
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
          if (h0 + u * kAtOnce >= s.H) break;
          const int h = h0 + u * kAtOnce + lane / LPR;
          Eight x = widen<X32>(raw[u], x_bf16);
          normalise<LPR>(x, a, inv_d, t.in);
#pragma unroll
          for (int i = 0; i < 8; ++i) x.v[i] = fmaf(x.v[i], w.v[i], bias.v[i]);
          if (t.turns) turn_pairs(x, angles, a.rope, 1.f);
          if (t.in && h < s.H) store8<O32>(s.out, to + h * a.L * a.D, t.a, t.b, x, o_bf16);
        }
      }
    }
  }
}

// Backward.  A lane's elements are the same in every row it meets, so it sums
// the parameter gradients of a position's heads in registers and adds them to
// shared memory of its own, [w and b of both sides][two quads][lane]; the block
// adds its lanes' and warps' at the end, in a fixed order, and writes one
// partial.
template <int LPR, bool X32, bool G32>
__global__ void __launch_bounds__(kThreads, 2) qk_bwd_rows_kernel(const QkArgs a) {
  extern __shared__ float smem[];
  constexpr int kAtOnce = 32 / LPR, kSteps = 2;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  float2 *cs = reinterpret_cast<float2 *>(smem) + warp * (a.R / 2);
  float4 *sums = reinterpret_cast<float4 *>(smem + kWarps * a.R);  // [kWarps][8][32]
  float4 *own = sums + warp * 8 * 32 + lane;
  if (a.partial)
#pragma unroll
    for (int q = 0; q < 8; ++q) own[q * 32] = make_float4(0.f, 0.f, 0.f, 0.f);
  const Lane t = lane_of<LPR>(lane, a.D, a.R, a.rope);
  const float4 *angles = reinterpret_cast<const float4 *>(cs) + 2 * (lane % LPR);
  const float inv_d = 1.f / a.D;
  const bool x_bf16 = a.x_dtype == AG_BF16, g_bf16 = a.o_dtype == AG_BF16;
  const uint32_t L = static_cast<uint32_t>(a.L), total = static_cast<uint32_t>(a.positions_total);
  for (uint32_t pos = blockIdx.x * kWarps + warp; pos < total; pos += gridDim.x * kWarps) {
    const uint32_t b32 = pos / L;
    const int64_t b = b32, l = pos - b32 * L;
    bool angles_ready = a.R == 0;
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      const QkSide &s = a.side[which];
      if (s.H == 0) continue;
      const int64_t x_at = b * s.sb + l * s.sl, g_at = (b * s.H * a.L + l) * a.D,
                    dx_at = b * s.dxb + l * s.dxl;
      const Eight w = t.in ? param8(s.w, t.a, t.b, 1.f) : Eight{};
      Eight dw{}, db{};
#pragma unroll 1
      for (int h0 = 0; h0 < s.H; h0 += kAtOnce * kSteps) {
        Raw<X32> raw_x[kSteps];
        Raw<G32> raw_g[kSteps];
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
          const int h = h0 + u * kAtOnce + lane / LPR;
          raw_x[u] = Raw<X32>{}, raw_g[u] = Raw<G32>{};
          if (t.in && h < s.H) {
            raw_x[u] = load8<X32>(s.x, x_at + h * s.sh, t.a, t.b);
            raw_g[u] = load8<G32>(s.g, g_at + h * a.L * a.D, t.a, t.b);
          }
        }
        if (!angles_ready) {  // while the first rows are on their way
          warp_angles(a, cs, b, l, lane);
          angles_ready = true;
        }
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
          if (h0 + u * kAtOnce >= s.H) break;
          const int h = h0 + u * kAtOnce + lane / LPR;
          const bool mine = t.in && h < s.H;
          Eight x = widen<X32>(raw_x[u], x_bf16), g = widen<G32>(raw_g[u], g_bf16);
          const float r = normalise<LPR>(x, a, inv_d, t.in);
          if (t.turns) turn_pairs(g, angles, a.rope, -1.f);
          float along = 0.f, total = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            // (A row of this step past the last head counts for nothing, also
            // when eps is zero and its norm is not a number.)
            if (mine) dw.v[i] = fmaf(g.v[i], x.v[i], dw.v[i]), db.v[i] += g.v[i];
            g.v[i] *= w.v[i];
            along = fmaf(g.v[i], x.v[i], along);
            total += g.v[i];
          }
          along = a.norm == AG_NORM_NONE ? 0.f : row_sum<LPR>(along) * inv_d;
          total = a.norm == AG_NORM_LAYER ? row_sum<LPR>(total) * inv_d : 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) g.v[i] = r * (fmaf(-x.v[i], along, g.v[i]) - total);
          if (mine) store8<X32>(s.dx, dx_at + h * s.dxh, t.a, t.b, g, x_bf16);
        }
      }
      if (a.partial) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float *v = (q < 2 ? dw.v : db.v) + 4 * (q & 1);
          float4 &o = own[(which * 4 + q) * 32];
          const float4 was = o;
          o = make_float4(was.x + v[0], was.y + v[1], was.z + v[2], was.w + v[3]);
        }
      }
    }
  }
  if (!a.partial) return;
  __syncthreads();
  for (int i = threadIdx.x; i < 4 * a.D; i += kThreads) {
    // Element e of array `which` lies in quad `quad` of lane `at` (lane_of).
    const int which = i / a.D, e = i % a.D;
    const bool half = a.rope == AG_ROPE_HALVES && e < a.R;
    const int quad = half ? e / (a.R / 2) : (e % 8) / 4, at = half ? e % (a.R / 2) / 4 : e / 8;
    const float *from = reinterpret_cast<const float *>(sums + (which * 2 + quad) * 32 + at) + e % 4;
    float v = 0.f;
    for (int w = 0; w < kWarps; ++w)
#pragma unroll
      for (int row = 0; row < kAtOnce; ++row) v += from[(w * 8 * 32 + row * LPR) * 4];
    a.partial[static_cast<int64_t>(blockIdx.x) * 4 * a.D + i] = v;
  }
}

// --------------------------------------------------------------------------
// General kernels.  One warp per (position, head) row, any D and any strides.
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

// A quad of elements can be loaded at every address of the tensor.
bool quads(const void *p, int dtype, int64_t s0, int64_t s1, int64_t s2) {
  return aligned(p, dtype == AG_F32 ? 16 : 8) && s0 % 4 == 0 && s1 % 4 == 0 && s2 % 4 == 0;
}
// Whether the rows kernels can take the call.
bool by_rows(const QkArgs &a, bool backward) {
  if (a.D % 8 || a.D > 256 || a.R % 8) return false;
  for (const QkSide &s : a.side) {
    if (s.H == 0) continue;
    if (!quads(s.x, a.x_dtype, s.sb, s.sl, s.sh)) return false;
    if (backward ? !quads(s.g, a.o_dtype, 0, 0, 0) || !quads(s.dx, a.x_dtype, s.dxb, s.dxl, s.dxh)
                 : !quads(s.out, a.o_dtype, 0, 0, 0))
      return false;
  }
  return true;
}

int bwd_warps(int D) { return D <= 512 ? 8 : 4; }
// Blocks of a backward, as many as its partial sums: the rows kernel's two to an
// SM, the general one's four, but no more than have work.
int bwd_blocks(int64_t total, int64_t each, int per_sm, int num_sms) {
  const int64_t turns = (total + each - 1) / each;
  return static_cast<int>(turns < per_sm * num_sms ? turns : per_sm * num_sms);
}

cudaError_t allow_smem(const void *kernel, size_t bytes) {
  return bytes <= 48 * 1024 ? cudaSuccess
                            : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(bytes));
}

}  // namespace

int64_t qk_bwd_workspace(int64_t positions_total, int64_t D, int num_sms) {
  return static_cast<int64_t>(bwd_blocks(positions_total, kPos, 4, num_sms)) * 4 * D * 4;
}

namespace {

using QkKernel = void (*)(QkArgs);
template <bool X32, bool O32>
QkKernel rows_kernel(int D, bool backward) {
  if (backward)
    return D <= 32    ? qk_bwd_rows_kernel<4, X32, O32>
           : D <= 64  ? qk_bwd_rows_kernel<8, X32, O32>
           : D <= 128 ? qk_bwd_rows_kernel<16, X32, O32>
                      : qk_bwd_rows_kernel<32, X32, O32>;
  return D <= 32    ? qk_fwd_rows_kernel<4, X32, O32>
         : D <= 64  ? qk_fwd_rows_kernel<8, X32, O32>
         : D <= 128 ? qk_fwd_rows_kernel<16, X32, O32>
                    : qk_fwd_rows_kernel<32, X32, O32>;
}
QkKernel rows_kernel(const QkArgs &a, bool backward) {
  const bool o32 = a.o_dtype == AG_F32;
  if (a.x_dtype == AG_F32)
    return o32 ? rows_kernel<true, true>(a.D, backward) : rows_kernel<true, false>(a.D, backward);
  return o32 ? rows_kernel<false, true>(a.D, backward) : rows_kernel<false, false>(a.D, backward);
}

}  // namespace

cudaError_t launch_qk_fwd(const QkArgs &a, int num_sms, cudaStream_t stream) {
  if (by_rows(a, false)) {
    const int64_t blocks = (a.positions_total + kWarps - 1) / kWarps;
    rows_kernel(a, false)<<<static_cast<unsigned>(blocks < 24 * num_sms ? blocks : 24 * num_sms),
                            kThreads, kWarps * a.R * 4, stream>>>(a);
    return cudaGetLastError();
  }
  const size_t smem = (static_cast<size_t>(kPos) * a.R + kWarps * static_cast<size_t>(a.D)) * 4;
  cudaError_t e = allow_smem(reinterpret_cast<const void *>(qk_fwd_kernel), smem);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (a.positions_total + kPos - 1) / kPos;
  qk_fwd_kernel<<<static_cast<unsigned>(blocks), kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_qk_bwd(const QkArgs &a, int num_sms, cudaStream_t stream) {
  int blocks;
  if (by_rows(a, true)) {
    blocks = bwd_blocks(a.positions_total, kWarps, 2, num_sms);
    rows_kernel(a, true)<<<blocks, kThreads, kWarps * (a.R + 8 * 32 * 4) * 4, stream>>>(a);
  } else {
    const int warps = bwd_warps(a.D);
    blocks = bwd_blocks(a.positions_total, kPos, 4, num_sms);
    const size_t smem = (static_cast<size_t>(kPos) * a.R + warps * 6 * static_cast<size_t>(a.D)) * 4;
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(qk_bwd_kernel), smem);
    if (e != cudaSuccess) return e;
    qk_bwd_kernel<<<blocks, warps * 32, smem, stream>>>(a, warps);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.partial) return e;
  qk_params_kernel<<<(4 * a.D + 31) / 32, 256, 0, stream>>>(
      a.partial, blocks, a.D, a.side[0].dw, a.side[0].db, a.side[1].dw, a.side[1].db);
  return cudaGetLastError();
}

}  // namespace ag
