// linear_epilogue.cuh -- what a linear layer does to a product's float32 sums
// before they are stored: bias, pre-activation output, activation or the
// derivative of one, residual, and the one rounding to the output's type.
// Used by every kernel that finishes a product (linear.cu, linear_sm100.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ag_internal.h"
#include "sm100.cuh"

namespace ag {

__device__ __forceinline__ float2 both(float c) { return make_float2(c, c); }

// Activations and their derivatives (AG_ACT_*) of two values at a time, in the
// two-lane float32 instructions.
//
// Phi(-|z|), the tail of the normal distribution, and exp(-z^2 / 2).  The tail is
// R exp(-z^2 / 2) with R = u P(u), u = 1 / (1 + 0.35 |z|), P of degree 6: a
// minimax fit on |z| <= 13.5 (a linear program over Chebyshev points) of the error
// relative to R, weighted by min(30, 1 / (2 tail max(|z|, 1))) and 9.1e-8 times that
// at most.  So the GELU is within 1.1e-7 and, where it is small, within 5e-6 of
// itself down to z = -8 (in float32; an erf would leave it 6e-8 and nothing of its
// digits beyond -5).  Two special-function instructions, shared by the GELU and
// its derivative; erff and expf cost some 40 instructions an element, which made
// the epilogue of a feed-forward layer slower than its product.
struct NormalTail {
  float2 tail, exp;
};
__device__ __forceinline__ NormalTail normal_tail(float2 x) {   // x = |z|
  const float2 d = __ffma2_rn(both(0.35f), x, both(1.f));
  const float2 u = make_float2(rcp_approx(d.x), rcp_approx(d.y));
  const float2 h = __fmul2_rn(__fmul2_rn(both(-0.72134752f), x), x);  // log2(e) / 2
  NormalTail n;
  n.exp = make_float2(ex2_approx(h.x), ex2_approx(h.y));
  float2 q = __ffma2_rn(both(0.045088783f), u, both(-0.18631811f));
  q = __ffma2_rn(q, u, both(0.21410257f));
  q = __ffma2_rn(q, u, both(0.0064734956f));
  q = __ffma2_rn(q, u, both(0.14421174f));
  q = __ffma2_rn(q, u, both(0.13664697f));
  q = __ffma2_rn(q, u, both(0.1397946f));
  n.tail = __fmul2_rn(__fmul2_rn(q, u), n.exp);
  return n;
}
// 1 / (1 + 2^u).
__device__ __forceinline__ float2 logistic2(float2 u) {
  const float2 d = __fadd2_rn(make_float2(ex2_approx(u.x), ex2_approx(u.y)), both(1.f));
  return make_float2(rcp_approx(d.x), rcp_approx(d.y));
}
// -2 log2(e) sqrt(2 / pi) (z + 0.044715 z^3): (1 + tanh) / 2 = logistic2 of it.
__device__ __forceinline__ float2 tanh_argument(float2 z) {
  const float2 w = __ffma2_rn(__fmul2_rn(both(-0.10294324f), z), z, both(-2.3022082f));
  return __fmul2_rn(w, z);
}

template <int ACT>
__device__ __forceinline__ float2 act_value2(float2 z) {
  if constexpr (ACT == AG_ACT_RELU)
    return make_float2(z.x > 0.f ? z.x : (z.x != z.x ? z.x : 0.f),
                       z.y > 0.f ? z.y : (z.y != z.y ? z.y : 0.f));
  if constexpr (ACT == AG_ACT_GELU) {
    // z Phi(z) = max(z, 0) - |z| Phi(-|z|).  The factor |z| stops at 30, where
    // the tail is zero, so that an infinity gives its limit; a NaN comes
    // through the tail.
    const float2 x = make_float2(fabsf(z.x), fabsf(z.y));
    return __ffma2_rn(make_float2(-fminf(x.x, 30.f), -fminf(x.y, 30.f)), normal_tail(x).tail,
                      make_float2(fmaxf(z.x, 0.f), fmaxf(z.y, 0.f)));
  }
  if constexpr (ACT == AG_ACT_GELU_TANH) return __fmul2_rn(z, logistic2(tanh_argument(z)));
  if constexpr (ACT == AG_ACT_SILU)
    return __fmul2_rn(z, logistic2(__fmul2_rn(both(-1.44269504f), z)));
  return z;
}
template <int ACT>
__device__ __forceinline__ float2 act_slope2(float2 z) {
  if constexpr (ACT == AG_ACT_RELU) return make_float2(z.x > 0.f ? 1.f : 0.f, z.y > 0.f ? 1.f : 0.f);
  if constexpr (ACT == AG_ACT_GELU) {
    const float2 x = make_float2(fabsf(z.x), fabsf(z.y));
    const NormalTail n = normal_tail(x);
    const float2 c = make_float2(copysignf(fminf(x.x, 30.f), z.x), copysignf(fminf(x.y, 30.f), z.y));
    return __ffma2_rn(__fmul2_rn(both(0.39894228f), c), n.exp,
                      make_float2(z.x > 0.f ? 1.f - n.tail.x : n.tail.x,
                                  z.y > 0.f ? 1.f - n.tail.y : n.tail.y));
  }
  if constexpr (ACT == AG_ACT_GELU_TANH) {
    const float2 p = logistic2(tanh_argument(z));
    const float2 r = __ffma2_rn(make_float2(-p.x, -p.y), p, p);  // p (1 - p)
    // (z^2 stops at 2^100: beyond that r is zero, and zero times infinity is not.)
    const float2 s = __fmul2_rn(z, z);
    const float2 k = __ffma2_rn(both(0.21406445f),
                                make_float2(fminf(s.x, 0x1p100f), fminf(s.y, 0x1p100f)),
                                both(1.5957691f));
    return __ffma2_rn(__fmul2_rn(z, r), k, p);
  }
  if constexpr (ACT == AG_ACT_SILU) {
    const float2 p = logistic2(__fmul2_rn(both(-1.44269504f), z));
    const float2 r = __ffma2_rn(make_float2(-p.x, -p.y), p, p);
    return __ffma2_rn(z, r, p);
  }
  return both(1.f);
}
// V values in place; the activation looked up once for all of them.
template <int ACT, bool SLOPE, int V>
__device__ __forceinline__ void act_all(float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    const float2 z = make_float2(v[i], i + 1 < V ? v[i + 1] : 0.f);
    const float2 y = SLOPE ? act_slope2<ACT>(z) : act_value2<ACT>(z);
    v[i] = y.x;
    if (i + 1 < V) v[i + 1] = y.y;
  }
}
template <bool SLOPE, int V>
__device__ __forceinline__ void act_all(float (&v)[V], int act) {
  switch (act) {
    case AG_ACT_RELU: return act_all<AG_ACT_RELU, SLOPE>(v);
    case AG_ACT_GELU: return act_all<AG_ACT_GELU, SLOPE>(v);
    case AG_ACT_GELU_TANH: return act_all<AG_ACT_GELU_TANH, SLOPE>(v);
    case AG_ACT_SILU: return act_all<AG_ACT_SILU, SLOPE>(v);
    default: return act_all<AG_ACT_NONE, SLOPE>(v);
  }
}

// V values of a type from p: 16-byte loads for V == 8 (p 16-byte aligned).
template <int V>
__device__ __forceinline__ void load_values(const void *base, int64_t at, int dtype, float (&v)[V]) {
  if (dtype == AG_F32) {
    const float *p = static_cast<const float *>(base) + at;
    if constexpr (V == 8) {
      const float4 a = *reinterpret_cast<const float4 *>(p);
      const float4 b = *reinterpret_cast<const float4 *>(p + 4);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = p[i];
    }
  } else {
    const uint16_t *p = static_cast<const uint16_t *>(base) + at;
    uint32_t w[(V + 1) / 2];
    if constexpr (V == 8) {
      const uint4 a = *reinterpret_cast<const uint4 *>(p);
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (i & 1) w[i / 2] |= static_cast<uint32_t>(p[i]) << 16;
        else w[i / 2] = p[i];
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t h = (w[i / 2] >> (16 * (i & 1))) & 0xFFFFu;
      v[i] = dtype == AG_BF16 ? __uint_as_float(h << 16)
                              : __half2float(__ushort_as_half(static_cast<uint16_t>(h)));
    }
  }
}

// N values `step` elements apart, those from n on zero, for readers that cannot
// take 16 bytes at a time.  All loads are issued before the first is converted:
// with each converted as it comes, the type's branch made every load wait for
// the one before (a 16-bit residual in 8192 x 2047 outputs took 80 us).
template <int N>
__device__ __forceinline__ void load_apart(const void *base, int64_t at, int64_t step, int n,
                                           int dtype, float (&v)[N]) {
  if (dtype == AG_F32) {
    const float *p = static_cast<const float *>(base) + at;
#pragma unroll
    for (int i = 0; i < N; ++i, p += step) v[i] = i < n ? *p : 0.f;
    return;
  }
  const uint16_t *p = static_cast<const uint16_t *>(base) + at;
  uint16_t h[N];
#pragma unroll
  for (int i = 0; i < N; ++i, p += step) h[i] = i < n ? *p : 0;
  if (dtype == AG_BF16) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __uint_as_float(static_cast<uint32_t>(h[i]) << 16);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __half2float(__ushort_as_half(h[i]));
  }
}

template <int V>
__device__ __forceinline__ void store_values(void *base, int64_t at, int dtype, const float (&v)[V]) {
  if (dtype == AG_F32) {
    float *p = static_cast<float *>(base) + at;
    if constexpr (V == 8) {
      *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) p[i] = v[i];
    }
  } else {
    uint16_t *p = static_cast<uint16_t *>(base) + at;
    uint16_t h[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
      h[i] = dtype == AG_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v[i]))
                              : __half_as_ushort(__float2half_rn(v[i]));
    if constexpr (V == 8) {
      uint4 a;
      a.x = h[0] | (static_cast<uint32_t>(h[1]) << 16);
      a.y = h[2] | (static_cast<uint32_t>(h[3]) << 16);
      a.z = h[4] | (static_cast<uint32_t>(h[5]) << 16);
      a.w = h[6] | (static_cast<uint32_t>(h[7]) << 16);
      *reinterpret_cast<uint4 *>(p) = a;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) p[i] = h[i];
    }
  }
}

// V consecutive columns of one row, from the product's float32 sums; V == 8
// needs e.vec8 and a column that is a multiple of 8.  `bias` holds the columns'
// bias, or zeros.
template <int V>
__device__ __forceinline__ void linear_finish(const LinearEpilogue &e, float (&v)[V],
                                              const float (&bias)[V], int64_t row, int64_t col) {
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] += bias[i];
  if (e.pre_out) store_values<V>(e.pre_out, row * e.ld_pre_out + col, e.dtype, v);
  if (e.pre_in) {
    float z[V];
    load_values<V>(e.pre_in, row * e.ld_pre_in + col, e.dtype, z);
    act_all<true>(z, e.act);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] *= z[i];
  } else if (e.act != AG_ACT_NONE) {
    act_all<false>(v, e.act);
  }
  if (e.residual) {
    float r[V];
    load_values<V>(e.residual, row * e.ld_res + col, e.out_dtype, r);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += r[i];
  }
  store_values<V>(e.out, row * e.ld_out + col, e.out_dtype, v);
}

}  // namespace ag
