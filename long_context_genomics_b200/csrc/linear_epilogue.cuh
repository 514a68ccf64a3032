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

// Phi(-|z|), the tail of the normal distribution, and exp(-z^2 / 2):
// Abramowitz and Stegun 7.1.26 for erfc(|z| / sqrt 2) / 2, within 7e-8 (so the
// GELU within 2.2e-7).  Two special-function instructions, shared by the GELU
// and its derivative; erff and expf cost some 40 instructions an element, which
// made the epilogue of a feed-forward layer slower than its product.
struct NormalTail {
  float tail, exp;
};
__device__ __forceinline__ NormalTail normal_tail(float x) {  // x = |z|
  const float t = rcp_approx(fmaf(0.23164189f, x, 1.f));      // 0.3275911 / sqrt 2
  NormalTail n;
  n.exp = ex2_approx(-0.72134752f * x * x);                   // log2(e) / 2
  float q = fmaf(0.5307027145f, t, -0.7265760135f);           // halves of the published a5 .. a1
  q = fmaf(q, t, 0.7107068705f);
  q = fmaf(q, t, -0.142248368f);
  q = fmaf(q, t, 0.127414796f);
  n.tail = q * t * n.exp;
  return n;
}
__device__ __forceinline__ float logistic(float u) {
  return rcp_approx(1.f + ex2_approx(-1.44269504f * u));
}

// Activations and their derivatives (AG_ACT_*).  In the GELU, |z| beyond 30
// counts as 30 beside a tail that is zero there, so that an infinity gives its
// limit.
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == AG_ACT_RELU) return z > 0.f ? z : (z != z ? z : 0.f);
  if constexpr (ACT == AG_ACT_GELU) {
    const float x = fminf(fabsf(z), 30.f);
    // z Phi(z) = max(z, 0) - |z| Phi(-|z|); z - z keeps a NaN.
    return fmaf(-x, normal_tail(x).tail, z > 0.f ? z : (z != z ? z : 0.f));
  }
  if constexpr (ACT == AG_ACT_GELU_TANH)  // (1 + tanh u) / 2 is the logistic of 2u
    return z * logistic(1.5957691f * z * fmaf(0.044715f * z, z, 1.f));
  if constexpr (ACT == AG_ACT_SILU) return z * logistic(z);
  return z;
}
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == AG_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  if constexpr (ACT == AG_ACT_GELU) {
    const float x = fminf(fabsf(z), 30.f);
    const NormalTail n = normal_tail(x);
    return fmaf(copysignf(x, z) * 0.39894228f, n.exp,
                z > 0.f ? 1.f - n.tail : (z != z ? z : n.tail));
  }
  if constexpr (ACT == AG_ACT_GELU_TANH) {
    const float p = logistic(1.5957691f * z * fmaf(0.044715f * z, z, 1.f));
    return fmaf(z * p * (1.f - p), 1.5957691f * fmaf(0.134145f * z, z, 1.f), p);
  }
  if constexpr (ACT == AG_ACT_SILU) {
    const float p = logistic(z);
    return p * fmaf(z, 1.f - p, 1.f);
  }
  return 1.f;
}
__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case AG_ACT_RELU: return act_value<AG_ACT_RELU>(z);
    case AG_ACT_GELU: return act_value<AG_ACT_GELU>(z);
    case AG_ACT_GELU_TANH: return act_value<AG_ACT_GELU_TANH>(z);
    case AG_ACT_SILU: return act_value<AG_ACT_SILU>(z);
    default: return z;
  }
}
__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case AG_ACT_RELU: return act_slope<AG_ACT_RELU>(z);
    case AG_ACT_GELU: return act_slope<AG_ACT_GELU>(z);
    case AG_ACT_GELU_TANH: return act_slope<AG_ACT_GELU_TANH>(z);
    case AG_ACT_SILU: return act_slope<AG_ACT_SILU>(z);
    default: return 1.f;
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
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] *= act_slope(z[i], e.act);
  } else if (e.act != AG_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = act_value(v[i], e.act);
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
