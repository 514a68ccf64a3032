// linear_epilogue.cuh -- what a linear layer does to a product's float32 sums
// before they are stored: bias, pre-activation output, activation or the
// derivative of one, residual, and the one rounding to the output's type.
// Used by every kernel that finishes a product (linear.cu, linear_sm100.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ag_internal.h"

namespace ag {

__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case AG_ACT_RELU: return z > 0.f ? z : (z != z ? z : 0.f);
    case AG_ACT_GELU: return 0.5f * z * (1.f + erff(z * 0.70710678f));
    case AG_ACT_GELU_TANH: {
      // (1 + tanh u) / 2 = 1 / (1 + exp(-2u)).
      const float u2 = 1.5957691f * (z + 0.044715f * z * z * z);
      return z / (1.f + __expf(-u2));
    }
    case AG_ACT_SILU: return z / (1.f + __expf(-z));
    default: return z;
  }
}

__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case AG_ACT_RELU: return z > 0.f ? 1.f : 0.f;
    case AG_ACT_GELU:
      return 0.5f * (1.f + erff(z * 0.70710678f)) + z * 0.39894228f * __expf(-0.5f * z * z);
    case AG_ACT_GELU_TANH: {
      const float u2 = 1.5957691f * (z + 0.044715f * z * z * z);
      const float p = 1.f / (1.f + __expf(-u2));
      return p + z * p * (1.f - p) * 1.5957691f * (1.f + 0.134145f * z * z);
    }
    case AG_ACT_SILU: {
      const float p = 1.f / (1.f + __expf(-z));
      return p * (1.f + z * (1.f - p));
    }
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
