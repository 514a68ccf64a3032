// qk_norm_rope.cu -- per-head norm of queries and keys with the rotation by
// position, from the projections' layout [B, L, H, D] to the attention's
// [B, H, L, D], and its gradients (ag_qk_norm_rope_fwd, ag_qk_norm_rope_bwd).
//
//   n = (x - mean) r,  v = n w + b,  out = R(position) v
//   g = R^T dout,  dw = sum g n,  db = sum g,  d = g w,
//   dx = r (d - n mean(d n) - mean d)
//
// Every element is read once and written once (the backward reads x and dout
// and writes dx), so memory would bound it; what does is said below.
//
// Rows kernels (heads of a multiple of 8 up to 256 elements, at addresses that
// 4 elements' loads can take; weights and biases 16-byte aligned): a group of
// D / 8 lanes takes one position and some of its heads, one after the other, so
// that the position's addresses and angles are formed once for them, by the
// groups of a warp side by side.  A lane holds eight elements of a row in two
// quads; where halves are rotated, those are 4 elements of the first half and
// their partners in the second, so no lane needs another's values but for the
// norm's sums.  Two rows (in the backward four) are loaded before the first is
// worked on and their norms' sums are formed side by side.  What bounds them is
// the instructions: some 85 for a warp's two rows, 140 for two positions' angles
// and 200 for their addresses and weights, and the latency of a row's chain of
// sums, at two thirds of the issue rate.  Full context (75 MB, 16384 positions,
// 8 + 1 heads of 128, bf16): 20.4 us in the forward; four rows at a time 24 us
// (fewer warps fit), sixteen elements to a lane 23 us, a fixed grid over
// positions 23.6 us.  Gradients of half of that (76 MB): 25 us.
// Instances of 32-bit q and k spill: up to 20 bytes in the forward (64 registers,
// four blocks an SM), up to 52 in the gradients (128, two blocks).
//
// General kernels: one warp per row through shared memory, any size or stride.  A
// block takes `at_once` positions a turn, enough for a row to each warp.  Bound by
// the instructions around each element: 8192 positions of 8 + 1 heads of 100 in
// bf16 57 us, the gradients 87 us; with the types looked up per element, divisions
// of 64 bits and the gradient turned back a second time 77 and 112 us.
#include "ag_internal.h"
#include "launch.cuh"
#include "linear_epilogue.cuh"

namespace ag {
namespace {

constexpr int kThreads = 256;  // 8 warps
constexpr int kWarps = kThreads / 32;

// cos and sin of position * frequency.  The product and its reduction are in 64
// bits (by a two-part 2 pi or pi / 2), so the phase of a far position is as exact
// as the frequency, up to angles of 2^50.
//
// Where the results are of 16 bits, the special-function unit's sine and cosine
// on [-pi, pi], within 2^-21 (CUDA's bound for the fast functions), are far
// below their rounding.  EXACT, for 32-bit results: the Taylor sums to r^9 and
// r^10 on [-pi / 4, pi / 4], where the next terms are below
// 2^-28; within 1.3 units of 2^-24.
template <bool EXACT>
__device__ __forceinline__ float2 turn(long long pos, double freq) {
  double a = static_cast<double>(pos) * freq;
  if constexpr (!EXACT) {
    const double n = rint(a * 0.15915494309189535);
    double r = fma(n, -6.283185307179586, a);
    r = fma(n, -2.4492935982947064e-16, r);
    float s, c;
    __sincosf(static_cast<float>(r), &s, &c);
    return make_float2(c, s);
  }
  // Angles of 2^51 and more have no quarter turn left that could be told: 0 (or NaN).
  if ((__double2hiint(a) & 0x7FFFFFFF) >= 0x43200000) a -= a;
  // Rounded by adding 1.5 * 2^52: the sum's lower word ends in the quarter turns.
  const double t = fma(a, 0.6366197723675814, 0x1.8p52), n = t - 0x1.8p52;
  const int turns = __double2loint(t);
  const float r = static_cast<float>(
      fma(n, -6.123233995736766e-17, fma(n, -1.5707963267948966, a)));
  const float q = r * r;
  float s = fmaf(q, 1.f / 362880, -1.f / 5040), c = fmaf(q, -1.f / 3628800, 1.f / 40320);
  s = fmaf(fmaf(s, q, 1.f / 120), q, -1.f / 6);
  c = fmaf(fmaf(fmaf(c, q, -1.f / 720), q, 1.f / 24), q, -0.5f);
  s = fmaf(s * q, r, r), c = fmaf(c, q, 1.f);
  const float cos = turns & 1 ? s : c, sin = turns & 1 ? c : s;
  const uint32_t top = 0x80000000u;
  return make_float2(
      __uint_as_float(__float_as_uint(cos) ^ ((static_cast<uint32_t>(turns) + 1) << 30 & top)),
      __uint_as_float(__float_as_uint(sin) ^ (static_cast<uint32_t>(turns) << 30 & top)));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int T>
__device__ __forceinline__ float load_one(const void *p, int64_t at) {
  float v[1];
  load_values<1>(p, at, T, v);
  return v[0];
}
template <int T>
__device__ __forceinline__ void store_one(void *p, int64_t at, float x) {
  const float v[1] = {x};
  store_values<1>(p, at, T, v);
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

// A lane's eight elements of a row, as loaded (of type T) from two places
// and as numbers: four pairs (A[i], B[i]) that turn together, A in v[0] and
// v[1], B in v[2] and v[3].  HALVES: the first place holds A and the second B;
// otherwise A are the even and B the odd elements of both.  Loading and
// widening are apart so that nothing waits for a load before all of them have
// been issued.
template <int T>
struct Raw {
  uint2 a, b;
};
template <>
struct Raw<AG_F32> {
  float4 a, b;
};
struct Eight {
  float2 v[4];
};

// Bytes of n elements of a type.
template <int T>
__device__ __forceinline__ int64_t bytes_of(int64_t n) {
  return T == AG_F32 ? n * 4 : n * 2;
}
// From the row's bytes at p, where the lane's first quad lies; its second is
// `apart` bytes on.
template <int T>
__device__ __forceinline__ Raw<T> load8(const char *p, int apart) {
  using Quad = decltype(Raw<T>::a);
  return {*reinterpret_cast<const Quad *>(p), *reinterpret_cast<const Quad *>(p + apart)};
}
template <int T>
__device__ __forceinline__ float2 widen2(uint32_t w) {
  if constexpr (T == AG_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <bool HALVES>
__device__ __forceinline__ Eight arrange(float2 p, float2 q, float2 s, float2 t) {
  if constexpr (HALVES) return {{p, q, s, t}};
  return {{make_float2(p.x, q.x), make_float2(s.x, t.x), make_float2(p.y, q.y),
           make_float2(s.y, t.y)}};
}
template <int T, bool HALVES>
__device__ __forceinline__ Eight widen(const Raw<T> &r) {
  if constexpr (T == AG_F32)
    return arrange<HALVES>(make_float2(r.a.x, r.a.y), make_float2(r.a.z, r.a.w),
                           make_float2(r.b.x, r.b.y), make_float2(r.b.z, r.b.w));
  else
    return arrange<HALVES>(widen2<T>(r.a.x), widen2<T>(r.a.y), widen2<T>(r.b.x), widen2<T>(r.b.y));
}
template <int T>
__device__ __forceinline__ uint32_t narrow2(float2 v) {
  if constexpr (T == AG_BF16) return pack_bf16x2(v.x, v.y);
  const __half2 h = __floats2half2_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t *>(&h);
}
template <int T, bool HALVES>
__device__ __forceinline__ void store8(char *p, int apart, const Eight &e) {
  float2 o[4] = {e.v[0], e.v[1], e.v[2], e.v[3]};
  if constexpr (!HALVES) {
    o[0] = make_float2(e.v[0].x, e.v[2].x), o[1] = make_float2(e.v[0].y, e.v[2].y);
    o[2] = make_float2(e.v[1].x, e.v[3].x), o[3] = make_float2(e.v[1].y, e.v[3].y);
  }
  if constexpr (T == AG_F32) {
    *reinterpret_cast<float4 *>(p) = make_float4(o[0].x, o[0].y, o[1].x, o[1].y);
    *reinterpret_cast<float4 *>(p + apart) = make_float4(o[2].x, o[2].y, o[3].x, o[3].y);
  } else {
    *reinterpret_cast<uint2 *>(p) = make_uint2(narrow2<T>(o[0]), narrow2<T>(o[1]));
    *reinterpret_cast<uint2 *>(p + apart) = make_uint2(narrow2<T>(o[2]), narrow2<T>(o[3]));
  }
}
// Sums over the LPR lanes of a row, of both numbers, for N rows side by side
// (one row's sum waits for each of its exchanges; several rows' cover each
// other's).
template <int LPR, int N>
__device__ __forceinline__ void row_sums(const float2 (&v)[N], float (&s)[N]) {
#pragma unroll
  for (int u = 0; u < N; ++u) s[u] = v[u].x + v[u].y;
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1)
#pragma unroll
    for (int u = 0; u < N; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], o);
}
__device__ __forceinline__ float2 twice(float c) { return make_float2(c, c); }
__device__ __forceinline__ float2 negated(float2 v) { return make_float2(-v.x, -v.y); }
__device__ __forceinline__ float2 sum4(const Eight &e) {
  return __fadd2_rn(__fadd2_rn(e.v[0], e.v[1]), __fadd2_rn(e.v[2], e.v[3]));
}

// Where a lane's elements lie (two quads, at a and b), and whether they turn.
struct Lane {
  int a, b;
  bool in, turns;
};
template <int LPR, bool HALVES>
__device__ __forceinline__ Lane lane_of(int lane, int D, int R) {
  const int l = lane % LPR;
  Lane t;
  t.in = 8 * l < D;
  t.turns = 8 * l < R;
  if (HALVES && t.turns)
    t.a = 4 * l, t.b = R / 2 + 4 * l;
  else
    t.a = 8 * l, t.b = 8 * l + 4;
  return t;
}
// The lane's part of a weight or bias, where there is one.
template <bool HALVES>
__device__ __forceinline__ Eight param8(const float *p, const Lane &t, float otherwise) {
  if (!p || !t.in) {
    const float2 c = twice(t.in ? otherwise : 0.f);
    return {{c, c, c, c}};
  }
  const float4 x = __ldg(reinterpret_cast<const float4 *>(p + t.a));
  const float4 y = __ldg(reinterpret_cast<const float4 *>(p + t.b));
  return arrange<HALVES>(make_float2(x.x, x.y), make_float2(x.z, x.w), make_float2(y.x, y.y),
                         make_float2(y.z, y.w));
}
// The lane's four pairs turned by the position's angles; BACK: the other way.
template <bool BACK>
__device__ __forceinline__ void turn_pairs(Eight &e, const float4 *cos4, const float4 *sin4) {
  const float4 c = *cos4, s = *sin4;
  const float2 cs[2] = {make_float2(c.x, c.y), make_float2(c.z, c.w)};
  const float2 sn[2] = {make_float2(s.x, s.y), make_float2(s.z, s.w)};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 x = e.v[i], y = e.v[i + 2], p = __fmul2_rn(y, sn[i]), q = __fmul2_rn(x, sn[i]);
    e.v[i] = __ffma2_rn(x, cs[i], BACK ? p : negated(p));
    e.v[i + 2] = __ffma2_rn(y, cs[i], BACK ? negated(q) : q);
  }
}

// The angles of the group's position into its own shared memory: R / 2 cosines,
// then as many sines.
template <int LPR, bool EXACT>
__device__ __forceinline__ void group_angles(const QkArgs &a, float *cs, int64_t b, int64_t l,
                                             int lane) {
  __syncwarp();
  const long long pos = a.positions ? a.positions[b * a.pos_sb + l] : l;
  const int half = a.R / 2;
  const auto one = [&](int i) {
    const float2 c = turn<EXACT>(pos, a.inv_freq[i]);
    cs[i] = c.x, cs[half + i] = c.y;
  };
  if constexpr (EXACT) {
    // (Four side by side, or their chains of products add up: 16384 positions of 9
    // heads of 128 from bf16 to fp32 27.3 us, so 26.6; with the fast sine and
    // cosine 26.3.)
#pragma unroll 4
    for (int i = lane % LPR; i < half; i += LPR) one(i);
  } else {
    for (int i = lane % LPR; i < half; i += LPR) one(i);
  }
  __syncwarp();
}

// n = (x - mean) r in place, and r, for N rows.  Lanes without elements hold
// zeros.
template <int LPR, int N>
__device__ __forceinline__ void normalise(Eight (&e)[N], float (&r)[N], const QkArgs &a, float inv_d,
                                          bool mine) {
  if (a.norm == AG_NORM_NONE) return;
  float2 part[N];
  float s[N];
  if (a.norm == AG_NORM_LAYER) {
#pragma unroll
    for (int u = 0; u < N; ++u) part[u] = sum4(e[u]);
    row_sums<LPR, N>(part, s);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const float2 mean = twice(mine ? -s[u] * inv_d : 0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) e[u].v[i] = __fadd2_rn(e[u].v[i], mean);
    }
  }
#pragma unroll
  for (int u = 0; u < N; ++u) {
    part[u] = __fmul2_rn(e[u].v[0], e[u].v[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) part[u] = __ffma2_rn(e[u].v[i], e[u].v[i], part[u]);
  }
  row_sums<LPR, N>(part, s);
#pragma unroll
  for (int u = 0; u < N; ++u) {
    // (A group past the last position counts for nothing, also when eps is zero.)
    r[u] = mine ? __frsqrt_rn(fmaf(s[u], inv_d, a.eps)) : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) e[u].v[i] = __fmul2_rn(e[u].v[i], twice(r[u]));
  }
}

// What the rows of one side share in the forward.
template <int LPR, int XT, int OT, bool HALVES>
struct FwdRows {
  const QkArgs &a;
  const Lane &t;
  const float4 *cos4, *sin4;
  bool mine;
  float inv_d;
  int x_apart, o_apart;
  int64_t x_step, o_step;
  const char *x_at;
  char *o_at;
  Eight w, bias;

  // N rows from here on; `between` runs while their loads are on their way.
  template <int N, typename F>
  __device__ __forceinline__ void rows(F between) {
    Raw<XT> raw[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      raw[u] = Raw<XT>{};
      if (mine) raw[u] = load8<XT>(x_at, x_apart);
      x_at += x_step;
    }
    between();
    Eight x[N];
    float r[N];
#pragma unroll
    for (int u = 0; u < N; ++u) x[u] = widen<XT, HALVES>(raw[u]);
    normalise<LPR, N>(x, r, a, inv_d, mine);
#pragma unroll
    for (int u = 0; u < N; ++u) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[u].v[i] = __ffma2_rn(x[u].v[i], w.v[i], bias.v[i]);
      if (t.turns) turn_pairs<false>(x[u], cos4, sin4);
      if (mine) store8<OT, HALVES>(o_at, o_apart, x[u]);
      o_at += o_step;
    }
  }
};

// A block's side and its heads from blockIdx.y: kChunk heads at a time, the
// queries' first.
constexpr int kChunk = 4;
struct Heads {
  int which, first, count;
};
__device__ __forceinline__ Heads heads_of(const QkArgs &a) {
  const int of_q = (a.side[0].H + kChunk - 1) / kChunk, y = static_cast<int>(blockIdx.y);
  Heads h;
  h.which = y >= of_q;
  h.first = (h.which ? y - of_q : y) * kChunk;
  h.count = min(kChunk, a.side[h.which].H - h.first);
  return h;
}

// With one block row a block takes all heads of its positions, otherwise its
// chunk of them.
template <int LPR, int XT, int OT, bool HALVES>
__global__ void __launch_bounds__(kThreads, 4) qk_fwd_rows_kernel(const QkArgs a) {
  extern __shared__ float smem[];
  begin_after_previous();
  constexpr int kGroups = 32 / LPR, kRows = 2;   // positions per warp; rows side by side
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  float *cs = smem + (warp * kGroups + lane / LPR) * a.R;
  const float4 *cos4 = reinterpret_cast<const float4 *>(cs) + lane % LPR, *sin4 = cos4 + a.R / 8;
  const Lane t = lane_of<LPR, HALVES>(lane, a.D, a.R);
  const uint32_t L = static_cast<uint32_t>(a.L), total = static_cast<uint32_t>(a.positions_total);
  const uint32_t start = (blockIdx.x * kWarps + warp) * kGroups;  // the warp's first position
  if (start >= total) return;
  const uint32_t pos = min(start + lane / LPR, total - 1);
  const bool mine = t.in && start + lane / LPR < total;
  const int64_t b = pos / L, l = pos % L;
  const Heads part = heads_of(a);
  bool ready = a.R == 0;
  const auto angles = [&] {  // while the first rows are on their way
    if (!ready) group_angles<LPR, OT == AG_F32>(a, cs, b, l, lane);
    ready = true;
  };
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const QkSide &s = a.side[which];
    const int first = gridDim.y == 1 ? 0 : part.first;
    int left = gridDim.y == 1 ? s.H : which == part.which ? part.count : 0;
    if (left == 0) continue;
    FwdRows<LPR, XT, OT, HALVES> f{
        a, t, cos4, sin4, mine, 1.f / a.D, static_cast<int>(bytes_of<XT>(t.b - t.a)),
        static_cast<int>(bytes_of<OT>(t.b - t.a)), bytes_of<XT>(s.sh), bytes_of<OT>(a.L * a.D),
        static_cast<const char *>(s.x) + bytes_of<XT>(b * s.sb + l * s.sl + first * s.sh + t.a),
        static_cast<char *>(s.out) + bytes_of<OT>(((b * s.H + first) * a.L + l) * a.D + t.a),
        param8<HALVES>(s.w, t, 1.f), param8<HALVES>(s.b, t, 0.f)};
#pragma unroll 1
    for (; left >= kRows; left -= kRows) f.template rows<kRows>(angles);
    if (left > 0) f.template rows<1>(angles);
  }
}

// What the rows of one side share in the backward.
template <int LPR, int XT, int GT, bool HALVES>
struct BwdRows {
  const QkArgs &a;
  const Lane &t;
  const float4 *cos4, *sin4;
  bool mine;
  float inv_d;
  int x_apart, g_apart;
  int64_t x_step, g_step, dx_step;
  const char *x_at, *g_at;
  char *dx_at;
  Eight w, dw, db;

  template <int N, typename F>
  __device__ __forceinline__ void rows(F between) {
    Raw<XT> raw_x[N];
    Raw<GT> raw_g[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      raw_x[u] = Raw<XT>{}, raw_g[u] = Raw<GT>{};
      if (mine) {
        raw_x[u] = load8<XT>(x_at, x_apart);
        raw_g[u] = load8<GT>(g_at, g_apart);
      }
      x_at += x_step, g_at += g_step;
    }
    between();
    Eight x[N], g[N];
    float r[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      x[u] = widen<XT, HALVES>(raw_x[u]), g[u] = widen<GT, HALVES>(raw_g[u]);
      r[u] = 1.f;
    }
    normalise<LPR, N>(x, r, a, inv_d, mine);
    float2 dot[N];
    float along[N], mean[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      if (t.turns) turn_pairs<true>(g[u], cos4, sin4);
      if (a.partial)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dw.v[i] = __ffma2_rn(g[u].v[i], x[u].v[i], dw.v[i]);
          db.v[i] = __fadd2_rn(db.v[i], g[u].v[i]);
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) g[u].v[i] = __fmul2_rn(g[u].v[i], w.v[i]);
    }
    if (a.norm != AG_NORM_NONE) {
#pragma unroll
      for (int u = 0; u < N; ++u) {
        dot[u] = __fmul2_rn(g[u].v[0], x[u].v[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) dot[u] = __ffma2_rn(g[u].v[i], x[u].v[i], dot[u]);
      }
      row_sums<LPR, N>(dot, along);
      if (a.norm == AG_NORM_LAYER) {
#pragma unroll
        for (int u = 0; u < N; ++u) dot[u] = sum4(g[u]);
        row_sums<LPR, N>(dot, mean);
      } else {
#pragma unroll
        for (int u = 0; u < N; ++u) mean[u] = 0.f;
      }
#pragma unroll
      for (int u = 0; u < N; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          g[u].v[i] = __fmul2_rn(__fadd2_rn(__ffma2_rn(x[u].v[i], twice(-along[u] * inv_d), g[u].v[i]),
                                            twice(-mean[u] * inv_d)),
                                 twice(r[u]));
    }
#pragma unroll
    for (int u = 0; u < N; ++u) {
      if (mine) store8<XT, HALVES>(dx_at, x_apart, g[u]);
      dx_at += dx_step;
    }
  }
};

// Backward.  A block keeps to its heads and goes over positions.  A lane's
// elements are the same in every row it meets, so it sums the parameter
// gradients in registers; at the end the block adds its lanes' and warps', in a
// fixed order, and writes one partial [w, b][D].
template <int LPR, int XT, int GT, bool HALVES>
__global__ void __launch_bounds__(kThreads, 2) qk_bwd_rows_kernel(const QkArgs a) {
  extern __shared__ float smem[];
  begin_after_previous();
  constexpr int kGroups = 32 / LPR;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  float *cs = smem + (warp * kGroups + lane / LPR) * a.R;
  const float4 *cos4 = reinterpret_cast<const float4 *>(cs) + lane % LPR, *sin4 = cos4 + a.R / 8;
  const Lane t = lane_of<LPR, HALVES>(lane, a.D, a.R);
  const uint32_t L = static_cast<uint32_t>(a.L), total = static_cast<uint32_t>(a.positions_total);
  const Heads h = heads_of(a);
  const QkSide &s = a.side[h.which];
  BwdRows<LPR, XT, GT, HALVES> f{a, t, cos4, sin4, false, 1.f / a.D,
                                 static_cast<int>(bytes_of<XT>(t.b - t.a)),
                                 static_cast<int>(bytes_of<GT>(t.b - t.a)), bytes_of<XT>(s.sh),
                                 bytes_of<GT>(a.L * a.D), bytes_of<XT>(s.dxh), nullptr, nullptr,
                                 nullptr, param8<HALVES>(s.w, t, 1.f), Eight{}, Eight{}};
  const uint32_t stride = gridDim.x * kWarps * kGroups;
  for (uint32_t first = (blockIdx.x * kWarps + warp) * kGroups; first < total; first += stride) {
    const uint32_t pos = min(first + lane / LPR, total - 1);
    const int64_t b = pos / L, l = pos % L;
    f.mine = t.in && first + lane / LPR < total;
    f.x_at = static_cast<const char *>(s.x) +
             bytes_of<XT>(b * s.sb + l * s.sl + h.first * s.sh + t.a);
    f.g_at = static_cast<const char *>(s.g) +
             bytes_of<GT>(((b * s.H + h.first) * a.L + l) * a.D + t.a);
    f.dx_at = static_cast<char *>(s.dx) +
              bytes_of<XT>(b * s.dxb + l * s.dxl + h.first * s.dxh + t.a);
    const auto angles = [&] {
      if (a.R) group_angles<LPR, XT == AG_F32>(a, cs, b, l, lane);
    };
    if (h.count == kChunk) {
      f.template rows<kChunk>(angles);
    } else {
      f.template rows<1>(angles);
#pragma unroll 1
      for (int i = 1; i < h.count; ++i) f.template rows<1>([] {});
    }
  }
  if (!a.partial) return;
  float4 *sums = reinterpret_cast<float4 *>(smem + kWarps * kGroups * a.R);  // [kWarps][4][32]
#pragma unroll
  for (int q = 0; q < 4; ++q) {  // w and b, A and B
    const float2 *v = (q < 2 ? f.dw.v : f.db.v) + 2 * (q & 1);
    sums[(warp * 4 + q) * 32 + lane] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.D; i += kThreads) {
    // Element e of w or b: number `at` of A or B of lane `l` (lane_of).
    const int which = i / a.D, e = i % a.D;
    int l = e / 8, second = HALVES ? (e % 8) / 4 : e % 2, at = HALVES ? e % 4 : e % 8 / 2;
    if (HALVES && e < a.R) {
      const int pair = e % (a.R / 2);
      l = pair / 4, at = pair % 4, second = e / (a.R / 2);
    }
    const float *from = reinterpret_cast<const float *>(sums + (which * 2 + second) * 32 + l) + at;
    float v = 0.f;
    for (int w = 0; w < kWarps; ++w)
#pragma unroll
      for (int row = 0; row < kGroups; ++row) v += from[(w * 4 * 32 + row * LPR) * 4];
    a.partial[(static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * 2 * a.D + i] = v;
  }
}

// --------------------------------------------------------------------------
// General kernels.  One warp per (position, head) row, any D and any strides.
// Row t of a block's positions from p0 on: all heads of each position in turn.
struct Row {
  int which, h, p;
  int64_t b, l;
};
// (Positions and rows are below 2^31: the divisions are of 32 bits.)
__device__ __forceinline__ Row row_of(const QkArgs &a, uint32_t p0, int t, int heads) {
  Row w;
  w.p = static_cast<uint32_t>(t) / static_cast<uint32_t>(heads);
  w.h = t - w.p * heads;
  w.which = w.h >= a.side[0].H;
  if (w.which) w.h -= a.side[0].H;
  const uint32_t pos = p0 + w.p, L = static_cast<uint32_t>(a.L);
  w.b = pos / L;
  w.l = pos % L;
  return w;
}
// Blocks to an SM.
constexpr int kGeneralBlocks = 6;

// A row into shared memory, four loads of a lane at a time on their way.
template <int T>
__device__ __forceinline__ void load_row_to(float *row, const void *x, int64_t at, int D,
                                            int lane) {
  for (int i = lane; i < D; i += 128) {
    float v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = i + 32 * u < D ? load_one<T>(x, at + i + 32 * u) : 0.f;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + 32 * u < D) row[i + 32 * u] = v[u];
  }
}
// The angles of np positions, by the whole block.
template <bool EXACT>
__device__ __forceinline__ void block_angles(const QkArgs &a, float2 *cs, uint32_t p0, int np,
                                             int half) {
  const uint32_t L = static_cast<uint32_t>(a.L);
  for (int i = threadIdx.x; i < np * half; i += blockDim.x) {
    const uint32_t p = static_cast<uint32_t>(i) / static_cast<uint32_t>(half), pos = p0 + p;
    const int64_t b = pos / L, l = pos % L;
    cs[i] = turn<EXACT>(a.positions ? a.positions[b * a.pos_sb + l] : l, a.inv_freq[i - p * half]);
  }
}

template <int XT, int OT>
__global__ void __launch_bounds__(kThreads, kGeneralBlocks) qk_fwd_kernel(const QkArgs a, int at_once) {
  extern __shared__ float smem[];
  begin_after_previous();
  const int half = a.R >> 1, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  float2 *cs = reinterpret_cast<float2 *>(smem);
  float *row = smem + 2 * at_once * half + warp * a.D;
  const uint32_t p0 = blockIdx.x * at_once;
  const int np = static_cast<int>(min(static_cast<int64_t>(at_once), a.positions_total - p0));
  const int heads = a.side[0].H + a.side[1].H, rows = np * heads;
  Row w;
  const auto load = [&](int t) {
    w = row_of(a, p0, t, heads);
    const QkSide &s = a.side[w.which];
    load_row_to<XT>(row, s.x, w.b * s.sb + w.l * s.sl + w.h * s.sh, a.D, lane);
  };
  if (warp < rows) load(warp);  // (on its way while the angles are formed)
  block_angles<OT == AG_F32>(a, cs, p0, np, half);
  __syncthreads();
  for (int t = warp; t < rows; t += kWarps) {
    if (t != warp) load(t);
    const QkSide &s = a.side[w.which];
    float mean, r;
    row_stats(row, a.D, a.norm, a.eps, lane, mean, r);
    for (int i = lane; i < a.D; i += 32) {
      float v = (row[i] - mean) * r;
      if (s.w) v *= s.w[i];
      if (s.b) v += s.b[i];
      row[i] = v;
    }
    __syncwarp();
    const int64_t to = ((w.b * s.H + w.h) * a.L + w.l) * a.D;
    for (int i = lane; i < a.D; i += 32) {
      float v = row[i];
      if (i < a.R) {
        const Pair q = pair_of(i, a.R, a.rope);
        const float2 c = cs[w.p * half + q.angle];
        v = fmaf(v, c.x, q.second ? row[q.other] * c.y : -row[q.other] * c.y);
      }
      store_one<OT>(s.out, to + i, v);
    }
    __syncwarp();
  }
}

// Backward: the same rows.  Each warp adds its rows' parameter gradients to
// its own part of shared memory (element i always by lane i % 32: no atomics),
// the block then adds its warps' in order and writes one partial per block;
// qk_params_kernel adds those.
template <int XT, int GT>
__global__ void __launch_bounds__(kThreads, kGeneralBlocks) qk_bwd_kernel(const QkArgs a, int warps, int at_once) {
  extern __shared__ float smem[];
  begin_after_previous();
  const int half = a.R >> 1, warp = threadIdx.x / 32, lane = threadIdx.x % 32, D = a.D;
  float2 *cs = reinterpret_cast<float2 *>(smem);
  float *row = smem + 2 * at_once * half + warp * 3 * D, *grad = row + D, *back = grad + D;
  float *sums = smem + 2 * at_once * half + warps * 3 * D;  // [warps][2 sides][w, b][D]
  float *own = sums + warp * 4 * D;
  for (int i = lane; i < 4 * D; i += 32) own[i] = 0.f;
  const int heads = a.side[0].H + a.side[1].H;
  // (positions_total < 2^31 and a grid's turn is below 2^16: p0 stays in 32 bits)
  for (uint32_t p0 = blockIdx.x * at_once; p0 < a.positions_total; p0 += gridDim.x * at_once) {
    const int np = static_cast<int>(min(static_cast<int64_t>(at_once), a.positions_total - p0));
    const int rows = np * heads;
    Row w;
    const auto load = [&](int t) {
      w = row_of(a, p0, t, heads);
      const QkSide &s = a.side[w.which];
      load_row_to<XT>(row, s.x, w.b * s.sb + w.l * s.sl + w.h * s.sh, D, lane);
      load_row_to<GT>(grad, s.g, ((w.b * s.H + w.h) * a.L + w.l) * D, D, lane);
    };
    if (warp < rows) load(warp);  // (on its way while the angles are formed)
    __syncthreads();              // the angles of the turn before are no longer read
    block_angles<XT == AG_F32>(a, cs, p0, np, half);
    __syncthreads();
    for (int t = warp; t < rows; t += warps) {
      if (t != warp) load(t);
      const QkSide &s = a.side[w.which];
      float mean, r;
      row_stats(row, D, a.norm, a.eps, lane, mean, r);
      __syncwarp();
      float along = 0.f, total = 0.f;
      for (int i = lane; i < D; i += 32) {
        float g = grad[i];
        if (i < a.R) {
          const Pair q = pair_of(i, a.R, a.rope);
          const float2 c = cs[w.p * half + q.angle];
          g = fmaf(g, c.x, q.second ? -grad[q.other] * c.y : grad[q.other] * c.y);
        }
        const float n = (row[i] - mean) * r;
        if (a.partial) own[w.which * 2 * D + i] += g * n, own[w.which * 2 * D + D + i] += g;
        const float d = s.w ? g * s.w[i] : g;
        row[i] = n, back[i] = d;  // (an element stays with its lane)
        along = fmaf(d, n, along);
        total += d;
      }
      along = a.norm == AG_NORM_NONE ? 0.f : warp_sum(along) / D;
      total = a.norm == AG_NORM_LAYER ? warp_sum(total) / D : 0.f;
      const int64_t to = w.b * s.dxb + w.l * s.dxl + w.h * s.dxh;
      for (int i = lane; i < D; i += 32)
        store_one<XT>(s.dx, to + i, r * (back[i] - row[i] * along - total));
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

// The parameter gradients: side `blockIdx.y`'s sums of partials [w, b][D], `step`
// floats apart, `count` of them from `first` on; 32 columns per block, 32 warps
// over the partials, in 64 bits and a fixed order.
struct Partials {
  int64_t first[2];
  int count[2], step;
};
__global__ void __launch_bounds__(1024)
    qk_params_kernel(const float *partial, Partials p, int D, float *qw, float *qb, float *kw,
                     float *kb) {
  __shared__ double part[32][32];
  begin_after_previous();
  const int c = threadIdx.x % 32, r = threadIdx.x / 32, n = blockIdx.x * 32 + c;
  const int side = blockIdx.y;
  double t = 0.0;
  if (n < 2 * D)
    for (int i = r; i < p.count[side]; i += 32)
      t += partial[p.first[side] + static_cast<int64_t>(i) * p.step + n];
  part[r][c] = t;
  __syncthreads();
  if (r != 0 || n >= 2 * D) return;
  for (int i = 1; i < 32; ++i) t += part[i][c];
  float *to = side == 0 ? (n < D ? qw : qb) : (n < D ? kw : kb);
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
    if (!quads(s.x, a.x_dtype, s.sb, s.sl, s.sh) || !aligned(s.w, 16) || !aligned(s.b, 16))
      return false;
    if (backward ? !quads(s.g, a.o_dtype, 0, 0, 0) || !quads(s.dx, a.x_dtype, s.dxb, s.dxl, s.dxh)
                 : !quads(s.out, a.o_dtype, 0, 0, 0))
      return false;
  }
  return true;
}

int chunks_of(const QkArgs &a, int side) { return (a.side[side].H + kChunk - 1) / kChunk; }

int bwd_warps(int D) { return D <= 512 ? 8 : 4; }
// Positions a turn of the general kernels: a row to each of 8 warps.
int positions_at_once(int heads) { return heads >= 8 ? 1 : (8 + heads - 1) / heads; }
// Blocks along the positions of a backward, and so of its partial sums: of the
// rows kernel with `chunks` chunks of heads, two to an SM; of the general one,
// six; but no more than have work.
int64_t blocks_for(int64_t total, int64_t each, int64_t most) {
  const int64_t turns = (total + each - 1) / each;
  return turns < most ? turns : most < 1 ? 1 : most;
}
int64_t rows_blocks(int64_t total, int D, int chunks, int num_sms) {
  return blocks_for(total, kWarps * (D <= 64 ? 4 : D <= 128 ? 2 : 1), 2 * num_sms / chunks);
}
int64_t general_blocks(int64_t total, int heads, int num_sms) {
  return blocks_for(total, positions_at_once(heads), kGeneralBlocks * num_sms);
}

// The most that the general kernels take: angles of 8 positions of 1024 elements,
// and seven rows of 1024 for each of 4 warps (of 512 for 8).
constexpr int kMostSmem = (8 * 1024 + 7 * 4 * 1024) * 4;
// Always the same limit: a call's own would be taken back by a smaller call of
// another thread before its launch.
cudaError_t allow_smem(const void *kernel, size_t bytes) {
  return bytes <= 48 * 1024 ? cudaSuccess
                            : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kMostSmem);
}

}  // namespace

// The larger of what the two kinds of kernel write (which of them runs hangs on
// addresses that the query does not see).
int64_t qk_bwd_workspace(int64_t positions_total, int Hq, int Hk, int D, int num_sms) {
  const int chunks = (Hq + kChunk - 1) / kChunk + (Hk + kChunk - 1) / kChunk;
  const int64_t rows = rows_blocks(positions_total, D, chunks, num_sms) * chunks * 2 * D,
                general = general_blocks(positions_total, Hq + Hk, num_sms) * 4 * D;
  return (rows > general ? rows : general) * 4;
}

namespace {

// Positions that a warp of the rows kernels takes.
int groups_of(int D) { return D <= 64 ? 4 : D <= 128 ? 2 : 1; }
using QkKernel = void (*)(QkArgs);
template <int XT, int OT, bool HALVES>
QkKernel rows_kernel(int D, bool backward) {
  if (backward)
    return D <= 64    ? qk_bwd_rows_kernel<8, XT, OT, HALVES>
           : D <= 128 ? qk_bwd_rows_kernel<16, XT, OT, HALVES>
                      : qk_bwd_rows_kernel<32, XT, OT, HALVES>;
  return D <= 64    ? qk_fwd_rows_kernel<8, XT, OT, HALVES>
         : D <= 128 ? qk_fwd_rows_kernel<16, XT, OT, HALVES>
                    : qk_fwd_rows_kernel<32, XT, OT, HALVES>;
}
template <int XT, bool HALVES>
QkKernel rows_kernel(const QkArgs &a, bool backward) {
  return a.o_dtype == AG_F32    ? rows_kernel<XT, AG_F32, HALVES>(a.D, backward)
         : a.o_dtype == AG_BF16 ? rows_kernel<XT, AG_BF16, HALVES>(a.D, backward)
                                : rows_kernel<XT, AG_F16, HALVES>(a.D, backward);
}
template <bool HALVES>
QkKernel rows_kernel(const QkArgs &a, bool backward) {
  return a.x_dtype == AG_F32    ? rows_kernel<AG_F32, HALVES>(a, backward)
         : a.x_dtype == AG_BF16 ? rows_kernel<AG_BF16, HALVES>(a, backward)
                                : rows_kernel<AG_F16, HALVES>(a, backward);
}
QkKernel rows_kernel(const QkArgs &a, bool backward) {
  return a.rope == AG_ROPE_HALVES ? rows_kernel<true>(a, backward) : rows_kernel<false>(a, backward);
}

// The general kernels by type.
template <int XT>
void (*general_fwd(const QkArgs &a))(QkArgs, int) {
  return a.o_dtype == AG_F32    ? qk_fwd_kernel<XT, AG_F32>
         : a.o_dtype == AG_BF16 ? qk_fwd_kernel<XT, AG_BF16>
                                : qk_fwd_kernel<XT, AG_F16>;
}
template <int XT>
void (*general_bwd(const QkArgs &a))(QkArgs, int, int) {
  return a.o_dtype == AG_F32    ? qk_bwd_kernel<XT, AG_F32>
         : a.o_dtype == AG_BF16 ? qk_bwd_kernel<XT, AG_BF16>
                                : qk_bwd_kernel<XT, AG_F16>;
}

}  // namespace

cudaError_t launch_qk_fwd(const QkArgs &a, int num_sms, cudaStream_t stream) {
  if (by_rows(a, false)) {
    const int each = kWarps * groups_of(a.D);
    // Few positions do not fill the GPU: their heads are then spread over blocks
    // (4 positions of 8 + 1 heads 2.7 us against 4.9; but 16384 positions 26 us
    // against 20.4, each chunk forming its positions' angles again).
    const int64_t blocks = (a.positions_total + each - 1) / each;
    const dim3 grid(static_cast<unsigned>(blocks),
                    blocks < num_sms ? chunks_of(a, 0) + chunks_of(a, 1) : 1);
    return launch_after_previous(rows_kernel(a, false), grid, kThreads, each * a.R * 4, stream, a);
  }
  const int at_once = positions_at_once(a.side[0].H + a.side[1].H);
  const size_t smem = (static_cast<size_t>(at_once) * a.R + kWarps * static_cast<size_t>(a.D)) * 4;
  const auto kernel = a.x_dtype == AG_F32    ? general_fwd<AG_F32>(a)
                      : a.x_dtype == AG_BF16 ? general_fwd<AG_BF16>(a)
                                             : general_fwd<AG_F16>(a);
  cudaError_t e = allow_smem(reinterpret_cast<const void *>(kernel), smem);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (a.positions_total + at_once - 1) / at_once;
  return launch_after_previous(kernel, static_cast<unsigned>(blocks), kThreads, smem, stream,
                               a, at_once);
}

cudaError_t launch_qk_bwd(const QkArgs &a, int num_sms, cudaStream_t stream) {
  Partials p;
  cudaError_t e;
  if (by_rows(a, true)) {
    const int of_q = chunks_of(a, 0), chunks = of_q + chunks_of(a, 1);
    const int blocks = static_cast<int>(rows_blocks(a.positions_total, a.D, chunks, num_sms));
    const int groups = kWarps * groups_of(a.D);
    e = launch_after_previous(rows_kernel(a, true), dim3(blocks, chunks), kThreads,
                              (groups * a.R + kWarps * 4 * 32 * 4) * 4, stream, a);
    p.first[0] = 0, p.count[0] = of_q * blocks;
    p.first[1] = static_cast<int64_t>(of_q) * blocks * 2 * a.D, p.count[1] = (chunks - of_q) * blocks;
    p.step = 2 * a.D;
  } else {
    const int heads = a.side[0].H + a.side[1].H;
    const int warps = bwd_warps(a.D), at_once = positions_at_once(heads);
    const int blocks = static_cast<int>(general_blocks(a.positions_total, heads, num_sms));
    const size_t smem =
        (static_cast<size_t>(at_once) * a.R + warps * 7 * static_cast<size_t>(a.D)) * 4;
    const auto kernel = a.x_dtype == AG_F32    ? general_bwd<AG_F32>(a)
                        : a.x_dtype == AG_BF16 ? general_bwd<AG_BF16>(a)
                                               : general_bwd<AG_F16>(a);
    e = allow_smem(reinterpret_cast<const void *>(kernel), smem);
    if (e != cudaSuccess) return e;
    e = launch_after_previous(kernel, blocks, warps * 32, smem, stream, a, warps, at_once);
    p.first[0] = 0, p.first[1] = 2 * a.D;
    p.count[0] = p.count[1] = blocks;
    p.step = 4 * a.D;
  }
  if (e != cudaSuccess || !a.partial) return e;
  return launch_after_previous(qk_params_kernel, dim3((2 * a.D + 31) / 32, 2), 1024, 0, stream,
                               a.partial, p, a.D, a.side[0].dw, a.side[0].db, a.side[1].dw,
                               a.side[1].db);
}

}  // namespace ag
