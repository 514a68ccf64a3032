// ag_layers_api.cu -- the extern "C" entry points of the layers around the
// attention (include/ag.h): linear layers, query and key norm with rotation,
// gradient clipping.  As in ag_api.cu, everything is checked on the host
// before anything is launched.
#include <algorithm>
#include <cmath>
#include <cstdlib>

#include "ag_internal.h"

namespace ag {
namespace {

constexpr int64_t kMaxRows = int64_t(1) << 26, kMaxCols = int64_t(1) << 20,
                  kMaxStride = int64_t(1) << 28, kMaxMatrix = int64_t(1) << 38;

bool is_dtype(int d) { return d == AG_F32 || d == AG_BF16 || d == AG_F16; }
int size_of(int d) { return d == AG_F32 ? 4 : 2; }

// A row-major matrix argument: rows x cols elements of `size` bytes, ld apart.
struct Mat {
  const void *p;
  int64_t rows, cols, ld;
  int size;
  uint64_t row_bytes() const { return static_cast<uint64_t>(cols) * size; }
  uint64_t ld_bytes() const { return static_cast<uint64_t>(ld) * size; }
  uint64_t span() const { return rows > 0 ? (rows - 1) * ld_bytes() + row_bytes() : 0; }
};

// Whether two matrices share an address.  With equal row strides (two column
// ranges of one wider matrix) this is exact; otherwise it goes by their spans.
bool mats_overlap(const Mat &a, const Mat &b) {
  if (!a.p || !b.p || !overlap(a.p, a.span(), b.p, b.span())) return false;
  if (a.ld_bytes() != b.ld_bytes()) return true;
  const uint64_t ld = a.ld_bytes();
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  const uint64_t d = y >= x ? (y - x) % ld : (ld - (x - y) % ld) % ld;  // b's column after a's
  return !(d >= a.row_bytes() && d + b.row_bytes() <= ld);
}

// Row strides: at least the row, at most kMaxStride.  Of one row the stride is
// never used, so any will do (the last position of a long sequence, say): a
// longer one becomes a plain one.
ag_status check_ld(int64_t &ld, int64_t rows, int64_t cols) {
  if (ld < cols) return AG_ERR_SHAPE;
  if (ld > kMaxStride && rows <= 1) ld = (cols + 7) / 8 * 8;
  return ld > kMaxStride ? AG_ERR_UNSUPPORTED : AG_OK;
}

ag_status check_linear_sizes(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 1 || K < 1) return AG_ERR_SHAPE;
  if (M > kMaxRows || N > kMaxCols || K > kMaxCols) return AG_ERR_UNSUPPORTED;
  // Keeps a product's tiles (of at least 2^15 outputs, in up to 32 splits)
  // below 2^31; the longest sum, over M, has at most 2^20 64-deep tiles.
  if (M * N > kMaxMatrix || M * K > kMaxMatrix || N * K > kMaxMatrix) return AG_ERR_UNSUPPORTED;
  return AG_OK;
}

bool is_half(int d) { return d == AG_BF16 || d == AG_F16; }

// Whether rows of the matrix can be read and written in 16-byte groups of
// 8 columns (two of them for float32).
bool vec8(const void *p, int64_t ld, int size) {
  return !p || (aligned(p, 16) && (ld * size) % 16 == 0);
}

struct Device {
  DeviceInfo *info = nullptr;
  EncodeTiledFn encode = nullptr;
};
ag_status device_and_encoder(Device *d) {
  const ag_status st = device_info(&d->info);
  return st != AG_OK ? st : get_encoder(&d->encode);
}

}  // namespace
}  // namespace ag

using ag::Mat;

extern "C" {

ag_status ag_linear_fwd_workspace(const void *x, int64_t ldx, const void *W, int64_t ldw,
                                  int64_t M, int64_t N, int64_t K, int64_t *bytes) {
  if (!bytes) return AG_ERR_NULL;
  ag_status st = ag::check_linear_sizes(M, N, K);
  if (st == AG_OK) st = ag::check_ld(ldx, M, K);
  if (st == AG_OK) st = ag::check_ld(ldw, N, K);
  if (st != AG_OK) return st;
  *bytes = 0;
  if (M == 0) return AG_OK;
  ag::DeviceInfo *dev = nullptr;
  st = ag::device_info(&dev);
  if (st != AG_OK) return st;
  ag::LinearFwd a{};
  a.x = x, a.W = W, a.ldx = ldx, a.ldw = ldw, a.M = M, a.N = N, a.K = K;
  a.num_sms = dev->num_sms;
  return ag::from_cuda(ag::linear_fwd_workspace(a, bytes));
}

ag_status ag_linear_fwd(const void *x, int64_t ldx, const void *W, int64_t ldw,
                        const float *bias, const void *residual, int64_t ldr, int64_t M,
                        int64_t N, int64_t K, int dtype, int act, void *preact, int64_t ldz,
                        void *y, int64_t ldy, int y_dtype, void *workspace,
                        int64_t workspace_bytes, void *stream) {
  ag_status st = ag::check_linear_sizes(M, N, K);
  if (st == AG_OK) st = ag::check_ld(ldx, M, K);
  if (st == AG_OK) st = ag::check_ld(ldw, N, K);
  if (st == AG_OK) st = ag::check_ld(ldy, M, N);
  if (st == AG_OK && residual) st = ag::check_ld(ldr, M, N);
  if (st == AG_OK && preact) st = ag::check_ld(ldz, M, N);
  if (st != AG_OK) return st;
  if (!ag::is_half(dtype) || (y_dtype != dtype && y_dtype != AG_F32) || act < AG_ACT_NONE ||
      act > AG_ACT_SILU)
    return AG_ERR_VALUE;
  if (M == 0) return AG_OK;
  if (!x || !W || !y) return AG_ERR_NULL;
  const int es = ag::size_of(dtype), os = ag::size_of(y_dtype);
  if (!ag::aligned(x, es) || !ag::aligned(W, es) || !ag::aligned(y, os) ||
      !ag::aligned(bias, 4) || !ag::aligned(residual, os) || !ag::aligned(preact, es) ||
      !ag::aligned(workspace, 256))
    return AG_ERR_ALIGN;
  const Mat mx{x, M, K, ldx, es}, mw{W, N, K, ldw, es}, mb{bias, 1, N, N, 4},
      mr{residual, M, N, ldr, os}, my{y, M, N, ldy, os}, mz{preact, M, N, ldz, es};
  const bool in_place = residual == y && ldr == ldy;
  for (const Mat *in : {&mx, &mw, &mb, &mr}) {
    if (ag::mats_overlap(mz, *in)) return AG_ERR_ALIAS;
    if (!(in == &mr && in_place) && ag::mats_overlap(my, *in)) return AG_ERR_ALIAS;
  }
  if (ag::mats_overlap(my, mz)) return AG_ERR_ALIAS;
  ag::Device dev;
  st = ag::device_and_encoder(&dev);
  if (st != AG_OK) return st;
  ag::LinearFwd a{};
  a.x = x, a.W = W, a.ldx = ldx, a.ldw = ldw, a.M = M, a.N = N, a.K = K;
  a.epi.bias = bias;
  a.epi.pre_out = preact, a.epi.ld_pre_out = ldz;
  a.epi.residual = residual, a.epi.ld_res = ldr;
  a.epi.out = y, a.epi.ld_out = ldy;
  a.epi.act = act, a.epi.dtype = dtype, a.epi.out_dtype = y_dtype;
  a.epi.vec8 = N % 8 == 0 && ag::vec8(y, ldy, os) && ag::vec8(residual, ldr, os) &&
               ag::vec8(preact, ldz, es);
  a.workspace = workspace;
  a.num_sms = dev.info->num_sms, a.err = dev.info->err, a.encode = dev.encode;
  a.stream = static_cast<cudaStream_t>(stream);
  int64_t need = 0;
  st = ag::from_cuda(ag::linear_fwd_workspace(a, &need));
  if (st != AG_OK) return st;
  if (need > 0 && (!workspace || workspace_bytes < need)) return AG_ERR_SCRATCH;
  const Mat ms{need > 0 ? workspace : nullptr, 1, need, need, 1};
  for (const Mat *m : {&mx, &mw, &mb, &mr, &my, &mz})
    if (ag::mats_overlap(ms, *m)) return AG_ERR_ALIAS;
  return ag::from_cuda(ag::launch_linear_fwd(a));
}

ag_status ag_linear_bwd_workspace(const void *dy, int64_t lddy, const void *x, int64_t ldx,
                                  const void *W, int64_t ldw, int64_t M, int64_t N, int64_t K,
                                  const void *dx, const void *dW, const float *db,
                                  int64_t *bytes) {
  if (!bytes) return AG_ERR_NULL;
  ag_status st = ag::check_linear_sizes(M, N, K);
  if (st == AG_OK) st = ag::check_ld(lddy, M, N);
  if (st == AG_OK && dW) st = ag::check_ld(ldx, M, K);
  if (st == AG_OK && dx) st = ag::check_ld(ldw, N, K);
  if (st != AG_OK) return st;
  *bytes = 0;
  if (M == 0) return AG_OK;
  ag::DeviceInfo *dev = nullptr;
  st = ag::device_info(&dev);
  if (st != AG_OK) return st;
  ag::LinearBwd a{};
  a.dy = dy, a.x = x, a.W = W, a.lddy = lddy, a.ldx = ldx, a.ldw = ldw;
  a.M = M, a.N = N, a.K = K;
  a.dx.out = const_cast<void *>(dx), a.dW.out = const_cast<void *>(dW);
  a.db = const_cast<float *>(db);
  a.num_sms = dev->num_sms;
  return ag::from_cuda(ag::linear_bwd_workspace(a, bytes));
}

ag_status ag_linear_bwd(const void *dy, int64_t lddy, const void *x, int64_t ldx,
                        const void *W, int64_t ldw, const void *preact, int64_t ldz, int act,
                        int64_t M, int64_t N, int64_t K, int dtype, void *dx, int64_t lddx,
                        int dx_dtype, void *dW, int64_t lddw, int dW_dtype, float *db,
                        void *workspace, int64_t workspace_bytes, void *stream) {
  ag_status st = ag::check_linear_sizes(M, N, K);
  if (st == AG_OK) st = ag::check_ld(lddy, M, N);
  if (st == AG_OK && dW) st = ag::check_ld(ldx, M, K);
  if (st == AG_OK && dW) st = ag::check_ld(lddw, N, K);
  if (st == AG_OK && dx) st = ag::check_ld(ldw, N, K);
  if (st == AG_OK && dx) st = ag::check_ld(lddx, M, K);
  if (st == AG_OK && dx && preact) st = ag::check_ld(ldz, M, K);
  if (st != AG_OK) return st;
  if (!ag::is_half(dtype) || act < AG_ACT_NONE || act > AG_ACT_SILU ||
      (dx && dx_dtype != dtype && dx_dtype != AG_F32) ||
      (dW && dW_dtype != dtype && dW_dtype != AG_F32) || (dx && act != AG_ACT_NONE && !preact))
    return AG_ERR_VALUE;
  const int es = ag::size_of(dtype), xs = ag::size_of(dx_dtype), ws = ag::size_of(dW_dtype);
  if ((dW && !ag::aligned(dW, ws)) || !ag::aligned(db, 4)) return AG_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {
    // No rows: the sums over them are zero.
    if (!dW && !db) return AG_OK;
    const Mat mw{dW, N, K, lddw, ws}, mb{db, 1, N, N, 4};
    if (ag::mats_overlap(mw, mb)) return AG_ERR_ALIAS;
    ag::DeviceInfo *dev = nullptr;
    st = ag::device_info(&dev);
    if (st != AG_OK) return st;
    cudaError_t e = cudaSuccess;
    if (dW) e = cudaMemset2DAsync(dW, mw.ld_bytes(), 0, mw.row_bytes(), N, s);
    if (db && e == cudaSuccess) e = cudaMemsetAsync(db, 0, N * 4, s);
    return ag::from_cuda(e);
  }
  if (!dx && !dW && !db) return AG_OK;
  if (!dy || (dW && !x) || (dx && !W)) return AG_ERR_NULL;
  if (!ag::aligned(dy, es) || (dW && !ag::aligned(x, es)) || (dx && !ag::aligned(W, es)) ||
      (dx && !ag::aligned(preact, es)) || (dx && !ag::aligned(dx, xs)) ||
      !ag::aligned(workspace, 256))
    return AG_ERR_ALIGN;
  const bool slope = dx && act != AG_ACT_NONE;
  const Mat mdy{dy, M, N, lddy, es}, mx{dW ? x : nullptr, M, K, ldx, es},
      mw{dx ? W : nullptr, N, K, ldw, es}, mz{slope ? preact : nullptr, M, K, ldz, es},
      mdx{dx, M, K, lddx, xs}, mdw{dW, N, K, lddw, ws}, mdb{db, 1, N, N, 4};
  const Mat *outs[3] = {&mdx, &mdw, &mdb};
  for (int o = 0; o < 3; ++o) {
    for (const Mat *in : {&mdy, &mx, &mw, &mz})
      if (ag::mats_overlap(*outs[o], *in)) return AG_ERR_ALIAS;
    for (int u = o + 1; u < 3; ++u)
      if (ag::mats_overlap(*outs[o], *outs[u])) return AG_ERR_ALIAS;
  }
  ag::Device dev;
  st = ag::device_and_encoder(&dev);
  if (st != AG_OK) return st;
  ag::LinearBwd a{};
  a.dy = dy, a.x = x, a.W = W, a.lddy = lddy, a.ldx = ldx, a.ldw = ldw;
  a.M = M, a.N = N, a.K = K, a.db = db;
  a.dx.pre_in = slope ? preact : nullptr, a.dx.ld_pre_in = ldz, a.dx.act = act;
  a.dx.out = dx, a.dx.ld_out = lddx, a.dx.dtype = dtype, a.dx.out_dtype = dx_dtype;
  a.dx.vec8 = K % 8 == 0 && ag::vec8(dx, lddx, xs) && ag::vec8(a.dx.pre_in, ldz, es);
  a.dW.out = dW, a.dW.ld_out = lddw, a.dW.dtype = dtype, a.dW.out_dtype = dW_dtype;
  a.dW.act = AG_ACT_NONE;
  a.dW.vec8 = K % 8 == 0 && ag::vec8(dW, lddw, ws);
  a.workspace = workspace;
  a.num_sms = dev.info->num_sms, a.err = dev.info->err, a.encode = dev.encode;
  a.stream = s;
  int64_t need = 0;
  st = ag::from_cuda(ag::linear_bwd_workspace(a, &need));
  if (st != AG_OK) return st;
  if (need > 0 && (!workspace || workspace_bytes < need)) return AG_ERR_SCRATCH;
  const Mat ms{need > 0 ? workspace : nullptr, 1, need, need, 1};
  for (const Mat *m : {&mdy, &mx, &mw, &mz, &mdx, &mdw, &mdb})
    if (ag::mats_overlap(ms, *m)) return AG_ERR_ALIAS;
  return ag::from_cuda(ag::launch_linear_bwd(a));
}

}  // extern "C"

namespace ag {
namespace {

// A [B, L, H, D] argument with element strides over b, l, h and dense D.
struct Heads {
  const void *p;
  int64_t n[3], s[3];  // sizes and strides of b, l, h
  int64_t D;
  int size;
  bool empty() const { return n[0] == 0 || n[1] == 0 || n[2] == 0; }
  // Elements from the first to the last, both included.
  int64_t extent() const {
    int64_t e = D;
    for (int i = 0; i < 3; ++i) e += (n[i] - 1) * s[i];
    return e;
  }
  uint64_t bytes() const { return empty() ? 0 : static_cast<uint64_t>(extent()) * size; }
};

// No dimension spans more than this many elements, so that offsets and byte
// ranges stay far below 2^63.
constexpr int64_t kMaxSpan = int64_t(1) << 50;
bool span_too_long(int64_t n, int64_t stride) { return n > 1 && stride > kMaxSpan / (n - 1); }

ag_status check_strides(const Heads &h) {
  if (h.empty()) return AG_OK;
  for (int i = 0; i < 3; ++i) {
    if (h.s[i] < 0) return AG_ERR_SHAPE;
    if (span_too_long(h.n[i], h.s[i])) return AG_ERR_UNSUPPORTED;
  }
  return AG_OK;
}

// Whether every element has an address of its own: taken from the smallest
// stride up, each dimension steps over all that lies inside it.
bool distinct(const Heads &h) {
  if (h.empty()) return true;
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int a, int b) { return h.s[a] < h.s[b]; });
  int64_t inner = h.D;
  for (int i : order) {
    if (h.n[i] == 1) continue;
    if (h.s[i] < inner) return false;
    inner += (h.n[i] - 1) * h.s[i];
  }
  return true;
}

bool heads_overlap(const Heads &a, const Heads &b) {
  return overlap(a.p, a.bytes(), b.p, b.bytes());
}

// Dimensions of more than one index, from the largest stride down.
struct Dims {
  int n = 0;
  int64_t count[3], stride[3];
  explicit Dims(const Heads &h) {
    for (int i = 0; i < 3; ++i) {
      if (h.n[i] == 1) continue;
      int at = n++;
      for (; at > 0 && stride[at - 1] < h.s[i]; --at)
        count[at] = count[at - 1], stride[at] = stride[at - 1];
      count[at] = h.n[i], stride[at] = h.s[i];
    }
  }
  // Elements from the first to the last that the dimensions from `from` on span.
  int64_t extent(int from, int64_t D) const {
    int64_t e = D;
    for (int i = from; i < n; ++i) e += (count[i] - 1) * stride[i];
    return e;
  }
};

// The most pairs of slices of two outputs that are compared.
constexpr int kMostPairs = 4096;

// Whether the runs of D elements of a (dimensions from ia on, starting at 0) and
// of b (from ib on, starting at `gap`) share no element.  Both step over what lies
// inside a dimension (distinct), so of two dimensions with one stride only
// neighbouring slices can meet.  Unequal strides where more than `left` pairs of
// slices might meet count as sharing one.
bool apart(const Dims &a, int ia, const Dims &b, int ib, int64_t gap, int64_t D, int &left) {
  if (left-- <= 0) return false;
  if (gap >= a.extent(ia, D) || gap + b.extent(ib, D) <= 0) return true;
  const bool in_a = ia < a.n, in_b = ib < b.n;
  if (!in_a && !in_b) return false;
  const bool both = in_a && in_b && a.stride[ia] == b.stride[ib];
  const bool step_a = both || (in_a && (!in_b || a.stride[ia] > b.stride[ib]));
  const int na = ia + (step_a ? 1 : 0), nb = ib + (both || !step_a ? 1 : 0);
  const int64_t s = step_a ? a.stride[ia] : b.stride[ib];
  // b's slice j against a's slice i lies k = j - i strides further.
  const int64_t first = step_a ? 1 - a.count[ia] : 0, last = nb > ib ? b.count[ib] - 1 : 0;
  int64_t from = (-b.extent(nb, D) - gap) / s, to = (a.extent(na, D) - gap) / s;
  from = from - 1 > first ? from - 1 : first, to = to + 1 < last ? to + 1 : last;
  for (int64_t k = from; k <= to; ++k)
    if (!apart(a, na, b, nb, gap + k * s, D, left)) return false;
  return true;
}

// Two outputs may lie between each other's heads or rows in one buffer, as the
// slices of a fused projection's gradient do, but not share an element.
bool outputs_overlap(const Heads &a, const Heads &b) {
  if (!heads_overlap(a, b)) return false;
  const int64_t gap = reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p);
  if (gap % a.size) return true;
  int left = kMostPairs;
  return !apart(Dims(a), 0, Dims(b), 0, gap / a.size, a.D, left);
}

// Size and value checks shared by the two directions.
ag_status check_qk(int64_t B, int64_t Hq, int64_t Hk, int64_t L, int64_t D, int64_t R,
                   int norm, float eps, int rope, int x_dtype, int o_dtype, int64_t pos_sb) {
  if (B < 0 || Hq < 0 || Hk < 0 || L < 0 || D < 1 || R < 0 || R > D || R % 2 || pos_sb < 0)
    return AG_ERR_SHAPE;
  if (norm < AG_NORM_NONE || norm > AG_NORM_LAYER || !(eps >= 0.f) || std::isinf(eps) ||
      (rope != AG_ROPE_HALVES && rope != AG_ROPE_INTERLEAVED) || !is_dtype(x_dtype) ||
      !is_dtype(o_dtype))
    return AG_ERR_VALUE;
  constexpr int64_t kMost = 0x7FFFFFFF;
  if (D > 1024 || B > kMost || L > kMost || Hq > 65536 || Hk > 65536 ||
      span_too_long(B, pos_sb))
    return AG_ERR_UNSUPPORTED;
  // B * L first: the product of three sizes could pass 64 bits.
  if (B * L > kMost || (B * L) * (Hq + Hk) > kMost) return AG_ERR_UNSUPPORTED;
  return AG_OK;
}

}  // namespace
}  // namespace ag

using ag::Heads;

extern "C" {

ag_status ag_qk_norm_rope_fwd(const void *q, int64_t q_sb, int64_t q_sl, int64_t q_sh,
                              const void *k, int64_t k_sb, int64_t k_sl, int64_t k_sh,
                              int x_dtype, const float *q_weight, const float *q_bias,
                              const float *k_weight, const float *k_bias, int norm, float eps,
                              const double *inv_freq, int64_t R, int rope,
                              const int64_t *positions, int64_t pos_sb, int64_t B, int64_t Hq,
                              int64_t Hk, int64_t L, int64_t D, void *q_out, void *k_out,
                              int out_dtype, void *stream) {
  ag_status st =
      ag::check_qk(B, Hq, Hk, L, D, R, norm, eps, rope, x_dtype, out_dtype, pos_sb);
  if (st != AG_OK) return st;
  const int xs = ag::size_of(x_dtype), os = ag::size_of(out_dtype);
  const Heads in[2] = {{q, {B, L, Hq}, {q_sb, q_sl, q_sh}, D, xs},
                       {k, {B, L, Hk}, {k_sb, k_sl, k_sh}, D, xs}};
  for (const Heads &h : in)
    if ((st = ag::check_strides(h)) != AG_OK) return st;
  if (B == 0 || L == 0 || Hq + Hk == 0) return AG_OK;
  if ((Hq && (!q || !q_out)) || (Hk && (!k || !k_out)) || (R && !inv_freq)) return AG_ERR_NULL;
  const float *params[4] = {q_weight, q_bias, k_weight, k_bias};
  if ((Hq && (!ag::aligned(q, xs) || !ag::aligned(q_out, os))) ||
      (Hk && (!ag::aligned(k, xs) || !ag::aligned(k_out, os))) || !ag::aligned(inv_freq, 8) ||
      !ag::aligned(positions, 8))
    return AG_ERR_ALIGN;
  for (const float *p : params)
    if (!ag::aligned(p, 4)) return AG_ERR_ALIGN;
  const void *outs[2] = {Hq ? q_out : nullptr, Hk ? k_out : nullptr};
  const uint64_t sizes[2] = {static_cast<uint64_t>(B) * L * Hq * D * os,
                             static_cast<uint64_t>(B) * L * Hk * D * os};
  for (int o = 0; o < 2; ++o) {
    for (const Heads &h : in)
      if (ag::overlap(outs[o], sizes[o], h.p, h.bytes())) return AG_ERR_ALIAS;
    for (const float *p : params)
      if (p && ag::overlap(outs[o], sizes[o], p, D * 4)) return AG_ERR_ALIAS;
    if (R && ag::overlap(outs[o], sizes[o], inv_freq, R / 2 * 8)) return AG_ERR_ALIAS;
    if (positions && ag::overlap(outs[o], sizes[o], positions, ((B - 1) * pos_sb + L) * 8))
      return AG_ERR_ALIAS;
  }
  if (ag::overlap(outs[0], sizes[0], outs[1], sizes[1])) return AG_ERR_ALIAS;
  ag::DeviceInfo *dev = nullptr;
  st = ag::device_info(&dev);
  if (st != AG_OK) return st;
  ag::QkArgs a{};
  for (int i = 0; i < 2; ++i) {
    ag::QkSide &s = a.side[i];
    s.x = in[i].p, s.sb = in[i].s[0], s.sl = in[i].s[1], s.sh = in[i].s[2];
    s.H = static_cast<int>(in[i].n[2]);
    s.w = params[2 * i], s.b = params[2 * i + 1];
    s.out = const_cast<void *>(outs[i]);
  }
  a.inv_freq = inv_freq, a.positions = positions, a.pos_sb = pos_sb;
  a.positions_total = B * L, a.B = B, a.L = L;
  a.D = static_cast<int>(D), a.R = static_cast<int>(R);
  a.norm = norm, a.rope = rope, a.x_dtype = x_dtype, a.o_dtype = out_dtype, a.eps = eps;
  return ag::from_cuda(ag::launch_qk_fwd(a, dev->num_sms, static_cast<cudaStream_t>(stream)));
}

ag_status ag_qk_norm_rope_bwd_workspace(int64_t B, int64_t Hq, int64_t Hk, int64_t L, int64_t D,
                                        int wants_params, int64_t *bytes) {
  if (!bytes) return AG_ERR_NULL;
  const ag_status st = ag::check_qk(B, Hq, Hk, L, D, 0, AG_NORM_NONE, 0.f, 0, AG_F32, AG_F32, 0);
  if (st != AG_OK) return st;
  *bytes = 0;
  if (!wants_params || B * L == 0 || Hq + Hk == 0) return AG_OK;
  ag::DeviceInfo *dev = nullptr;
  const ag_status ds = ag::device_info(&dev);
  if (ds != AG_OK) return ds;
  *bytes = ag::qk_bwd_workspace(B * L, static_cast<int>(Hq), static_cast<int>(Hk),
                                static_cast<int>(D), dev->num_sms);
  return AG_OK;
}

ag_status ag_qk_norm_rope_bwd(const void *dq_out, const void *dk_out, int g_dtype,
                              const void *q, int64_t q_sb, int64_t q_sl, int64_t q_sh,
                              const void *k, int64_t k_sb, int64_t k_sl, int64_t k_sh,
                              int x_dtype, const float *q_weight, const float *k_weight,
                              int norm, float eps, const double *inv_freq, int64_t R, int rope,
                              const int64_t *positions, int64_t pos_sb, int64_t B, int64_t Hq,
                              int64_t Hk, int64_t L, int64_t D, void *dq, int64_t dq_sb,
                              int64_t dq_sl, int64_t dq_sh, void *dk, int64_t dk_sb,
                              int64_t dk_sl, int64_t dk_sh, float *dq_weight, float *dq_bias,
                              float *dk_weight, float *dk_bias, void *workspace,
                              int64_t workspace_bytes, void *stream) {
  ag_status st = ag::check_qk(B, Hq, Hk, L, D, R, norm, eps, rope, x_dtype, g_dtype, pos_sb);
  if (st != AG_OK) return st;
  const int xs = ag::size_of(x_dtype), gs = ag::size_of(g_dtype);
  const Heads in[2] = {{q, {B, L, Hq}, {q_sb, q_sl, q_sh}, D, xs},
                       {k, {B, L, Hk}, {k_sb, k_sl, k_sh}, D, xs}};
  const Heads out[2] = {{dq, {B, L, Hq}, {dq_sb, dq_sl, dq_sh}, D, xs},
                        {dk, {B, L, Hk}, {dk_sb, dk_sl, dk_sh}, D, xs}};
  for (int i = 0; i < 2; ++i) {
    if ((st = ag::check_strides(in[i])) != AG_OK || (st = ag::check_strides(out[i])) != AG_OK)
      return st;
    if (!ag::distinct(out[i])) return AG_ERR_SHAPE;
  }
  float *params[4] = {dq_weight, dq_bias, dk_weight, dk_bias};
  bool wants = false;
  for (int i = 0; i < 4; ++i) {
    wants = wants || params[i];
    if (!ag::aligned(params[i], 4)) return AG_ERR_ALIGN;
    for (int j = 0; j < i; ++j)
      if (params[i] && params[j] && ag::overlap(params[i], D * 4, params[j], D * 4))
        return AG_ERR_ALIAS;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (B == 0 || L == 0 || Hq + Hk == 0) {
    if (!wants) return AG_OK;
    ag::DeviceInfo *dev = nullptr;
    st = ag::device_info(&dev);
    if (st != AG_OK) return st;
    for (float *p : params)
      if (p && cudaMemsetAsync(p, 0, D * 4, s) != cudaSuccess) return AG_ERR_CUDA;
    return AG_OK;
  }
  const void *g[2] = {Hq ? dq_out : nullptr, Hk ? dk_out : nullptr};
  const uint64_t g_bytes[2] = {static_cast<uint64_t>(B) * L * Hq * D * gs,
                               static_cast<uint64_t>(B) * L * Hk * D * gs};
  const float *weights[2] = {q_weight, k_weight};
  for (int i = 0; i < 2; ++i)
    if (in[i].n[2] && (!in[i].p || !out[i].p || !g[i])) return AG_ERR_NULL;
  if (R && !inv_freq) return AG_ERR_NULL;
  for (int i = 0; i < 2; ++i)
    if ((in[i].n[2] && (!ag::aligned(in[i].p, xs) || !ag::aligned(out[i].p, xs) ||
                        !ag::aligned(g[i], gs))) ||
        !ag::aligned(weights[i], 4))
      return AG_ERR_ALIGN;
  if (!ag::aligned(inv_freq, 8) || !ag::aligned(positions, 8) || !ag::aligned(workspace, 256))
    return AG_ERR_ALIGN;
  // Every output against every input, then against the other outputs.
  struct Range {
    const void *p;
    uint64_t n;
  };
  const uint64_t row = static_cast<uint64_t>(D) * 4, freqs = static_cast<uint64_t>(R) * 4,
                 places = static_cast<uint64_t>((B - 1) * pos_sb + L) * 8;
  const Range ins[8] = {{in[0].p, in[0].bytes()},
                        {in[1].p, in[1].bytes()},
                        {g[0], g_bytes[0]},
                        {g[1], g_bytes[1]},
                        {q_weight, q_weight ? row : 0},
                        {k_weight, k_weight ? row : 0},
                        {inv_freq, freqs},
                        {positions, positions ? places : 0}};
  Range outs[7] = {{out[0].p, out[0].bytes()}, {out[1].p, out[1].bytes()}};
  for (int i = 0; i < 4; ++i) outs[2 + i] = {params[i], params[i] ? row : 0};
  ag::DeviceInfo *dev = nullptr;
  st = ag::device_info(&dev);
  int64_t need = 0;
  if (st == AG_OK && wants)
    need = ag::qk_bwd_workspace(B * L, static_cast<int>(Hq), static_cast<int>(Hk),
                                static_cast<int>(D), dev->num_sms);
  outs[6] = {workspace, workspace ? static_cast<uint64_t>(need) : 0u};
  for (int o = 0; o < 7; ++o) {
    for (const Range &r : ins)
      if (ag::overlap(outs[o].p, outs[o].n, r.p, r.n)) return AG_ERR_ALIAS;
    for (int u = o + 1; u < 7; ++u) {
      if (o == 0 && u == 1) continue;
      if (ag::overlap(outs[o].p, outs[o].n, outs[u].p, outs[u].n)) return AG_ERR_ALIAS;
    }
  }
  if (ag::outputs_overlap(out[0], out[1])) return AG_ERR_ALIAS;
  if (st != AG_OK) return st;
  if (need > 0 && (!workspace || workspace_bytes < need)) return AG_ERR_SCRATCH;
  ag::QkArgs a{};
  for (int i = 0; i < 2; ++i) {
    ag::QkSide &t = a.side[i];
    t.x = in[i].p, t.sb = in[i].s[0], t.sl = in[i].s[1], t.sh = in[i].s[2];
    t.H = static_cast<int>(in[i].n[2]);
    t.w = weights[i], t.g = g[i];
    t.dx = const_cast<void *>(out[i].p);
    t.dxb = out[i].s[0], t.dxl = out[i].s[1], t.dxh = out[i].s[2];
    t.dw = params[2 * i], t.db = params[2 * i + 1];
  }
  a.inv_freq = inv_freq, a.positions = positions, a.pos_sb = pos_sb;
  a.positions_total = B * L, a.B = B, a.L = L;
  a.D = static_cast<int>(D), a.R = static_cast<int>(R);
  a.norm = norm, a.rope = rope, a.x_dtype = x_dtype, a.o_dtype = g_dtype, a.eps = eps;
  a.partial = wants ? static_cast<float *>(workspace) : nullptr;
  return ag::from_cuda(ag::launch_qk_bwd(a, dev->num_sms, s));
}

ag_status ag_grad_clip_workspace(int64_t n, int64_t *bytes) {
  if (!bytes) return AG_ERR_NULL;
  if (n < 0) return AG_ERR_SHAPE;
  if (n > (int64_t(1) << 20)) return AG_ERR_UNSUPPORTED;
  ag::DeviceInfo *dev = nullptr;
  const ag_status st = ag::device_info(&dev);
  if (st != AG_OK) return st;
  *bytes = ag::grad_clip_workspace(n, dev->num_sms);
  return AG_OK;
}

ag_status ag_grad_clip(void *const *grads, const int64_t *counts, const int *dtypes, int64_t n,
                       float max_norm, float eps, float *norm_out, void *workspace,
                       int64_t workspace_bytes, void *stream) {
  if (n < 0) return AG_ERR_SHAPE;
  if (n > (int64_t(1) << 20)) return AG_ERR_UNSUPPORTED;
  if (!(max_norm >= 0.f) || !(eps >= 0.f)) return AG_ERR_VALUE;
  if (!norm_out || (n && (!grads || !counts || !dtypes))) return AG_ERR_NULL;
  int64_t total = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (counts[i] < 0 || counts[i] > (int64_t(1) << 40)) return AG_ERR_SHAPE;
    if (!ag::is_dtype(dtypes[i])) return AG_ERR_VALUE;
    total += counts[i];
    if (total > (int64_t(1) << 42)) return AG_ERR_UNSUPPORTED;
    if (counts[i] && !grads[i]) return AG_ERR_NULL;
    if (counts[i] && !ag::aligned(grads[i], ag::size_of(dtypes[i]))) return AG_ERR_ALIGN;
  }
  if (!ag::aligned(norm_out, 4) || !ag::aligned(workspace, 256)) return AG_ERR_ALIGN;
  ag::DeviceInfo *dev = nullptr;
  const ag_status ds = ag::device_info(&dev);
  const int64_t need = ds == AG_OK ? ag::grad_clip_workspace(n, dev->num_sms) : 0;
  // Address ranges in order: no two may overlap (a tensor listed twice would
  // be scaled twice).
  struct Range {
    uintptr_t at;
    uint64_t n;
  };
  Range *r = static_cast<Range *>(std::malloc((n + 2) * sizeof(Range)));
  if (!r) return AG_ERR_SCRATCH;
  int64_t m = 0;
  r[m++] = {reinterpret_cast<uintptr_t>(norm_out), 4};
  if (workspace && need)
    r[m++] = {reinterpret_cast<uintptr_t>(workspace), static_cast<uint64_t>(need)};
  for (int64_t i = 0; i < n; ++i)
    if (counts[i])
      r[m++] = {reinterpret_cast<uintptr_t>(grads[i]),
                static_cast<uint64_t>(counts[i]) * ag::size_of(dtypes[i])};
  std::sort(r, r + m, [](const Range &a, const Range &b) { return a.at < b.at; });
  bool clash = false;
  for (int64_t i = 0; i + 1 < m; ++i) clash = clash || r[i].at + r[i].n > r[i + 1].at;
  std::free(r);
  if (clash) return AG_ERR_ALIAS;
  if (ds != AG_OK) return ds;
  if (!workspace || workspace_bytes < need) return AG_ERR_SCRATCH;
  return ag::from_cuda(ag::launch_grad_clip(grads, counts, dtypes, n, max_norm, eps, norm_out,
                                            static_cast<double *>(workspace), dev->num_sms,
                                            static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
