// linear_sm100.cu -- the linear layers' products on the tensor cores of
// sm_100a: C[m, n] = sum_k A(m, k) B(n, k) for 16-bit A and B, with the layer's
// epilogue.
//
// Tiles.  A 2-CTA cluster owns a 256 x BN tile of C: tcgen05.mma with
// cta_group::2 covers M = 256 over both SMs, each CTA staging its own 128 rows
// of A and half of B's BN rows, 64 of the summed dimension per pipeline stage,
// by TMA in the 128-byte swizzle.  A and B may each lie with the summed
// dimension dense (K-major) or the other one (MN-major), so that y = x W^T,
// dx = dy W and dW = dy^T x all read their operands as they are.
//
// Sums.  The tensor core's float32 accumulator truncates: over 8192 terms of
// random sign a plain product is 9e-6 of its size off (measured; 1e-6 over
// 1024), where a float32 sum rounds to 1e-6.  So the accumulator is taken over
// after every 512 terms by the epilogue warps, which add it to float32
// registers (4.7e-7 off at 1024 terms; 32768 positive terms are 1.6e-4 off without
// this, below 6e-6 with it).  With two accumulators in tensor memory
// the tensor core goes on with the next 512 terms meanwhile; the same path also
// overlaps one tile's epilogue with the next tile's products.  Terms per
// takeover, us for 8192 x 1024 x 1536, 16384 x 4096 x 1024 and 8192 x 8192 x 8192:
// 128: 24.7, 116, 782; 256: 25.3, 114, 790; 512: 23.0, 102, 740; 1024: 22.8, 101,
// 739.
//
// Roles per CTA: warp 0 loads, warp 1 of the even CTA issues the products (both
// CTAs' loads count on its barriers), warps 4 to 19 take over the accumulators
// and finish the tile.  With eight such warps instead of sixteen their latencies,
// not the products, set the pace: 16384 x 4096 x 1024 with a GELU took 142 us
// against 112.  Each of them holds 32 rows x BN / 4 columns of sums in
// registers, one row per lane.  Where every array of the epilogue is one that TMA
// can address, a warp reads the residual (or the pre-activation of a derivative)
// and writes the results as 32-row boxes of shared memory, so that the tile's
// memory traffic is asynchronous and whole lines; odd row strides take plain
// loads and stores, turned through shared memory so that they are at least
// contiguous.
//
// Registers.  The 256-wide kernels with a derivative in the epilogue, and those of
// both gradients, hold more than 96 a thread: they spill 64 to 228 bytes (loads
// 104 to 252) around the epilogue, whose sums alone are 64 registers; the others
// spill nothing.
//
// Bounds.  16384 x 4096 x 1024 without an activation takes 100 to 102 us, 1.36
// PFLOP/s: the products, at the clock that the board's power leaves (the
// library's product takes 100).  8192 x 1024 x 1536 takes 22.4 us with bias and
// residual: 128 tiles over 74 pairs are two rounds, the second 73 % full, and the
// first loads and last stores are not hidden.
//
// Both gradients of a layer run in one launch (linear_gemm_pair_kernel): the
// roles go from dW's tiles to dx's without a pause, and the clusters that have a
// tile of dW less take more of dx (Turns).
//
// A small C does not fill the GPU: the summed dimension is then split between
// clusters, each writing float32 partial sums that a second kernel
// (linear_join_kernel) adds in order and finishes.
#include <mutex>

#include "ag_internal.h"
#include "linear_epilogue.cuh"
#include "launch.cuh"
#include "linear_gemm.h"
#include "linear_ptx.cuh"

namespace ag {
namespace gemm {

constexpr int kThreads = 640;
constexpr int kEpiWarps = 16;
constexpr int kFirstEpiWarp = 4;
constexpr int kStepBytes = 128;                  // 64 16-bit terms
constexpr int kPromote = 8;                      // k tiles per accumulator: 512 terms
constexpr uint32_t kRegsLaunch = 96, kRegsLow = 56, kRegsHigh = 104;
static_assert(128 * kRegsLow + 32 * kEpiWarps * kRegsHigh <= kThreads * kRegsLaunch,
              "the epilogue's registers come out of the role warps' release");

template <int BN>
struct Shape {
  static constexpr int kStages = BN == 256 ? 5 : 6;
  static constexpr int kABytes = 128 * kStepBytes;
  static constexpr int kBBytes = BN / 2 * kStepBytes;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kCols = 2 * BN;           // tensor-memory columns
};
// Per epilogue warp: a box of 32 rows x 128 bytes.
constexpr int kBoxBytes = 32 * 128;
constexpr int kStageOutBytes = kEpiWarps * kBoxBytes;

struct Barriers {
  uint64_t full[8], empty[8];
  uint64_t acc_full[2], acc_free[2];
  uint64_t in_full[kEpiWarps];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};
template <int BN>
constexpr size_t smem_bytes() {
  return 1024 + Shape<BN>::kStages * Shape<BN>::kStageBytes + kStageOutBytes + sizeof(Barriers);
}
static_assert(smem_bytes<256>() <= 227 * 1024 && smem_bytes<128>() <= 227 * 1024, "shared memory");

enum Site : unsigned {
  kSiteLoad = 30, kSiteIssue = 32, kSiteAccFree = 33, kSiteAccFull = 34,
  kSiteIn = 35
};

struct Params {
  int64_t M, N;               // rows and columns of C
  int items;                  // tiles x splits (below 2^31: see check_linear_sizes)
  int tiles_m, tiles_n, k_tiles, splits;
  Turns turns;
  int boxes;                  // every array of the epilogue is TMA's to read or write
  int wide;                   // the output is float32
  uint32_t idesc;
  unsigned *err;
  LinearEpilogue epi;
};

// Work item -> tile and range of k tiles.  Tiles go in groups of 8 along M, a
// group's tiles along M first: the clusters at work then cover about 8 x 9
// tiles, so that what they read between them stays in L2.
struct Item {
  int tm, tn, split, kb, ke;
};
constexpr int kGroup = 8;
__device__ __forceinline__ Item item_at(const Params &p, int i) {
  Item t;
  const int tiles = p.tiles_m * p.tiles_n, per_group = kGroup * p.tiles_n;
  t.split = i / tiles;
  const int r = i - t.split * tiles, group = r / per_group;
  const int rest = r - group * per_group, high = min(kGroup, p.tiles_m - group * kGroup);
  t.tn = rest / high;
  t.tm = group * kGroup + rest - t.tn * high;
  t.kb = p.k_tiles * t.split / p.splits;  // k_tiles <= 2^20, splits <= 32
  t.ke = p.k_tiles * (t.split + 1) / p.splits;
  return t;
}

// This cluster's item of round r (by the product's turns, or with one product in
// the launch all clusters in every round); past the last one at or after p.items.
template <bool TURNS>
__device__ __forceinline__ int item_of(const Params &p, int r) {
  const int c = blockIdx.x / 2, all = gridDim.x / 2;
  if constexpr (!TURNS) return c;
  const int few = all - p.turns.from;
  if (c < p.turns.from) return p.turns.extra * few + r * all + c;
  return r < p.turns.extra ? r * few + c - p.turns.from
                           : p.turns.extra * few + (r - p.turns.extra) * all + c;
}

template <bool TURNS>
__device__ __forceinline__ int next_item(const Params &p, int i, int &r) {
  return TURNS ? item_of<true>(p, ++r) : i + static_cast<int>(gridDim.x / 2);
}

// One 64-deep tile of `rows` rows of an operand: K-major, one box of 64 terms
// x rows; MN-major, boxes of 64 rows x 64 terms.
template <bool MN, int ROWS>
__device__ __forceinline__ void load_tile(uint8_t *dst, const CUtensorMap *map, uint32_t bar,
                                          int row, int k) {
  if constexpr (MN) {
#pragma unroll
    for (int q = 0; q < ROWS / 64; ++q)
      tma_load_2d_pair(dst + q * 64 * kStepBytes, map, bar, row + 64 * q, k);
  } else {
    tma_load_2d_pair(dst, map, bar, k, row);
  }
}

// The roles' loops over a product's items.  n counts k tiles and acc accumulators,
// through both products where a launch has two.
template <int BN, bool A_MN, bool B_MN, bool TURNS>
__device__ __forceinline__ bool load_items(const CUtensorMap *ma, const CUtensorMap *mb,
                                           uint8_t *ring, Barriers *bars, const Params &p,
                                           uint32_t rank, volatile int *abort, uint32_t &n) {
  using S = Shape<BN>;
  const uint32_t full0 = cluster_addr(&bars->full[0], 0);
  bool ok = true;
  for (int r = 0, i = item_of<TURNS>(p, 0); ok && i < p.items; i = next_item<TURNS>(p, i, r)) {
    const Item t = item_at(p, i);
    const int row_a = t.tm * 256 + static_cast<int>(rank) * 128;
    const int row_b = t.tn * BN + static_cast<int>(rank) * (BN / 2);
    for (int k = t.kb; k < t.ke; ++k) {
      const uint32_t s = n % S::kStages;
      ok = mbar_wait(&bars->empty[s], ((n / S::kStages) & 1u) ^ 1u, abort, p.err, kSiteLoad);
      if (!ok) break;
      uint8_t *at = ring + s * S::kStageBytes;
      // Both CTAs' bytes count on the even CTA's barrier.  The odd CTA's may
      // come first: the phase cannot end before the even CTA's arrival.
      const uint32_t bar = full0 + 8 * s;
      if (rank == 0) mbar_arrive_expect_tx(&bars->full[s], 2 * S::kStageBytes);
      load_tile<A_MN, 128>(at, ma, bar, row_a, k * 64);
      load_tile<B_MN, BN / 2>(at + S::kABytes, mb, bar, row_b, k * 64);
      ++n;
    }
  }
  return ok;
}
// Every copy of the pair lands before its CTAs exit: the products wait for
// all of them, so only after a failure may some be on their way.
template <int BN>
__device__ __forceinline__ void load_drain(Barriers *bars, uint32_t rank, uint32_t n) {
  using S = Shape<BN>;
  if (rank == 0) {
    for (uint32_t i = n > S::kStages ? n - S::kStages : 0; i < n; ++i) {
      const uint32_t a = smem_u32(&bars->full[i % S::kStages]);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_test(a, (i / S::kStages) & 1u))
        if (globaltimer_ns() - t0 > kWaitLimitNs) break;
    }
  }
  const uint64_t t0 = globaltimer_ns();  // loads that the even CTA never counted
  while (globaltimer_ns() - t0 < kWaitLimitNs / 1000) {
  }
}

// The whole warp of the even CTA; one elected lane issues.
template <int BN, bool A_MN, bool B_MN, bool TURNS>
__device__ __forceinline__ bool issue_items(uint8_t *ring, Barriers *bars, uint32_t tmem,
                                            const Params &p, volatile int *abort, uint32_t &n,
                                            uint32_t &acc) {
  using S = Shape<BN>;
  constexpr uint32_t kHi = desc_sw128_hi(1024);  // 8-row groups 1 KB apart, either major
  constexpr uint32_t kAtom = 64 * kStepBytes;    // MN-major: the next 64 rows
  // 16 terms further: 32 bytes along a K-major row, 16 rows of an MN-major tile.
  constexpr uint32_t kAStep = (A_MN ? 16 * kStepBytes : 32) >> 4;
  constexpr uint32_t kBStep = (B_MN ? 16 * kStepBytes : 32) >> 4;
  bool ok = true;
  for (int r = 0, i = item_of<TURNS>(p, 0); ok && i < p.items; i = next_item<TURNS>(p, i, r)) {
    const Item t = item_at(p, i);
    for (int k0 = t.kb; ok && k0 < t.ke; k0 += kPromote, ++acc) {
      const uint32_t b = acc & 1u, use = acc >> 1;
      if (use > 0) {
        ok = mbar_wait_warp(&bars->acc_free[b], (use - 1) & 1u, abort, p.err, kSiteAccFree);
        if (!ok) break;
        tc_fence_after();
      }
      const int end = min(k0 + kPromote, t.ke);
      for (int k = k0; k < end; ++k, ++n) {
        const uint32_t s = n % S::kStages;
        ok = mbar_wait_warp(&bars->full[s], (n / S::kStages) & 1u, abort, p.err, kSiteIssue);
        if (!ok) break;
        tc_fence_after();
        const uint32_t at = smem_u32(ring + s * S::kStageBytes);
        const uint32_t a_lo = desc_sw128_lo(at, A_MN ? kAtom : 16);
        const uint32_t b_lo = desc_sw128_lo(at + S::kABytes, B_MN ? kAtom : 16);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          umma2_ss_w(tmem + BN * b, a_lo + q * kAStep, b_lo + q * kBStep, kHi, p.idesc,
                     (k > k0 || q > 0) ? 1u : 0u);
        umma2_commit_both_w(&bars->empty[s]);
      }
      if (ok) umma2_commit_both_w(&bars->acc_full[b]);
    }
  }
  return ok;
}
// Everything this warp issued completes before tensor memory is freed.
__device__ __forceinline__ void issue_drain(Barriers *bars) {
  umma2_commit_self_w(&bars->drain);
  const uint32_t a = smem_u32(&bars->drain);
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_test(a, 0))
    if (globaltimer_ns() - t0 > kWaitLimitNs) break;
}

// Tensor maps of the epilogue's arrays (read when p.boxes): the output, or with
// splits the partial sums [splits][M][N]; the residual or the pre-activation
// that is read; the pre-activation that is written.
struct EpiMaps {
  CUtensorMap out, in, pre;
};

__device__ __forceinline__ uint32_t pack2(float2 v, bool bf16) {
  if (bf16) return pack_bf16x2(v.x, v.y);
  const __half2 h = __floats2half2_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack2(uint32_t w, bool bf16) {
  if (bf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// One warp's 32 rows x COLS columns through its box, kWidth columns at a time:
// the residual or the pre-activation is read into the box while the products
// run, each lane replaces its row's values by the results, and the box is
// stored.  (A pre-activation to be written goes through the box before.)
// WIDE: float32 results.
template <int COLS, int ACT, bool SLOPE, bool WIDE>
struct BoxEpilogue {
  static constexpr int kWidth = WIDE ? 32 : COLS, kPieces = COLS / kWidth;
  static constexpr int kRow = kWidth * (WIDE ? 4 : 2), kPreRow = kWidth * 2;  // bytes
  static_assert(kRow == 128 || kRow == 64, "a box row is a swizzle span");
  const Params &p;
  const EpiMaps *maps;
  uint8_t *own;
  uint64_t *in_full;
  volatile int *abort;
  int lane;
  uint32_t started = 0, waited = 0;  // reads into the box

  __device__ bool writes_pre() const { return !SLOPE && p.epi.pre_out; }
  __device__ bool reads() const { return SLOPE || p.epi.residual; }
  __device__ bool valid(int64_t row0, int64_t col0, int j) const {
    return row0 < p.M && col0 + j * kWidth < p.N;
  }
  // 16-byte chunk c of this lane's row, as TMA's swizzle places it.
  template <int ROW>
  __device__ uint4 *chunk(int c) const {
    const int s = ROW == 128 ? c ^ (lane & 7) : c ^ ((lane >> 1) & 3);
    return reinterpret_cast<uint4 *>(own + lane * ROW + (s << 4));
  }
  __device__ void box_free() const {
    if (lane == 0) bulk_wait_read_all();
    __syncwarp();
  }
  __device__ void store(const CUtensorMap *map, int64_t row0, int64_t col, int part) const {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_3d(map, own, static_cast<int>(col), static_cast<int>(row0), part);
      bulk_commit_group();
    }
  }
  // The box's earlier stores have been read out; its earlier reads by the lanes
  // are ordered by the fence before those stores.
  __device__ void start_read(int64_t row0, int64_t col0, int j) {
    if (!valid(row0, col0, j)) return;
    ++started;
    if (lane != 0) return;
    bulk_wait_read_all();
    mbar_arrive_expect_tx(in_full, 32 * (SLOPE ? kPreRow : kRow));
    tma_load_2d(own, &maps->in, in_full, static_cast<int>(col0) + j * kWidth,
                static_cast<int>(row0));
  }
  __device__ void begin(int64_t row0, int64_t col0) {
    if (reads() && !writes_pre()) start_read(row0, col0, 0);
  }
  // Every copy this warp started is done with the CTA's memory before the CTA
  // ends.
  __device__ void drain() const {
    if (lane == 0) {
      const uint64_t t0 = globaltimer_ns();
      while (started != waited && !mbar_test(smem_u32(in_full), waited & 1u))
        if (globaltimer_ns() - t0 > kWaitLimitNs) break;
      bulk_wait_read_all();  // (the grid's end waits for the writes themselves)
    }
    __syncwarp();
  }

  __device__ bool finish(const float2 (&sum)[COLS / 2], int64_t row0, int64_t col0, int part) {
    const bool bf16 = p.epi.dtype == AG_BF16;
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      if (!valid(row0, col0, j)) break;
      const int64_t col = col0 + j * kWidth;
      const float2 *s = sum + j * kWidth / 2;
      if (writes_pre()) {
        box_free();
#pragma unroll
        for (int c = 0; c < kWidth / 8; ++c)
          *chunk<kPreRow>(c) = make_uint4(pack2(s[4 * c], bf16), pack2(s[4 * c + 1], bf16),
                                          pack2(s[4 * c + 2], bf16), pack2(s[4 * c + 3], bf16));
        store(&maps->pre, row0, col, 0);
        if (reads()) start_read(row0, col0, j);
      }
      uint4 pre[kPreRow / 16];
      if (reads()) {
        if (!mbar_wait_warp(in_full, waited & 1u, abort, p.err, kSiteIn)) return false;
        ++waited;
        if constexpr (SLOPE && kRow != kPreRow) {
          // Rows of another length: all are read before any is replaced.
#pragma unroll
          for (int c = 0; c < kPreRow / 16; ++c) pre[c] = *chunk<kPreRow>(c);
          __syncwarp();
        }
      } else {
        box_free();
      }
#pragma unroll
      for (int c = 0; c < kRow / 16; ++c) {
        if constexpr (WIDE) {
          float2 v[2] = {s[2 * c], s[2 * c + 1]};
          if constexpr (SLOPE) {
            const uint32_t w[2] = {c & 1 ? pre[c / 2].z : pre[c / 2].x,
                                   c & 1 ? pre[c / 2].w : pre[c / 2].y};
#pragma unroll
            for (int i = 0; i < 2; ++i) v[i] = __fmul2_rn(v[i], act_slope2<ACT>(unpack2(w[i], bf16)));
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) v[i] = act_value2<ACT>(v[i]);
            if (p.epi.residual) {
              const float4 r = *reinterpret_cast<const float4 *>(chunk<kRow>(c));
              v[0] = __fadd2_rn(v[0], make_float2(r.x, r.y));
              v[1] = __fadd2_rn(v[1], make_float2(r.z, r.w));
            }
          }
          *reinterpret_cast<float4 *>(chunk<kRow>(c)) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
        } else {
          uint4 in = make_uint4(0, 0, 0, 0);
          if (reads()) in = *chunk<kRow>(c);
          const uint32_t w[4] = {in.x, in.y, in.z, in.w};
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float2 v = s[4 * c + i];
            if constexpr (SLOPE) {
              v = __fmul2_rn(v, act_slope2<ACT>(unpack2(w[i], bf16)));
            } else {
              v = act_value2<ACT>(v);
              if (p.epi.residual) v = __fadd2_rn(v, unpack2(w[i], bf16));
            }
            o[i] = pack2(v, bf16);
          }
          *chunk<kRow>(c) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      store(&maps->out, row0, col, part);
      if (reads() && !writes_pre() && j + 1 < kPieces) start_read(row0, col0, j + 1);
    }
    return true;
  }
};

// The sums start from the bias (its loads run while the products do).
template <int COLS>
__device__ __forceinline__ void start_sums(float2 (&sum)[COLS / 2], const float *bias, int64_t col0,
                                           int64_t N) {
  const bool vec = (reinterpret_cast<uintptr_t>(bias) & 15) == 0;
#pragma unroll
  for (int c = 0; c < COLS; c += 4) {
    float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
    if (bias && col0 + c < N) {
      const float *at = bias + col0 + c;
      if (vec && col0 + c + 4 <= N) {
        b = __ldg(reinterpret_cast<const float4 *>(at));
      } else {
        b.x = __ldg(at);
        if (col0 + c + 1 < N) b.y = __ldg(at + 1);
        if (col0 + c + 2 < N) b.z = __ldg(at + 2);
        if (col0 + c + 3 < N) b.w = __ldg(at + 3);
      }
    }
    sum[c / 2] = make_float2(b.x, b.y);
    sum[c / 2 + 1] = make_float2(b.z, b.w);
  }
}

// Eight rows of one column (the rows from r on of the 32 in `stage`).
__device__ __forceinline__ void finish_column(const LinearEpilogue &e, const float *stage, int r,
                                              int lane, int64_t row, int64_t rows, int64_t col) {
  const int n = static_cast<int>(min(static_cast<int64_t>(8), rows - row));
  float v[8], x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = stage[(r + i) * 32 + (((lane >> 2) ^ ((r + i) & 7)) << 2) + (lane & 3)];
  const auto store = [&](void *p, int64_t ld, int dtype) {
    int64_t at = row * ld + col;
#pragma unroll
    for (int i = 0; i < 8; ++i, at += ld) {
      const float one[1] = {v[i]};
      if (i < n) store_values<1>(p, at, dtype, one);
    }
  };
  if (e.pre_out) store(e.pre_out, e.ld_pre_out, e.dtype);
  if (e.pre_in) {
    load_apart<8>(e.pre_in, row * e.ld_pre_in + col, e.ld_pre_in, n, e.dtype, x);
    act_all<true>(x, e.act);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= x[i];
  } else if (e.act != AG_ACT_NONE) {
    act_all<false>(v, e.act);
  }
  if (e.residual) {
    load_apart<8>(e.residual, row * e.ld_res + col, e.ld_res, n, e.out_dtype, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += x[i];
  }
  store(e.out, e.ld_out, e.out_dtype);
}

// The same without boxes: 32 columns at a time through a box's memory (float4
// q of row r in slot q ^ (r % 8)), then a lane per column, eight rows at a time.
template <int COLS>
__device__ __forceinline__ void plain_epilogue(const Params &p, const float2 (&sum)[COLS / 2],
                                               float *stage, int64_t row0, int64_t col0, int lane) {
#pragma unroll
  for (int c = 0; c < COLS; c += 32) {
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float2 a = sum[c / 2 + 2 * q], b = sum[c / 2 + 2 * q + 1];
      *reinterpret_cast<float4 *>(stage + lane * 32 + ((q ^ (lane & 7)) << 2)) =
          make_float4(a.x, a.y, b.x, b.y);
    }
    __syncwarp();
    const int64_t col = col0 + c + lane;
    if (col < p.N) {
#pragma unroll 1
      for (int r = 0; r < 32; r += 8)
        if (row0 + r < p.M) finish_column(p.epi, stage, r, lane, row0 + r, p.M, col);
    }
  }
}

template <int BN, int ACT, bool SLOPE, bool WIDE, bool BOXES, bool TURNS>
__device__ __forceinline__ bool finish_items_as(uint8_t *stage, Barriers *bars, uint32_t tmem,
                                             const Params &p, const EpiMaps *maps, uint32_t rank,
                                             int warp, int lane, volatile int *abort,
                                             uint32_t &acc) {
  constexpr int kCols = BN / 4;                  // columns per warp
  const int quarter = warp % 4, part = (warp - kFirstEpiWarp) / 4;
  const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t free_bar = cluster_addr(&bars->acc_free[0], 0);
  uint8_t *own = stage + (warp - kFirstEpiWarp) * kBoxBytes;
  BoxEpilogue<kCols, ACT, SLOPE, WIDE> boxes{
      p, maps, own, &bars->in_full[warp - kFirstEpiWarp], abort, lane};
  bool ok = true;
  for (int r = 0, i = item_of<TURNS>(p, 0); ok && i < p.items; i = next_item<TURNS>(p, i, r)) {
    const Item t = item_at(p, i);
    const int64_t row0 = static_cast<int64_t>(t.tm) * 256 + rank * 128 + quarter * 32;
    const int64_t col0 = static_cast<int64_t>(t.tn) * BN + kCols * part;
    if constexpr (BOXES) boxes.begin(row0, col0);
    float2 sum[kCols / 2];
    start_sums<kCols>(sum, p.epi.bias, col0, p.N);
    for (int k0 = t.kb; k0 < t.ke; k0 += kPromote, ++acc) {
      const uint32_t b = acc & 1u;
      ok = mbar_wait_warp(&bars->acc_full[b], (acc >> 1) & 1u, abort, p.err, kSiteAccFull);
      if (!ok) break;
      tc_fence_after();
      const uint32_t at = tmem + lanes + BN * b + kCols * part;
#pragma unroll
      for (int c = 0; c < kCols; c += 16) {  // (32 at a time would not fit the registers)
        uint32_t r[16];
        tmem_ld16(at + c, r);
        tmem_wait_ld16(r);
#pragma unroll
        for (int q = 0; q < 8; ++q)
          sum[c / 2 + q] = __fadd2_rn(sum[c / 2 + q], make_float2(__uint_as_float(r[2 * q]),
                                                                  __uint_as_float(r[2 * q + 1])));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(free_bar + 8 * b);
    }
    if (!ok) break;
    if constexpr (BOXES) {
      ok = boxes.finish(sum, row0, col0, t.split);
    } else {
      plain_epilogue<kCols>(p, sum, reinterpret_cast<float *>(own), row0, col0, lane);
    }
  }
  if constexpr (BOXES) boxes.drain();
  return ok;
}
template <int BN, int ACT, bool SLOPE, bool BOXES, bool TURNS>
__device__ __forceinline__ bool finish_items(uint8_t *stage, Barriers *bars, uint32_t tmem,
                                             const Params &p, const EpiMaps *maps, uint32_t rank,
                                             int warp, int lane, volatile int *abort,
                                             uint32_t &acc) {
  if (BOXES && p.wide)
    return finish_items_as<BN, ACT, SLOPE, true, BOXES, TURNS>(stage, bars, tmem, p, maps, rank,
                                                               warp, lane, abort, acc);
  return finish_items_as<BN, ACT, SLOPE, false, BOXES, TURNS>(stage, bars, tmem, p, maps, rank,
                                                              warp, lane, abort, acc);
}

// A product as a kernel's argument.
struct Product {
  CUtensorMap ma, mb;
  EpiMaps maps;
  Params p;
};

// A CTA's setup, its roles (each returns whether all its waits ended) and its end.
template <int BN, typename Load, typename Issue, typename Finish>
__device__ __forceinline__ void run_roles(const CUtensorMap *ma, const CUtensorMap *mb, Load load,
                                          Issue issue, Finish finish) {
  using S = Shape<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *stage = ring + S::kStages * S::kStageBytes;
  Barriers *bars = reinterpret_cast<Barriers *>(stage + kStageOutBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  if (threadIdx.x == 0) {
    griddep_launch_dependents();
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->acc_full[b], 1);
      mbar_init(&bars->acc_free[b], 2 * kEpiWarps);
    }
    for (int w = 0; w < kEpiWarps; ++w) mbar_init(&bars->in_full[w], 1);
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    fence_mbar_init();
    prefetch_tensormap(ma);
    prefetch_tensormap(mb);
  }
  if (warp == 1) {
    tmem_alloc2(&bars->tmem_base, S::kCols);
    tmem_relinquish2();
  }
  griddep_wait();  // nothing before this touches what the kernel before wrote or read
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  volatile int *abort = &bars->abort;
  if (warp < kFirstEpiWarp) {
    regs_dec<kRegsLow>();
    if (warp == 1 && rank == 0) {
      uint32_t n = 0, acc = 0;
      issue(ring, bars, tmem, abort, n, acc);
      issue_drain(bars);
    } else if (warp == 0 && lane == 0) {
      uint32_t n = 0;
      if (!load(ring, bars, rank, abort, n)) load_drain<BN>(bars, rank, n);
    }
  } else {
    regs_inc<kRegsHigh>();
    uint32_t acc = 0;
    finish(stage, bars, tmem, rank, warp, lane, abort, acc);
  }
  __syncwarp();
  // Neither CTA leaves while the other may use its shared or tensor memory.
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc2(tmem, S::kCols);
  }
}

template <int BN, bool A_MN, bool B_MN, int ACT, bool SLOPE, bool BOXES>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    linear_gemm_kernel(const __grid_constant__ Product a) {
  run_roles<BN>(
      &a.ma, &a.mb,
      [&](uint8_t *ring, Barriers *bars, uint32_t rank, volatile int *abort, uint32_t &n) {
        return load_items<BN, A_MN, B_MN, false>(&a.ma, &a.mb, ring, bars, a.p, rank, abort, n);
      },
      [&](uint8_t *ring, Barriers *bars, uint32_t tmem, volatile int *abort, uint32_t &n,
          uint32_t &acc) { issue_items<BN, A_MN, B_MN, false>(ring, bars, tmem, a.p, abort, n, acc); },
      [&](uint8_t *stage, Barriers *bars, uint32_t tmem, uint32_t rank, int warp, int lane,
          volatile int *abort, uint32_t &acc) {
        finish_items<BN, ACT, SLOPE, BOXES, false>(stage, bars, tmem, a.p, &a.maps, rank, warp, lane,
                                            abort, acc);
      });
}

// Two products one after the other, without a pause between them: dW = dy^T x,
// then dx = (dy W) times the activation's derivative.
template <int BN, int ACT, bool SLOPE, bool W_BOXES, bool X_BOXES>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    linear_gemm_pair_kernel(const __grid_constant__ Product a, const __grid_constant__ Product b) {
  run_roles<BN>(
      &a.ma, &a.mb,
      [&](uint8_t *ring, Barriers *bars, uint32_t rank, volatile int *abort, uint32_t &n) {
        return load_items<BN, true, true, false>(&a.ma, &a.mb, ring, bars, a.p, rank, abort, n) &&
               load_items<BN, false, true, true>(&b.ma, &b.mb, ring, bars, b.p, rank, abort, n);
      },
      [&](uint8_t *ring, Barriers *bars, uint32_t tmem, volatile int *abort, uint32_t &n,
          uint32_t &acc) {
        if (issue_items<BN, true, true, false>(ring, bars, tmem, a.p, abort, n, acc))
          issue_items<BN, false, true, true>(ring, bars, tmem, b.p, abort, n, acc);
      },
      [&](uint8_t *stage, Barriers *bars, uint32_t tmem, uint32_t rank, int warp, int lane,
          volatile int *abort, uint32_t &acc) {
        if (finish_items<BN, AG_ACT_NONE, false, W_BOXES, false>(stage, bars, tmem, a.p, &a.maps, rank, warp,
                                                       lane, abort, acc))
          finish_items<BN, ACT, SLOPE, X_BOXES, true>(stage, bars, tmem, b.p, &b.maps, rank, warp, lane,
                                             abort, acc);
      });
}

// kKernel(products...) on so many clusters.
template <int BN, auto kKernel, typename... P>
cudaError_t launch_clusters(int clusters, cudaStream_t stream, const P &...products) {
  static std::once_flag once[64];
  static cudaError_t once_err[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::call_once(once[dev], [&] {
    once_err[dev] = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem_bytes<BN>()));
    // The register split waits for ever on a launch with fewer registers.
    cudaFuncAttributes fa;
    if (once_err[dev] == cudaSuccess) once_err[dev] = cudaFuncGetAttributes(&fa, kKernel);
    if (once_err[dev] == cudaSuccess && static_cast<uint32_t>(fa.numRegs) < kRegsLaunch)
      once_err[dev] = cudaErrorInvalidConfiguration;
  });
  if (once_err[dev] != cudaSuccess) return once_err[dev];
  return launch_after_previous(kKernel, 2 * clusters, kThreads, smem_bytes<BN>(), stream,
                               products...);
}

template <int BN, bool A_MN, bool B_MN, bool SLOPE>
cudaError_t launch_act(const Gemm &g, const Product &a) {
  // The activation is compiled into the box epilogue; the plain one looks it up.
  // Partial sums have none yet.
  const int n = min(a.p.items, g.num_sms / 2);
  const cudaStream_t s = g.stream;
  if (!a.p.boxes)
    return launch_clusters<BN, linear_gemm_kernel<BN, A_MN, B_MN, AG_ACT_NONE, false, false>>(n, s, a);
  if constexpr (!A_MN) {
    switch (a.p.epi.act) {
      case AG_ACT_RELU:
        return launch_clusters<BN, linear_gemm_kernel<BN, A_MN, B_MN, AG_ACT_RELU, SLOPE, true>>(n, s, a);
      case AG_ACT_GELU:
        return launch_clusters<BN, linear_gemm_kernel<BN, A_MN, B_MN, AG_ACT_GELU, SLOPE, true>>(n, s, a);
      case AG_ACT_GELU_TANH:
        return launch_clusters<BN, linear_gemm_kernel<BN, A_MN, B_MN, AG_ACT_GELU_TANH, SLOPE, true>>(n, s, a);
      case AG_ACT_SILU:
        return launch_clusters<BN, linear_gemm_kernel<BN, A_MN, B_MN, AG_ACT_SILU, SLOPE, true>>(n, s, a);
      default: break;
    }
  }
  return launch_clusters<BN, linear_gemm_kernel<BN, A_MN, B_MN, AG_ACT_NONE, false, true>>(n, s, a);
}

template <int BN>
cudaError_t launch_pair(const Gemm &g, const Product &a, const Product &b) {
  const int n = g.num_sms / 2;
  const cudaStream_t s = g.stream;
  constexpr int kNone = AG_ACT_NONE;
  if (!b.p.boxes)
    return a.p.boxes
               ? launch_clusters<BN, linear_gemm_pair_kernel<BN, kNone, false, true, false>>(n, s, a, b)
               : launch_clusters<BN, linear_gemm_pair_kernel<BN, kNone, false, false, false>>(n, s, a, b);
  switch (b.p.epi.act) {
    case AG_ACT_RELU:
      return launch_clusters<BN, linear_gemm_pair_kernel<BN, AG_ACT_RELU, true, true, true>>(n, s, a, b);
    case AG_ACT_GELU:
      return launch_clusters<BN, linear_gemm_pair_kernel<BN, AG_ACT_GELU, true, true, true>>(n, s, a, b);
    case AG_ACT_GELU_TANH:
      return launch_clusters<BN, linear_gemm_pair_kernel<BN, AG_ACT_GELU_TANH, true, true, true>>(n, s, a, b);
    case AG_ACT_SILU:
      return launch_clusters<BN, linear_gemm_pair_kernel<BN, AG_ACT_SILU, true, true, true>>(n, s, a, b);
    default:
      return launch_clusters<BN, linear_gemm_pair_kernel<BN, kNone, false, true, true>>(n, s, a, b);
  }
}

// A matrix [parts][rows][cols] (cols dense, ld apart) in boxes of `box_rows`
// rows x `box_cols` columns, whose rows are 64 or 128 bytes.
bool encode_map(const Gemm &g, CUtensorMap *m, const void *at, int size, int64_t parts, int64_t rows,
                int64_t cols, int64_t ld, int box_rows, int box_cols) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(parts)};
  // (With one part the outer stride is never used, but has to be a valid one.)
  const cuuint64_t row = static_cast<cuuint64_t>(ld) * size;
  const cuuint64_t strides[2] = {row, parts > 1 ? row * rows : row};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t step[3] = {1, 1, 1};
  return g.encode(m,
                  size == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16,
                  parts ? 3 : 2, const_cast<void *>(at), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE,
                  box_cols * size == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool boxable(const void *p, int64_t ld, int size) {
  return !p || (aligned(p, 16) && ld * size % 16 == 0);
}

}  // namespace gemm

namespace gemm {
namespace {
// The kernel's argument for a product; false if a tensor map cannot be made.
bool prepare(const Gemm &g, Turns turns, Product *a) {
  Params &p = a->p;
  p = Params{};
  p.M = g.M, p.N = g.N;
  p.tiles_m = static_cast<int>((g.M + 255) / 256);
  p.tiles_n = static_cast<int>((g.N + g.plan.bn - 1) / g.plan.bn);
  p.k_tiles = static_cast<int>((g.K + 63) / 64);
  p.splits = g.plan.splits;
  p.items = p.tiles_m * p.tiles_n * p.splits;
  p.turns = turns;
  p.idesc = idesc_half_f32(256, g.plan.bn, g.epi.dtype == AG_BF16, g.a_mn, g.b_mn);
  p.err = g.err;
  p.epi = g.epi;
  if (p.splits > 1) {  // plain float32 sums; linear_join_kernel does the rest
    p.epi = LinearEpilogue{};
    p.epi.out = g.partial, p.epi.ld_out = partial_ld(g.N);
    p.epi.out_dtype = AG_F32, p.epi.dtype = g.epi.dtype;
  }
  const LinearEpilogue &e = p.epi;
  const int out_size = e.out_dtype == AG_F32 ? 4 : 2;
  p.wide = e.out_dtype == AG_F32;
  p.boxes = boxable(e.out, e.ld_out, out_size) && boxable(e.residual, e.ld_res, out_size) &&
            boxable(e.pre_in, e.ld_pre_in, 2) && boxable(e.pre_out, e.ld_pre_out, 2);
  a->maps = EpiMaps{};
  const Operand &A = g.A, &B = g.B;
  bool ok = encode_map(g, &a->ma, A.p, 2, 0, A.rows, A.cols, A.ld, g.a_mn ? 64 : 128, 64) &&
            encode_map(g, &a->mb, B.p, 2, 0, B.rows, B.cols, B.ld, g.b_mn ? 64 : g.plan.bn / 2, 64);
  if (p.boxes) {
    EpiMaps &maps = a->maps;
    const int width = p.wide ? 32 : g.plan.bn / 4;
    ok = ok && encode_map(g, &maps.out, e.out, out_size, p.splits, g.M, g.N, e.ld_out, 32, width);
    if (e.residual)
      ok = ok && encode_map(g, &maps.in, e.residual, out_size, 0, g.M, g.N, e.ld_res, 32, width);
    if (e.pre_in)
      ok = ok && encode_map(g, &maps.in, e.pre_in, 2, 0, g.M, g.N, e.ld_pre_in, 32, width);
    if (e.pre_out)
      ok = ok && encode_map(g, &maps.pre, e.pre_out, 2, 1, g.M, g.N, e.ld_pre_out, 32, width);
  }
  return ok;
}
}  // namespace
}  // namespace gemm

cudaError_t launch_gemm(const Gemm &g) {
  using namespace gemm;
  Product a;
  if (!prepare(g, Turns{0, 0}, &a)) return cudaErrorInvalidValue;
  if (g.plan.bn == 256) {
    if (g.a_mn) return launch_act<256, true, true, false>(g, a);
    return g.b_mn ? launch_act<256, false, true, true>(g, a)
                  : launch_act<256, false, false, false>(g, a);
  }
  if (g.a_mn) return launch_act<128, true, true, false>(g, a);
  return g.b_mn ? launch_act<128, false, true, true>(g, a)
                : launch_act<128, false, false, false>(g, a);
}

cudaError_t launch_gemm_pair(const Gemm &dW, const Gemm &dx, Turns turns, bool *done) {
  using namespace gemm;
  Product a, b;
  *done = false;
  if (!prepare(dW, Turns{0, 0}, &a) || !prepare(dx, turns, &b)) return cudaErrorInvalidValue;
  if (!a.p.boxes && b.p.boxes) return cudaSuccess;
  *done = true;
  return dx.plan.bn == 256 ? launch_pair<256>(dx, a, b) : launch_pair<128>(dx, a, b);
}

}  // namespace ag
