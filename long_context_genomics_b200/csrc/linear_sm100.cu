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
// registers.  With two accumulators in tensor memory the tensor core goes on
// with the next 512 terms meanwhile, so this costs no time: the same path also
// overlaps one tile's epilogue with the next tile's products.
//
// Roles per CTA: warp 0 loads, warp 1 issues the products (even CTA) or tells
// the even CTA that this one's loads have landed (odd CTA), warps 4 to 11 take
// over the accumulators and finish the tile.  Each of those holds 32 rows x
// BN / 2 columns of sums in registers, turns them through shared memory 32
// columns at a time, and applies the epilogue to whole rows' pieces.
//
// A small C does not fill the GPU: the summed dimension is then split between
// clusters, each writing float32 partial sums that a second kernel
// (linear_join_kernel) adds in order and finishes.
#include <mutex>

#include "ag_internal.h"
#include "linear_epilogue.cuh"
#include "linear_gemm.h"
#include "sm100.cuh"

namespace ag {
namespace gemm {

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kFirstEpiWarp = 4;
constexpr int kStepBytes = 128;                  // 64 16-bit terms
constexpr int kPromote = 8;                      // k tiles per accumulator: 512 terms
constexpr uint32_t kRegsLaunch = 168, kRegsLow = 72, kRegsHigh = 216;
static_assert(128 * kRegsLow + 256 * kRegsHigh <= kThreads * kRegsLaunch,
              "the epilogue's registers come out of the role warps' release");

template <int BN>
struct Shape {
  static constexpr int kStages = BN == 256 ? 6 : 8;
  static constexpr int kABytes = 128 * kStepBytes;
  static constexpr int kBBytes = BN / 2 * kStepBytes;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kCols = 2 * BN;           // tensor-memory columns
};
constexpr int kStageOutBytes = kEpiWarps * 32 * 32 * 4;

struct Barriers {
  uint64_t full[8], empty[8];
  uint64_t acc_full[2], acc_free[2];
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
  kSiteLoad = 30, kSiteRelay = 31, kSiteIssue = 32, kSiteAccFree = 33, kSiteAccFull = 34
};

struct Params {
  int64_t M, N;               // rows and columns of C
  int64_t items;              // tiles x splits
  int tiles_m, tiles_n, k_tiles, splits;
  float *partial;             // splits > 1: [splits][M][ld_partial]
  int64_t ld_partial;
  uint32_t idesc;
  unsigned *err;
  LinearEpilogue epi;
};

// Work item -> tile and range of k tiles.  Tiles along M come first, so that
// the clusters at work share B's tiles and pass over A together.
struct Item {
  int tm, tn, split, kb, ke;
};
__device__ __forceinline__ Item item_at(const Params &p, int64_t i) {
  Item t;
  const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
  t.split = static_cast<int>(i / tiles);
  const int64_t r = i - t.split * tiles;
  t.tn = static_cast<int>(r / p.tiles_m);
  t.tm = static_cast<int>(r - static_cast<int64_t>(t.tn) * p.tiles_m);
  t.kb = static_cast<int>(static_cast<int64_t>(p.k_tiles) * t.split / p.splits);
  t.ke = static_cast<int>(static_cast<int64_t>(p.k_tiles) * (t.split + 1) / p.splits);
  return t;
}

// One 64-deep tile of `rows` rows of an operand: K-major, one box of 64 terms
// x rows; MN-major, boxes of 64 rows x 64 terms.
template <bool MN, int ROWS>
__device__ __forceinline__ void load_tile(uint8_t *dst, const CUtensorMap *map, uint64_t *bar,
                                          int row, int k) {
  if constexpr (MN) {
#pragma unroll
    for (int q = 0; q < ROWS / 64; ++q)
      tma_load_2d(dst + q * 64 * kStepBytes, map, bar, row + 64 * q, k);
  } else {
    tma_load_2d(dst, map, bar, k, row);
  }
}

template <int BN, bool A_MN, bool B_MN>
__device__ __forceinline__ void load_role(const CUtensorMap *ma, const CUtensorMap *mb,
                                          uint8_t *ring, Barriers *bars, const Params &p,
                                          uint32_t rank, volatile int *abort) {
  using S = Shape<BN>;
  uint32_t n = 0;
  bool ok = true;
  for (int64_t i = blockIdx.x / 2; ok && i < p.items; i += gridDim.x / 2) {
    const Item t = item_at(p, i);
    const int row_a = t.tm * 256 + static_cast<int>(rank) * 128;
    const int row_b = t.tn * BN + static_cast<int>(rank) * (BN / 2);
    for (int k = t.kb; k < t.ke; ++k) {
      const uint32_t s = n % S::kStages;
      ok = mbar_wait(&bars->empty[s], ((n / S::kStages) & 1u) ^ 1u, abort, p.err, kSiteLoad);
      if (!ok) break;
      uint8_t *at = ring + s * S::kStageBytes;
      mbar_arrive_expect_tx(&bars->full[s], S::kStageBytes);
      load_tile<A_MN, 128>(at, ma, &bars->full[s], row_a, k * 64);
      load_tile<B_MN, BN / 2>(at + S::kABytes, mb, &bars->full[s], row_b, k * 64);
      ++n;
    }
  }
  // Every copy this thread started lands before the CTA exits.
  for (uint32_t i = n > S::kStages ? n - S::kStages : 0; i < n; ++i) {
    const uint32_t a = smem_u32(&bars->full[i % S::kStages]);
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_test(a, (i / S::kStages) & 1u))
      if (globaltimer_ns() - t0 > kWaitLimitNs) break;
  }
}

template <int BN>
__device__ __forceinline__ void relay_role(Barriers *bars, const Params &p, volatile int *abort) {
  using S = Shape<BN>;
  uint32_t n = 0;
  for (int64_t i = blockIdx.x / 2; i < p.items; i += gridDim.x / 2) {
    const Item t = item_at(p, i);
    for (int k = t.kb; k < t.ke; ++k, ++n) {
      const uint32_t s = n % S::kStages;
      if (!mbar_wait(&bars->full[s], (n / S::kStages) & 1u, abort, p.err, kSiteRelay)) return;
      mbar_arrive_cluster(cluster_addr(&bars->full[s], 0));
    }
  }
}

// The whole warp of the even CTA; one elected lane issues.
template <int BN, bool A_MN, bool B_MN>
__device__ __forceinline__ void issue_role(uint8_t *ring, Barriers *bars, uint32_t tmem,
                                           const Params &p, volatile int *abort) {
  using S = Shape<BN>;
  constexpr uint32_t kHi = desc_sw128_hi(1024);  // 8-row groups 1 KB apart, either major
  constexpr uint32_t kAtom = 64 * kStepBytes;    // MN-major: the next 64 rows
  // 16 terms further: 32 bytes along a K-major row, 16 rows of an MN-major tile.
  constexpr uint32_t kAStep = (A_MN ? 16 * kStepBytes : 32) >> 4;
  constexpr uint32_t kBStep = (B_MN ? 16 * kStepBytes : 32) >> 4;
  uint32_t n = 0, acc = 0;
  bool ok = true;
  for (int64_t i = blockIdx.x / 2; ok && i < p.items; i += gridDim.x / 2) {
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
  // Everything this warp issued completes before tensor memory is freed.
  umma2_commit_self_w(&bars->drain);
  const uint32_t a = smem_u32(&bars->drain);
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_test(a, 0))
    if (globaltimer_ns() - t0 > kWaitLimitNs) break;
}

// 32 rows x 32 columns of sums (this lane's row in v) through the warp's part
// of shared memory and out.  Float4 q of row r lies in slot q ^ (r % 8) of its
// 128-byte row: neither the writes (8 lanes, 8 rows) nor the reads (4 pieces of
// 2 rows) meet in a bank.
template <int V>
__device__ __forceinline__ void finish_piece(const Params &p, float *stage, int64_t row0,
                                             int64_t col0, int split, int lane) {
  const LinearEpilogue &e = p.epi;
  constexpr int kLanes = 32 / V;                 // lanes per row
  const int64_t col = col0 + (lane % kLanes) * V;
  if (col >= p.N) return;
  float bias[V];
#pragma unroll
  for (int i = 0; i < V; ++i) bias[i] = p.splits == 1 && e.bias ? __ldg(e.bias + col + i) : 0.f;
#pragma unroll 1
  for (int r = lane / kLanes; r < 32; r += 32 / kLanes) {
    if (row0 + r >= p.M) break;
    float v[V];
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const int c = (lane % kLanes) * V + i;     // column within the piece
      if constexpr (V == 8) {
        const float4 f = *reinterpret_cast<const float4 *>(stage + r * 32 + (((c >> 2) ^ (r & 7)) << 2));
        v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
      } else {
        v[i] = stage[r * 32 + (((c >> 2) ^ (r & 7)) << 2) + (c & 3)];
      }
    }
    if (p.splits > 1)
      store_values<V>(p.partial, (split * p.M + row0 + r) * p.ld_partial + col, AG_F32, v);
    else
      linear_finish<V>(e, v, bias, row0 + r, col);
  }
}

template <int BN>
__device__ __forceinline__ void epilogue_role(float *stage, Barriers *bars, uint32_t tmem,
                                              const Params &p, uint32_t rank, int warp, int lane,
                                              volatile int *abort) {
  constexpr int kHalf = BN / 2;                  // columns per warp
  const int quarter = warp % 4, half = (warp - kFirstEpiWarp) / 4;
  const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t free_bar = cluster_addr(&bars->acc_free[0], 0);
  float *own = stage + (warp - kFirstEpiWarp) * 32 * 32;
  uint32_t acc = 0;
  for (int64_t i = blockIdx.x / 2; i < p.items; i += gridDim.x / 2) {
    const Item t = item_at(p, i);
    float sum[kHalf];
#pragma unroll
    for (int c = 0; c < kHalf; ++c) sum[c] = 0.f;
    for (int k0 = t.kb; k0 < t.ke; k0 += kPromote, ++acc) {
      const uint32_t b = acc & 1u;
      if (!mbar_wait_warp(&bars->acc_full[b], (acc >> 1) & 1u, abort, p.err, kSiteAccFull)) return;
      tc_fence_after();
      const uint32_t at = tmem + lanes + BN * b + kHalf * half;
#pragma unroll
      for (int c = 0; c < kHalf; c += 32) {
        uint32_t r[32];
        tmem_ld32(at + c, r);
        tmem_wait_ld(r);
#pragma unroll
        for (int q = 0; q < 32; ++q) sum[c + q] += __uint_as_float(r[q]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(free_bar + 8 * b);
    }
    const int64_t row0 = static_cast<int64_t>(t.tm) * 256 + rank * 128 + quarter * 32;
    const int64_t col0 = static_cast<int64_t>(t.tn) * BN + kHalf * half;
#pragma unroll
    for (int c = 0; c < kHalf; c += 32) {
      __syncwarp();
#pragma unroll
      for (int q = 0; q < 8; ++q)
        *reinterpret_cast<float4 *>(own + lane * 32 + ((q ^ (lane & 7)) << 2)) =
            make_float4(sum[c + 4 * q], sum[c + 4 * q + 1], sum[c + 4 * q + 2], sum[c + 4 * q + 3]);
      __syncwarp();
      if (p.splits > 1 || p.epi.vec8)
        finish_piece<8>(p, own, row0, col0 + c, t.split, lane);
      else
        finish_piece<1>(p, own, row0, col0 + c, t.split, lane);
    }
  }
}

template <int BN, bool A_MN, bool B_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    linear_gemm_kernel(const __grid_constant__ CUtensorMap ma,
                       const __grid_constant__ CUtensorMap mb, const __grid_constant__ Params p) {
  using S = Shape<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float *stage = reinterpret_cast<float *>(ring + S::kStages * S::kStageBytes);
  Barriers *bars = reinterpret_cast<Barriers *>(reinterpret_cast<uint8_t *>(stage) + kStageOutBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&bars->full[s], rank == 0 ? 2 : 1);  // own loads (+ the odd CTA's relay)
      mbar_init(&bars->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->acc_full[b], 1);
      mbar_init(&bars->acc_free[b], 2 * kEpiWarps);
    }
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    fence_mbar_init();
    prefetch_tensormap(&ma);
    prefetch_tensormap(&mb);
  }
  if (warp == 1) {
    tmem_alloc2(&bars->tmem_base, S::kCols);
    tmem_relinquish2();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  volatile int *abort = &bars->abort;
  if (warp < kFirstEpiWarp) {
    regs_dec<kRegsLow>();
    if (warp == 1 && rank == 0) {
      issue_role<BN, A_MN, B_MN>(ring, bars, tmem, p, abort);
    } else if (lane == 0) {
      if (warp == 0)
        load_role<BN, A_MN, B_MN>(&ma, &mb, ring, bars, p, rank, abort);
      else if (warp == 1)
        relay_role<BN>(bars, p, abort);
    }
  } else {
    regs_inc<kRegsHigh>();
    epilogue_role<BN>(stage, bars, tmem, p, rank, warp, lane, abort);
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

template <int BN, bool A_MN, bool B_MN>
cudaError_t launch(const Gemm &g, const Params &p, const CUtensorMap &ma, const CUtensorMap &mb) {
  static std::once_flag once[64];
  static cudaError_t once_err[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  auto *kernel = linear_gemm_kernel<BN, A_MN, B_MN>;
  std::call_once(once[dev], [&] {
    once_err[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem_bytes<BN>()));
    // The register split waits for ever on a launch with fewer registers.
    cudaFuncAttributes fa;
    if (once_err[dev] == cudaSuccess) once_err[dev] = cudaFuncGetAttributes(&fa, kernel);
    if (once_err[dev] == cudaSuccess && static_cast<uint32_t>(fa.numRegs) < kRegsLaunch)
      once_err[dev] = cudaErrorInvalidConfiguration;
  });
  if (once_err[dev] != cudaSuccess) return once_err[dev];
  const int64_t clusters = p.items < g.num_sms / 2 ? p.items : g.num_sms / 2;
  kernel<<<static_cast<unsigned>(2 * clusters), kThreads, smem_bytes<BN>(), g.stream>>>(ma, mb, p);
  return cudaGetLastError();
}

// A 16-bit operand [rows][cols] (cols dense, ld apart) as boxes of 64 columns
// and `box_rows` rows.
bool encode_map(const Gemm &g, CUtensorMap *m, const Operand &o, int box_rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(o.cols), static_cast<cuuint64_t>(o.rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(o.ld) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t step[2] = {1, 1};
  return g.encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void *>(o.p), dims, strides, box,
                  step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace gemm

cudaError_t launch_gemm(const Gemm &g) {
  using namespace gemm;
  Params p{};
  p.M = g.M, p.N = g.N;
  p.tiles_m = static_cast<int>((g.M + 255) / 256);
  p.tiles_n = static_cast<int>((g.N + g.plan.bn - 1) / g.plan.bn);
  p.k_tiles = static_cast<int>((g.K + 63) / 64);
  p.splits = g.plan.splits;
  p.items = static_cast<int64_t>(p.tiles_m) * p.tiles_n * p.splits;
  p.partial = g.partial, p.ld_partial = partial_ld(g.N);
  p.idesc = idesc_half_f32(256, g.plan.bn, g.epi.dtype == AG_BF16, g.a_mn, g.b_mn);
  p.err = g.err;
  p.epi = g.epi;
  CUtensorMap ma, mb;
  if (!encode_map(g, &ma, g.A, g.a_mn ? 64 : 128) ||
      !encode_map(g, &mb, g.B, g.b_mn ? 64 : g.plan.bn / 2))
    return cudaErrorInvalidValue;
  if (g.plan.bn == 256) {
    if (g.a_mn) return launch<256, true, true>(g, p, ma, mb);
    return g.b_mn ? launch<256, false, true>(g, p, ma, mb) : launch<256, false, false>(g, p, ma, mb);
  }
  if (g.a_mn) return launch<128, true, true>(g, p, ma, mb);
  return g.b_mn ? launch<128, false, true>(g, p, ma, mb) : launch<128, false, false>(g, p, ma, mb);
}

}  // namespace ag
