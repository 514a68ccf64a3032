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
// BN / 2 columns of sums in registers, one row per lane.  Where every array of
// the epilogue is one that TMA can address, a warp reads the residual (or the
// pre-activation of a derivative) and writes the results as 32-row boxes of
// shared memory, so that the tile's memory traffic is asynchronous and whole
// lines; odd row strides take plain loads and stores, turned through shared
// memory so that they are at least contiguous.
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
  static constexpr int kStages = BN == 256 ? 5 : 6;
  static constexpr int kABytes = 128 * kStepBytes;
  static constexpr int kBBytes = BN / 2 * kStepBytes;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kCols = 2 * BN;           // tensor-memory columns
};
// Per epilogue warp: two boxes of 32 rows x 128 bytes.
constexpr int kBoxBytes = 32 * 128;
constexpr int kStageOutBytes = kEpiWarps * 2 * kBoxBytes;

struct Barriers {
  uint64_t full[8], empty[8];
  uint64_t acc_full[2], acc_free[2];
  uint64_t in_full[kEpiWarps][2];
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
  kSiteLoad = 30, kSiteRelay = 31, kSiteIssue = 32, kSiteAccFree = 33, kSiteAccFull = 34,
  kSiteIn = 35
};

struct Params {
  int64_t M, N;               // rows and columns of C
  int64_t items;              // tiles x splits
  int tiles_m, tiles_n, k_tiles, splits;
  int boxes;                  // every array of the epilogue is TMA's to read or write
  int wide;                   // the output is float32
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

// Tensor maps of the epilogue's arrays (read when p.boxes): the output, or with
// splits the partial sums [splits][M][N]; the residual or the pre-activation
// that is read; the pre-activation that is written.
struct EpiMaps {
  CUtensorMap out, in, pre;
};

// Eight sums of a row -> the layer's eight results, in the order of the header:
// bias, pre-activation, activation (or a derivative), residual.
template <int ACT, bool SLOPE>
__device__ __forceinline__ void finish8(float (&v)[8], const float (&bias)[8], const float (&in)[8],
                                        bool residual) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (SLOPE) {
      v[i] *= act_slope<ACT>(in[i]);
    } else {
      v[i] = act_value<ACT>(v[i]);
      if (residual) v[i] += in[i];
    }
  }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8], bool bf16) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (bf16) {
      w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    } else {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void unpack8(uint4 u, bool bf16, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (bf16) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
}

// One warp's 32 rows x COLS columns through boxes of 128-byte rows.  WIDE:
// float32 results, 32 columns a box; otherwise 64 16-bit columns.  A box holds
// the residual first and the results in its place after; a pre-activation has
// the second box to itself (of 64-byte rows beside float32 results).
template <int COLS, int ACT, bool SLOPE, bool WIDE>
struct BoxEpilogue {
  static constexpr int kWidth = WIDE ? 32 : 64, kPieces = COLS / kWidth;
  const Params &p;
  const EpiMaps *maps;
  uint8_t *own;               // two boxes
  uint64_t *in_full;          // their barriers
  volatile int *abort;
  int lane;
  uint32_t phase = 0;         // bit b: parity of the next read of box b to wait for
  uint32_t issued = 0;        // bit b: parity of the next read of box b to start
  uint32_t turn = 0;          // pieces stored so far; without a pre_box() they alternate boxes

  __device__ bool pre_box() const { return SLOPE || p.epi.pre_out; }
  __device__ bool reads() const { return SLOPE || p.epi.residual; }
  __device__ bool valid(int64_t row0, int64_t col0, int j) const {
    return row0 < p.M && col0 + j * kWidth < p.N;
  }

  // Start reading piece j's residual or pre-activation, `ahead` pieces after
  // the next one to be stored.  The earlier stores out of both boxes have been
  // read out, and the box's earlier reads are ordered by the fence before those.
  __device__ void start_read(int64_t row0, int64_t col0, int j, int ahead) {
    if (!valid(row0, col0, j)) return;
    const int box = pre_box() ? (SLOPE ? 1 : 0) : ((turn + ahead) & 1);
    issued ^= 1u << box;
    if (lane != 0) return;
    bulk_wait_read_all();
    mbar_arrive_expect_tx(&in_full[box], SLOPE && WIDE ? kBoxBytes / 2 : kBoxBytes);
    tma_load_2d(own + box * kBoxBytes, &maps->in, &in_full[box], static_cast<int>(col0) + j * kWidth,
                static_cast<int>(row0));
  }
  __device__ void begin(int64_t row0, int64_t col0) {
    if (!reads()) return;
    start_read(row0, col0, 0, 0);
    if (!pre_box() && kPieces > 1) start_read(row0, col0, 1, 1);
  }
  // Every copy this warp started ends before the CTA does: its stores, and
  // after a failure the boxes still being read.
  __device__ void drain() {
    if (lane == 0) {
      for (int b = 0; b < 2; ++b) {
        const uint64_t t0 = globaltimer_ns();
        while (((issued ^ phase) >> b) & 1u) {
          if (mbar_test(smem_u32(&in_full[b]), (phase >> b) & 1u)) break;
          if (globaltimer_ns() - t0 > kWaitLimitNs) break;
        }
      }
      bulk_wait_all();
    }
    __syncwarp();
  }

  __device__ bool finish(const float2 (&sum)[COLS / 2], int64_t row0, int64_t col0, int split) {
    const bool bf16 = p.epi.dtype == AG_BF16, two = !pre_box(), in = reads();
    const float *bias_p = p.splits == 1 ? p.epi.bias : nullptr;
    const bool bias_vec = (reinterpret_cast<uintptr_t>(bias_p) & 15) == 0;
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      if (!valid(row0, col0, j)) break;
      const int64_t col = col0 + j * kWidth;
      const int box = two ? (turn & 1) : 0;
      uint8_t *y = own + box * kBoxBytes + lane * 128, *z = own + kBoxBytes;
      if (in) {
        const int ib = SLOPE ? 1 : box;
        if (!mbar_wait_warp(&in_full[ib], (phase >> ib) & 1u, abort, p.err, kSiteIn)) return false;
        phase ^= 1u << ib;  // (start_read has waited for the boxes' stores)
      } else {
        if (lane == 0) {
          if (two) bulk_wait_read_but_one();
          else bulk_wait_read_all();
        }
        __syncwarp();
      }
#pragma unroll
      for (int g = 0; g < kWidth / 8; ++g) {
        float v[8], b[8], x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 s = sum[(j * kWidth + g * 8) / 2 + i];
          v[2 * i] = s.x, v[2 * i + 1] = s.y;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = 0.f, x[i] = 0.f;
        if (bias_p) {
          const int64_t c = col + g * 8;
          if (bias_vec && c + 8 <= p.N) {
            const float4 lo = __ldg(reinterpret_cast<const float4 *>(bias_p + c));
            const float4 hi = __ldg(reinterpret_cast<const float4 *>(bias_p + c) + 1);
            b[0] = lo.x, b[1] = lo.y, b[2] = lo.z, b[3] = lo.w;
            b[4] = hi.x, b[5] = hi.y, b[6] = hi.z, b[7] = hi.w;
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (c + i < p.N) b[i] = __ldg(bias_p + c + i);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] += b[i];
        }
        // 16-byte chunks of this lane's row: of 128 bytes with the 128-byte
        // swizzle, of 64 bytes with the 64-byte one.
        uint4 *y16 = reinterpret_cast<uint4 *>(y + ((g ^ (lane & 7)) << 4));
        uint4 *z16 = reinterpret_cast<uint4 *>(
            WIDE ? z + lane * 64 + ((g ^ ((lane >> 1) & 3)) << 4)
                 : z + lane * 128 + ((g ^ (lane & 7)) << 4));
        float4 *yw0 = reinterpret_cast<float4 *>(y + (((2 * g) ^ (lane & 7)) << 4));
        float4 *yw1 = reinterpret_cast<float4 *>(y + (((2 * g + 1) ^ (lane & 7)) << 4));
        if constexpr (SLOPE) {
          unpack8(*z16, bf16, x);
        } else {
          if (p.epi.pre_out) *z16 = pack8(v, bf16);
          if (in) {
            if constexpr (WIDE) {
              const float4 lo = *yw0, hi = *yw1;
              x[0] = lo.x, x[1] = lo.y, x[2] = lo.z, x[3] = lo.w;
              x[4] = hi.x, x[5] = hi.y, x[6] = hi.z, x[7] = hi.w;
            } else {
              unpack8(*y16, bf16, x);
            }
          }
        }
        finish8<ACT, SLOPE>(v, b, x, in);
        if constexpr (WIDE) {
          *yw0 = make_float4(v[0], v[1], v[2], v[3]);
          *yw1 = make_float4(v[4], v[5], v[6], v[7]);
        } else {
          *y16 = pack8(v, bf16);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_3d(&maps->out, own + box * kBoxBytes, static_cast<int>(col),
                     static_cast<int>(row0), split);
        if (!SLOPE && p.epi.pre_out)
          tma_store_3d(&maps->pre, z, static_cast<int>(col), static_cast<int>(row0), 0);
        bulk_commit_group();
      }
      ++turn;
      const int ahead = two ? 1 : 0;
      if (in && j + 1 + ahead < kPieces) start_read(row0, col0, j + 1 + ahead, ahead);
    }
    return true;
  }
};

// The same without boxes: 32 columns at a time through a box's memory (float4
// q of row r in slot q ^ (r % 8)), then a lane per column, row by row.
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
      const float bias[1] = {p.epi.bias ? __ldg(p.epi.bias + col) : 0.f};
#pragma unroll 1
      for (int r = 0; r < 32 && row0 + r < p.M; ++r) {
        float v[1] = {stage[r * 32 + (((lane >> 2) ^ (r & 7)) << 2) + (lane & 3)]};
        linear_finish<1>(p.epi, v, bias, row0 + r, col);
      }
    }
  }
}

template <int BN, int ACT, bool SLOPE, bool WIDE, bool BOXES>
__device__ __forceinline__ void epilogue_role(uint8_t *stage, Barriers *bars, uint32_t tmem,
                                              const Params &p, const EpiMaps *maps, uint32_t rank,
                                              int warp, int lane, volatile int *abort) {
  constexpr int kHalf = BN / 2;                  // columns per warp
  const int quarter = warp % 4, half = (warp - kFirstEpiWarp) / 4;
  const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t free_bar = cluster_addr(&bars->acc_free[0], 0);
  uint8_t *own = stage + (warp - kFirstEpiWarp) * 2 * kBoxBytes;
  BoxEpilogue<kHalf, ACT, SLOPE, WIDE> boxes{
      p, maps, own, bars->in_full[warp - kFirstEpiWarp], abort, lane};
  uint32_t acc = 0;
  bool ok = true;
  for (int64_t i = blockIdx.x / 2; ok && i < p.items; i += gridDim.x / 2) {
    const Item t = item_at(p, i);
    const int64_t row0 = static_cast<int64_t>(t.tm) * 256 + rank * 128 + quarter * 32;
    const int64_t col0 = static_cast<int64_t>(t.tn) * BN + kHalf * half;
    if constexpr (BOXES) boxes.begin(row0, col0);
    float2 sum[kHalf / 2];
#pragma unroll
    for (int c = 0; c < kHalf / 2; ++c) sum[c] = make_float2(0.f, 0.f);
    for (int k0 = t.kb; k0 < t.ke; k0 += kPromote, ++acc) {
      const uint32_t b = acc & 1u;
      ok = mbar_wait_warp(&bars->acc_full[b], (acc >> 1) & 1u, abort, p.err, kSiteAccFull);
      if (!ok) break;
      tc_fence_after();
      const uint32_t at = tmem + lanes + BN * b + kHalf * half;
#pragma unroll
      for (int c = 0; c < kHalf; c += 32) {
        uint32_t r[32];
        tmem_ld32(at + c, r);
        tmem_wait_ld(r);
#pragma unroll
        for (int q = 0; q < 16; ++q)
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
      plain_epilogue<kHalf>(p, sum, reinterpret_cast<float *>(own), row0, col0, lane);
    }
  }
  if constexpr (BOXES) boxes.drain();
}

template <int BN, bool A_MN, bool B_MN, int ACT, bool SLOPE, bool BOXES>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    linear_gemm_kernel(const __grid_constant__ CUtensorMap ma,
                       const __grid_constant__ CUtensorMap mb,
                       const __grid_constant__ EpiMaps maps, const __grid_constant__ Params p) {
  using S = Shape<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *stage = ring + S::kStages * S::kStageBytes;
  Barriers *bars = reinterpret_cast<Barriers *>(stage + kStageOutBytes);
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
    for (int w = 0; w < kEpiWarps; ++w)
      for (int b = 0; b < 2; ++b) mbar_init(&bars->in_full[w][b], 1);
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
    if (BOXES && p.wide)
      epilogue_role<BN, ACT, SLOPE, true, BOXES>(stage, bars, tmem, p, &maps, rank, warp, lane,
                                                 abort);
    else
      epilogue_role<BN, ACT, SLOPE, false, BOXES>(stage, bars, tmem, p, &maps, rank, warp, lane,
                                                  abort);
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
cudaError_t launch(const Gemm &g, const Params &p, const CUtensorMap &ma, const CUtensorMap &mb,
                   const EpiMaps &maps) {
  static std::once_flag once[64];
  static cudaError_t once_err[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  auto *kernel = linear_gemm_kernel<BN, A_MN, B_MN, ACT, SLOPE, BOXES>;
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
  kernel<<<static_cast<unsigned>(2 * clusters), kThreads, smem_bytes<BN>(), g.stream>>>(ma, mb, maps,
                                                                                       p);
  return cudaGetLastError();
}

template <int BN, bool A_MN, bool B_MN, bool SLOPE>
cudaError_t launch_act(const Gemm &g, const Params &p, const CUtensorMap &ma, const CUtensorMap &mb,
                       const EpiMaps &maps) {
  // The activation is compiled into the box epilogue; the plain one looks it up.
  // Partial sums have none yet.
  if (!p.boxes) return launch<BN, A_MN, B_MN, AG_ACT_NONE, false, false>(g, p, ma, mb, maps);
  if constexpr (A_MN) {
    return launch<BN, A_MN, B_MN, AG_ACT_NONE, false, true>(g, p, ma, mb, maps);
  } else {
    switch (p.epi.act) {
      case AG_ACT_RELU: return launch<BN, A_MN, B_MN, AG_ACT_RELU, SLOPE, true>(g, p, ma, mb, maps);
      case AG_ACT_GELU: return launch<BN, A_MN, B_MN, AG_ACT_GELU, SLOPE, true>(g, p, ma, mb, maps);
      case AG_ACT_GELU_TANH:
        return launch<BN, A_MN, B_MN, AG_ACT_GELU_TANH, SLOPE, true>(g, p, ma, mb, maps);
      case AG_ACT_SILU: return launch<BN, A_MN, B_MN, AG_ACT_SILU, SLOPE, true>(g, p, ma, mb, maps);
      default: return launch<BN, A_MN, B_MN, AG_ACT_NONE, false, true>(g, p, ma, mb, maps);
    }
  }
}

// A matrix [parts][rows][cols] (cols dense, ld apart) in boxes of `box_rows`
// rows x `box_cols` columns, whose rows are 64 or 128 bytes.
bool encode_map(const Gemm &g, CUtensorMap *m, const void *at, int size, int64_t parts, int64_t rows,
                int64_t cols, int64_t ld, int box_rows, int box_cols) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(parts)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * size,
                                 static_cast<cuuint64_t>(ld) * size * rows};
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

cudaError_t launch_gemm(const Gemm &g) {
  using namespace gemm;
  Params p{};
  p.M = g.M, p.N = g.N;
  p.tiles_m = static_cast<int>((g.M + 255) / 256);
  p.tiles_n = static_cast<int>((g.N + g.plan.bn - 1) / g.plan.bn);
  p.k_tiles = static_cast<int>((g.K + 63) / 64);
  p.splits = g.plan.splits;
  p.items = static_cast<int64_t>(p.tiles_m) * p.tiles_n * p.splits;
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
  CUtensorMap ma, mb;
  EpiMaps maps{};
  const Operand &A = g.A, &B = g.B;
  bool ok = encode_map(g, &ma, A.p, 2, 0, A.rows, A.cols, A.ld, g.a_mn ? 64 : 128, 64) &&
            encode_map(g, &mb, B.p, 2, 0, B.rows, B.cols, B.ld, g.b_mn ? 64 : g.plan.bn / 2, 64);
  if (p.boxes) {
    const int width = p.wide ? 32 : 64;
    ok = ok && encode_map(g, &maps.out, e.out, out_size, p.splits, g.M, g.N, e.ld_out, 32, width);
    if (e.residual)
      ok = ok && encode_map(g, &maps.in, e.residual, out_size, 0, g.M, g.N, e.ld_res, 32, width);
    if (e.pre_in)
      ok = ok && encode_map(g, &maps.in, e.pre_in, 2, 0, g.M, g.N, e.ld_pre_in, 32, width);
    if (e.pre_out)
      ok = ok && encode_map(g, &maps.pre, e.pre_out, 2, 1, g.M, g.N, e.ld_pre_out, 32, width);
  }
  if (!ok) return cudaErrorInvalidValue;
  if (g.plan.bn == 256) {
    if (g.a_mn) return launch_act<256, true, true, false>(g, p, ma, mb, maps);
    return g.b_mn ? launch_act<256, false, true, true>(g, p, ma, mb, maps)
                  : launch_act<256, false, false, false>(g, p, ma, mb, maps);
  }
  if (g.a_mn) return launch_act<128, true, true, false>(g, p, ma, mb, maps);
  return g.b_mn ? launch_act<128, false, true, true>(g, p, ma, mb, maps)
                : launch_act<128, false, false, false>(g, p, ma, mb, maps);
}

}  // namespace ag
