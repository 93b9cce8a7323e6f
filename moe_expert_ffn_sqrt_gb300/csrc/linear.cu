// Matrix products with a fused epilogue, dense or with one weight per expert, and their gradients
// (bf16 or fp16 operands, fp32 accumulation), on tcgen05 (sm_103a).
//
//   forward   y[r, n]  = act( sum_k x[r, k] w[e, n, k] + bias[e, n] ) + residual[r, n]
//   input     dx[r, k] = sum_n dz[r, n] w[e, n, k] (+ residual[r, k])
//   weight    dw[e, n, k] = sum_r dz[r, n] x[r, k]        over expert e's rows
//
// All three are out[j, i] = sum_q A[i, q] B[j, q] with i the contiguous column of the output: i runs
// over the MMA's M rows (accumulator lanes) and j over its N columns.  So the tokens are on N, where the
// MMA takes any multiple of 16: a ragged or short expert segment costs what it holds.  What changes is
// which operand is contiguous along the sum: w is (forward), w and x are not (gradients); the
// shared-memory descriptors take either order, so no operand is ever transposed in memory.
//
// Rows of experts: expert e's rows start at seg_e = sum_{e' < e} round_up(counts[e'], align) (the layout
// of moe_permute).  Padding rows are never read into a result nor written: in the forward and the input
// gradient a padding row is a column of the product that is not stored; in the weight gradient, where
// rows are summed over, the last partial slab of a segment is fetched row by row with the padding
// rows replaced by out-of-range ones, which read as zeros.
//
// Two kernels:
//  * linear_pair_kernel: a CTA pair per 256 x 256 tile (cta_group::2, each CTA 128 output columns i and
//    half of the tile's rows j in shared memory), persistent, two accumulators so that one tile's
//    epilogue runs under the next tile's MMAs.
//  * linear_split_kernel: for dense problems with too few tiles to fill the GPU: a cluster of up to eight
//    CTAs per 128-column tile, each with a slice of the sum; the slices meet in shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kernels.h"
#include "rows.cuh"

namespace moe {

namespace {

constexpr int kLinThreads = 192;            // warp 0 loads, 1 MMA, 2..5 epilogue
constexpr int kLinBI = 128;                 // output columns i per CTA (accumulator lanes)
constexpr int kLinBJ = 256;                 // output rows j per tile (MMA N), at most
constexpr int kLinSlab = 64;                // terms of the sum per pipeline stage
constexpr int kLinABytes = kLinBI * 128;
constexpr int kLinMaxE = kLinearMaxExperts;
// pair kernel: a stage holds the CTA's 128 rows of A and up to 128 rows of B
constexpr int kPairB = 128 * 128;
constexpr int kPairStage = kLinABytes + kPairB;      // 32 KB
constexpr int kPairStages = 6;
constexpr int kPairSmem = 1024 + kPairStages * kPairStage + 256 + 2 * (kLinMaxE + 1) * 4;
// split kernel: stages of A and the tile's B rows, as many as fit
constexpr int kSplitRing = 208 * 1024;
constexpr int kSplitMaxStages = 12;
constexpr int kSplitSmem = 1024 + kSplitRing + 512;
static_assert(kPairSmem <= 227 * 1024 && kSplitSmem <= 227 * 1024, "shared memory budget");
static_assert(kSplitRing >= kLinBI * kLinBJ * 4, "the slices' sums fit the ring");

enum LinMode { kLinFwd = 0, kLinFwdGated = 1, kLinDx = 2, kLinDw = 3 };

struct LinArgs {
  const int32_t* counts;      // [E] rows per expert; nullptr: one dense segment of `rows` rows
  int E, align, rows;         // rows: rows of the row buffers
  int n_it;                   // i tiles
  int i_ext;                  // output columns (gated forward: of y; z has twice as many)
  int j_ext;                  // weight gradient: N
  int q_ext;                  // forward: K, input gradient: N
  int act, f16;
  int a_blocks, b_blocks;     // > 0: operand map with 64-column blocks as a dimension, blocks per copy
  int b_box;                  // rows of B per copy (operands contiguous along the sum)
  int split, bj, stages;      // split kernel: slices, rows j per tile, ring stages
  uint16_t* out;
  long long ldo;
  uint16_t* z;
  long long ldz;
  const uint16_t* res;
  long long ldr;
  const float* bias;          // [E, N]
  uint32_t* status;
};

// Tile copies (TMA).  PAIR: the completion is counted on the even CTA's barrier (`bar` is its
// shared::cluster address), whichever CTA of the pair the tile lands in.
template <bool PAIR>
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                            uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, int c4,
                                            uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
        : "memory");
}
// Four rows of a map with a one-row box; rows outside the matrix read as zeros.
__device__ __forceinline__ void tma_rows4_pair(uint32_t dst, const CUtensorMap* map, int c0, int y0, int y1, int y2, int y3,
                                               uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(y0), "r"(y1), "r"(y2), "r"(y3), "r"(bar)
      : "memory");
}

// Instruction descriptor of kind::f16 (bf16 or fp16 operands, fp32 accumulation); a_mn / b_mn: the
// operand's tile is contiguous along M / N instead of along the sum.
__device__ __forceinline__ uint32_t lin_idesc(int f16, int a_mn, int b_mn, uint32_t M, uint32_t N) {
  const uint32_t fmt = f16 ? 0u : 1u;
  return (1u << 4) | (fmt << 7) | (fmt << 10) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
         ((N >> 3) << 17) | ((M >> 4) << 24);
}

// 128-byte-swizzled operand tiles.  Contiguous along the sum: rows of 128 bytes (64 terms), 8-row
// groups 1024 bytes apart; one MMA step (16 terms) is 32 bytes further.  Contiguous along M / N: blocks
// of 64 columns x 64 terms (8 KB), each term a row of 128 bytes, 8-term groups 1024 bytes apart and
// blocks 8192 bytes apart; one MMA step is 2048 bytes further.
template <bool MN>
__device__ __forceinline__ uint64_t lin_desc(uint32_t addr) {
  return MN ? smem_desc(addr, 8192, 1024, 2) : smem_desc(addr, 16, 1024, 2);
}
template <bool MN>
constexpr int kLinStep = MN ? 2048 : 32;

// Rows j per tile when n rows are cut into ceil(n / 256) tiles of equal height, a multiple of the MMA's
// step in N (16, over a pair 32): equal tiles keep the CTAs' work even where 256 + a rest would not.
constexpr int kPairStep = 32, kSplitStep = 16;
__host__ __device__ __forceinline__ int lin_tile_rows(int n, int step) {
  const int nj = (n + kLinBJ - 1) / kLinBJ;
  return nj ? ((n + nj - 1) / nj + step - 1) / step * step : step;
}

struct LinTile {
  int e, it, row0, cnt, j0, ncols, slabs;
};

// Tiles in order of expert, then groups of 16 j tiles, then i tile, then j tile: the tiles that run at
// one time share their operands in L2 along both sides.
template <int MODE>
__device__ __forceinline__ LinTile lin_tile(const LinArgs& a, const int* seg, const int* pfx, int t) {
  LinTile r;
  int lo = 0, hi = a.E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pfx[mid] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  r.e = lo;
  r.row0 = seg[lo];
  r.cnt = a.counts ? min(max(__ldg(a.counts + lo), 0), max(a.rows - r.row0, 0)) : a.rows;
  int u = t - pfx[lo];
  const int n = MODE == kLinDw ? a.j_ext : r.cnt;
  const int bj = lin_tile_rows(n, kPairStep), nj = (n + bj - 1) / bj;
  const int g = u / (16 * a.n_it);
  u -= g * 16 * a.n_it;
  const int gj = min(16, nj - g * 16);
  r.it = u / gj;
  r.j0 = (g * 16 + u - r.it * gj) * bj;
  r.ncols = min(bj, n - r.j0);
  r.slabs = ((MODE == kLinDw ? r.cnt : a.q_ext) + kLinSlab - 1) / kLinSlab;
  return r;
}

__device__ __forceinline__ uint32_t lin_pack(float lo, float hi, int f16) {
  if (f16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 lin_unpack(uint32_t w, int f16) {
  if (f16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

__device__ __forceinline__ float lin_silu(float v) { return __fdividef(v, 1.f + __expf(-v)); }
// v Phi(v); erfc keeps its relative accuracy in the negative tail, where 1 + erf would cancel
__device__ __forceinline__ float lin_gelu(float v) { return 0.5f * v * erfcf(v * -0.70710678118654752f); }

// v holds 32 accumulator columns (output rows) of this lane's output column; neighbouring lanes
// exchange halves so that each holds two neighbouring columns of 16 output rows: pair p of an even
// lane is row 2p, of an odd lane row 2p + 1.
__device__ __forceinline__ void lin_pairs(const float (&v)[32], float (&lo)[16], float (&hi)[16]) {
  const bool odd = threadIdx.x & 1;
#pragma unroll
  for (int p = 0; p < 16; ++p) {
    const float got = __shfl_xor_sync(0xffffffffu, odd ? v[2 * p] : v[2 * p + 1], 1);
    lo[p] = odd ? got : v[2 * p];
    hi[p] = odd ? v[2 * p + 1] : got;
  }
}

// Where the epilogue's sums come from: this CTA's tensor memory, or the slices in the shared memory of
// the cluster's CTAs ([column][128 lanes] fp32), added in slice order.
struct TmemSums {
  uint32_t acc;               // this warp's lane quarter, accumulator column 0
  __device__ __forceinline__ void operator()(int c0, int, float (&v)[32]) const {
    uint32_t r[2][16];
    tc_ld_x16(acc + c0, r[0]);
    tc_ld_x16(acc + c0 + 16, r[1]);
    tc_wait_ld();
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j >> 4][j & 15]);
  }
};
struct ZeroSums {
  __device__ __forceinline__ void operator()(int, int, float (&v)[32]) const {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = 0.f;
  }
};
struct ClusterSums {
  uint32_t base;              // this lane's column 0 in the CTA's own shared memory
  int slices;
  __device__ __forceinline__ void operator()(int c0, int left, float (&v)[32]) const {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = 0.f;
    for (int s = 0; s < slices; ++s) {
      const uint32_t p = mapa_shared(base, static_cast<uint32_t>(s)) + static_cast<uint32_t>(c0) * (kLinBI * 4);
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j < left) {
          float x;
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(p + j * (kLinBI * 4)) : "memory");
          v[j] += x;
        }
    }
  }
};

// Turns the sums of output rows [j0 + cb, j0 + ce) of tile t into outputs; this warp has lanes 32q .. of
// the CTA's output columns, which start at column i0 (gated forward: at column i0 of y).
template <int MODE, class Sums>
__device__ __forceinline__ void lin_drain(const LinArgs& a, const LinTile& t, int i0, int cb, int ce, const Sums& sums, int q,
                                          int lane) {
  // output column of this lane.  Gated forward: lanes 0..7 are gate rows, 8..15 the up rows of the same
  // eight columns, 16..31 the next eight columns' likewise.
  const int up = MODE == kLinFwdGated ? (lane >> 3) & 1 : 0;
  const int i = MODE == kLinFwdGated ? i0 + q * 16 + (lane >> 4) * 8 + (lane & 7) : i0 + q * 32 + lane;
  const bool live = i < a.i_ext;           // i_ext is a multiple of 8
  const int i2 = i & ~1, odd = lane & 1;
  const int zcol = MODE == kLinFwdGated ? i + up * a.i_ext : i;
  const int n_all = MODE == kLinFwdGated ? 2 * a.i_ext : a.i_ext;
  float bias = 0.f;
  if ((MODE == kLinFwd || MODE == kLinFwdGated) && a.bias && live)
    bias = __ldg(a.bias + static_cast<size_t>(t.e) * n_all + zcol);
  // output row of accumulator column 0
  const long long jr = MODE == kLinDw ? static_cast<long long>(t.e) * a.j_ext + t.j0 : static_cast<long long>(t.row0) + t.j0;
  // the residual of the next 32 columns is on its way while these are worked on
  constexpr int kWords = MODE == kLinFwdGated ? 8 : 16;
  auto row_of = [&](int p) { return MODE == kLinFwdGated ? 2 * (2 * p + odd) + up : 2 * p + odd; };
  uint32_t res[kWords];
  auto fetch = [&](int c) {
    const uint16_t* rp = a.res + (jr + c) * a.ldr + i2;
#pragma unroll
    for (int p = 0; p < kWords; ++p)
      res[p] = live && c + row_of(p) < ce ? *reinterpret_cast<const uint32_t*>(rp + row_of(p) * a.ldr) : 0u;
  };
  const bool has_res = MODE != kLinDw && a.res != nullptr;
  if (has_res) fetch(cb);
#pragma unroll 1
  for (int c0 = cb; c0 < ce; c0 += 32) {
    const int left = ce - c0;
    float v[32];
    sums(c0, left, v);
    if (MODE == kLinFwd || MODE == kLinFwdGated) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] += bias;
      if (a.z) {
        float lo[16], hi[16];
        lin_pairs(v, lo, hi);
        uint16_t* zp = a.z + (jr + c0) * a.ldz + (zcol & ~1);
#pragma unroll
        for (int p = 0; p < 16; ++p) {
          const int j = 2 * p + odd;
          if (live && j < left) *reinterpret_cast<uint32_t*>(zp + j * a.ldz) = lin_pack(lo[p], hi[p], a.f16);
        }
      }
    }
    float lo[kWords], hi[kWords];
    if constexpr (MODE == kLinFwdGated) {
      // gate and up meet: the gate lanes take column 2p, the up lanes column 2p + 1
      float h[16];
#pragma unroll
      for (int p = 0; p < 16; ++p) {
        const float got = __shfl_xor_sync(0xffffffffu, up ? v[2 * p] : v[2 * p + 1], 8);
        h[p] = up ? lin_silu(got) * v[2 * p + 1] : lin_silu(v[2 * p]) * got;
      }
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        const float got = __shfl_xor_sync(0xffffffffu, odd ? h[2 * p] : h[2 * p + 1], 1);
        lo[p] = odd ? got : h[2 * p];
        hi[p] = odd ? h[2 * p + 1] : got;
      }
    } else {
      if (MODE == kLinFwd) {
        switch (a.act) {
          case kActRelu:
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = v[j] < 0.f ? 0.f : v[j];   // keeps NaN
            break;
          case kActSilu:
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = lin_silu(v[j]);
            break;
          case kActGelu:
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = lin_gelu(v[j]);
            break;
          default:
            break;
        }
      }
      lin_pairs(v, lo, hi);
    }
    if (has_res) {
#pragma unroll
      for (int p = 0; p < kWords; ++p) {
        const float2 x = lin_unpack(res[p], a.f16);
        lo[p] += x.x;
        hi[p] += x.y;
      }
      if (c0 + 32 < ce) fetch(c0 + 32);
    }
    uint16_t* op = a.out + (jr + c0) * a.ldo + i2;
#pragma unroll
    for (int p = 0; p < kWords; ++p)
      if (live && row_of(p) < left) *reinterpret_cast<uint32_t*>(op + row_of(p) * a.ldo) = lin_pack(lo[p], hi[p], a.f16);
  }
}

// Loads A's 128 output columns (from column i0; gated: i0 of y) and q0 .. of the sum.
template <int MODE, bool PAIR>
__device__ __forceinline__ void lin_load_a(const LinArgs& a, const CUtensorMap* map, uint32_t dst, const LinTile& t, int i0,
                                           int q0, uint32_t bar) {
  if (MODE == kLinFwd) {
    tma_load_4d<PAIR>(dst, map, q0, i0, t.e, 0, bar);
  } else if (MODE == kLinFwdGated) {
    tma_load_5d<PAIR>(dst, map, q0, 0, 0, i0 >> 3, t.e, bar);
  } else {
    // rows of the sum: of w[e] (input gradient) or of x (weight gradient)
    const int row = MODE == kLinDx ? q0 : t.row0 + q0, plane = MODE == kLinDx ? t.e : 0;
    if (a.a_blocks) {
      tma_load_4d<PAIR>(dst, map, 0, row, i0 >> 6, plane, bar);
    } else {
      tma_load_4d<PAIR>(dst, map, i0, row, 0, plane, bar);
      tma_load_4d<PAIR>(dst + 8192, map, i0 + 64, row, 0, plane, bar);
    }
  }
}

// Loads rows j .. j + n of B (n a multiple of 8), q0 .. of the sum: lin_b_bytes in all.
template <int MODE, bool PAIR>
__device__ __forceinline__ void lin_load_b(const LinArgs& a, const CUtensorMap* map, uint32_t dst, const LinTile& t, int j,
                                           int n, int q0, uint32_t bar) {
  if (MODE == kLinDw) {
    if (a.b_blocks) {
      tma_load_4d<PAIR>(dst, map, 0, t.row0 + q0, j >> 6, 0, bar);
    } else {
      for (int b = 0; b * 64 < n; ++b) tma_load_4d<PAIR>(dst + b * 8192, map, j + b * 64, t.row0 + q0, 0, 0, bar);
    }
  } else {
    for (int b = 0; b < n; b += a.b_box) tma_load_4d<PAIR>(dst + b * 128, map, q0, t.row0 + j + b, 0, 0, bar);
  }
}
template <int MODE>
__device__ __forceinline__ uint32_t lin_b_bytes(const LinArgs& a, int n) {
  if (MODE == kLinDw) return static_cast<uint32_t>(a.b_blocks ? a.b_blocks : (n + 63) / 64) * 8192u;
  return static_cast<uint32_t>((n + a.b_box - 1) / a.b_box * a.b_box) * 128u;
}

// ------------------------------------------------------------------------------------------

// mapa / mapb: maps of the operands (see the launches); mapa4 / mapb4: one-row boxes of the same rows
// for the weight gradient's partial slabs.
template <int MODE>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap mapa, const __grid_constant__ CUtensorMap mapb,
                       const __grid_constant__ CUtensorMap mapa4, const __grid_constant__ CUtensorMap mapb4,
                       const LinArgs a) {
  constexpr bool kAMn = MODE == kLinDx || MODE == kLinDw, kBMn = MODE == kLinDw;
  constexpr int kCtaI = MODE == kLinFwdGated ? 64 : kLinBI;     // output columns per CTA
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kPairStages * kPairStage);   // even CTA: both CTAs' tiles landed
  uint64_t* empty = full + kPairStages;        // each CTA: the pair's MMAs have read the stage
  uint64_t* acc_full = empty + kPairStages;    // [2] each CTA: accumulator written
  uint64_t* acc_empty = acc_full + 2;          // [2] even CTA: drained by both CTAs
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* seg = reinterpret_cast<int*>(smem + kPairStages * kPairStage + 256);   // [E + 1] first row of each expert
  int* pfx = seg + kLinMaxE + 1;                                              // [E + 1] tiles before each expert

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = static_cast<int>(cluster_ctarank());
  const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      mbar_init(smem_u32(full + s), 1);
      mbar_init(smem_u32(empty + s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(acc_full + b), 1);
      mbar_init(smem_u32(acc_empty + b), 2 * 4);
    }
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&mapa);
    prefetch_tmap(&mapb);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 2 * kLinBJ);
    tmem_relinquish_pair();
  }
  if (warp == 2) {
    // segment starts and tile counts; a segment that would leave the buffers is an error and is cut
    int srun = 0, prun = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      int c = 0;
      if (e < a.E) c = a.counts ? __ldg(a.counts + e) : a.rows;
      if (c < 0 || c > a.rows) {
        record_error(a.status, kDevErrIndex);
        c = c < 0 ? 0 : a.rows;
      }
      const int padded = a.counts ? (c + a.align - 1) / a.align * a.align : c;
      int s = padded;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s = min(s + o, 0x3fffffff);
      }
      const int start = min(srun + s - padded, 0x3fffffff);
      srun = min(srun + __shfl_sync(0xffffffffu, s, 31), 0x3fffffff);
      if (e < a.E && c > 0 && start + c > a.rows) {
        record_error(a.status, kDevErrIndex);
        c = max(a.rows - start, 0);
      }
      const int nj = MODE == kLinDw ? a.j_ext : c, bj = lin_tile_rows(nj, kPairStep);
      const int n = e < a.E ? a.n_it * ((nj + bj - 1) / bj) : 0;
      int p = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, p, d);
        if (lane >= d) p += o;
      }
      if (e < a.E) {
        seg[e] = start;
        pfx[e] = prun + p - n;
      }
      prun += __shfl_sync(0xffffffffu, p, 31);
    }
    if (lane == 0) pfx[a.E] = prun;
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();      // both CTAs' barriers exist before any cross-CTA arrival
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int n_tiles = pfx[a.E];

  if (warp == 0) {
    // ---------------- loads: this CTA's 128 columns of A, its half of B's rows ----------------
    const uint32_t full0 = mapa_shared(smem_u32(full), 0);
    int st = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int ti = pair; ok && ti < n_tiles; ti += pairs) {
      const LinTile t = lin_tile<MODE>(a, seg, pfx, ti);
      const int half = ((t.ncols + kPairStep - 1) & ~(kPairStep - 1)) / 2;
      const int i0 = (t.it * 2 + rank) * kCtaI, j0 = t.j0 + rank * half;
      const uint32_t bytes = kLinABytes + lin_b_bytes<MODE>(a, half);
      for (int s = 0; s < t.slabs; ++s) {
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(empty + st), ph ^ 1, a.status) && *abort_flag == 0);
        if (!ok) break;
        const uint32_t sa = smem_u32(smem + st * kPairStage), sb = sa + kLinABytes, fb = full0 + st * 8;
        const int q0 = s * kLinSlab;
        const bool partial = MODE == kLinDw && a.counts && t.cnt - q0 < kLinSlab;
        if (rank == 0 && lane == 0)
          mbar_arrive_expect_tx(smem_u32(full + st), 2 * (partial ? kPairStage : bytes));
        __syncwarp();
        if (partial) {
          // rows past the segment's end become row `rows`, which reads as zeros
          for (int u = lane; u < 4 * 16; u += 32) {
            const int b = u >> 4, r4 = (u & 15) * 4;
            int y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = q0 + r4 + k < t.cnt ? t.row0 + q0 + r4 + k : a.rows;
            const uint32_t dst = sa + b * 8192 + r4 * 128;
            // a block of columns past the matrix: any columns do, it is never stored
            const int col = b < 2 ? i0 + b * 64 : j0 + (b - 2) * 64;
            if (b < 2)
              tma_rows4_pair(dst, &mapa4, col < a.i_ext ? col : 0, y[0], y[1], y[2], y[3], fb);
            else
              tma_rows4_pair(dst, &mapb4, col < a.j_ext ? col : 0, y[0], y[1], y[2], y[3], fb);
          }
        } else if (lane == 0) {
          lin_load_a<MODE, true>(a, &mapa, sa, t, i0, q0, fb);
          lin_load_b<MODE, true>(a, &mapb, sb, t, j0, half, q0, fb);
        }
        __syncwarp();
        if (++st == kPairStages) {
          st = 0;
          ph ^= 1;
        }
      }
    }
    if (!ok) {
      *abort_flag = 1;
      // let every copy issued into the pair's shared memory land before the CTAs exit
      if (rank == 0)
        for (int s = 0; s < kPairStages; ++s) mbar_wait(smem_u32(full + s), s < st ? ph : (ph ^ 1), nullptr);
    } else {
      // every slot released: the pair MMA's commits into this CTA's barriers have all landed
      for (int s = 0; s < kPairStages; ++s) {
        mbar_wait(smem_u32(empty + st), ph ^ 1, a.status);
        if (++st == kPairStages) {
          st = 0;
          ph ^= 1;
        }
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issue: one thread of the even CTA ----------------
    if (rank == 0 && lane == 0) {
      int st = 0, b = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      const uint64_t da0 = lin_desc<kAMn>(smem_u32(smem)), db0 = lin_desc<kBMn>(smem_u32(smem) + kLinABytes);
      for (int ti = pair; ok && ti < n_tiles; ti += pairs) {
        const LinTile t = lin_tile<MODE>(a, seg, pfx, ti);
        if (t.slabs == 0) continue;
        const uint32_t id = lin_idesc(a.f16, kAMn, kBMn, 2 * kLinBI,
                                      static_cast<uint32_t>((t.ncols + kPairStep - 1) & ~(kPairStep - 1)));
        ok = mbar_wait(smem_u32(acc_empty + b), ((aph >> b) & 1u) ^ 1u, a.status) && *abort_flag == 0;
        if (!ok) break;
        tc_fence_after();
        for (int s = 0; s < t.slabs; ++s) {
          ok = mbar_wait(smem_u32(full + st), ph, a.status);
          if (!ok) break;
          tc_fence_after();
          // descriptor addresses count 16-byte units
          const uint64_t da = da0 + static_cast<uint64_t>(st * (kPairStage >> 4));
          const uint64_t db = db0 + static_cast<uint64_t>(st * (kPairStage >> 4));
#pragma unroll
          for (int k = 0; k < kLinSlab / 16; ++k)
            mma_bf16_pair(tmem + static_cast<uint32_t>(b * kLinBJ), da + static_cast<uint64_t>(k * (kLinStep<kAMn> >> 4)),
                          db + static_cast<uint64_t>(k * (kLinStep<kBMn> >> 4)), id, (s > 0 || k > 0) ? 1u : 0u);
          tc_commit_pair(smem_u32(empty + st), 0x3);
          if (++st == kPairStages) {
            st = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
        tc_commit_pair(smem_u32(acc_full + b), 0x3);
        aph ^= 1u << b;
        b ^= 1;
      }
      if (!ok) *abort_flag = 1;
    }
    __syncwarp();
  } else {
    // ---------------- epilogue: this CTA's 128 output columns ----------------
    const int q = warp & 3;      // the TMEM lane quarter this warp may read
    const uint32_t acc_empty0 = mapa_shared(smem_u32(acc_empty), 0);
    int b = 0;
    uint32_t aph = 0;
    bool ok = true;
    for (int ti = pair; ok && ti < n_tiles; ti += pairs) {
      const LinTile t = lin_tile<MODE>(a, seg, pfx, ti);
      const int i0 = (t.it * 2 + rank) * kCtaI;
      if (t.slabs == 0) {
        lin_drain<MODE>(a, t, i0, 0, t.ncols, ZeroSums{}, q, lane);
        continue;
      }
      ok = mbar_wait(smem_u32(acc_full + b), (aph >> b) & 1u, a.status) && *abort_flag == 0;
      ok = named_barrier_and(1, 128, ok);
      if (!ok) break;
      tc_fence_after();
      lin_drain<MODE>(a, t, i0, 0, t.ncols,
                      TmemSums{tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(b * kLinBJ)}, q, lane);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(acc_empty0 + b * 8);
      aph ^= 1u << b;
      b ^= 1;
    }
    if (!ok) *abort_flag = 1;
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();      // no CTA leaves while the pair's MMAs or the other CTA's arrivals may touch it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 2 * kLinBJ);
  }
}

// ------------------------------------------------------------------------------------------

// Dense problems with few tiles: cluster c computes tile c, its CTA r the r-th slice of the sum.
template <int MODE>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_split_kernel(const __grid_constant__ CUtensorMap mapa, const __grid_constant__ CUtensorMap mapb, const LinArgs a) {
  constexpr bool kAMn = MODE == kLinDx || MODE == kLinDw, kBMn = MODE == kLinDw;
  constexpr int kCtaI = MODE == kLinFwdGated ? 64 : kLinBI;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kSplitRing);
  uint64_t* empty = full + kSplitMaxStages;
  uint64_t* acc_full = empty + kSplitMaxStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int S = a.split, slice = static_cast<int>(blockIdx.x) % S, tile = static_cast<int>(blockIdx.x) / S;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(smem_u32(full + s), 1);
      mbar_init(smem_u32(empty + s), 1);
    }
    mbar_init(smem_u32(acc_full), 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&mapa);
    prefetch_tmap(&mapb);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kLinBJ);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  LinTile t;
  t.e = 0;
  t.row0 = 0;
  t.cnt = a.rows;
  t.it = tile % a.n_it;
  t.j0 = tile / a.n_it * a.bj;
  t.ncols = min(a.bj, (MODE == kLinDw ? a.j_ext : a.rows) - t.j0);
  t.slabs = ((MODE == kLinDw ? a.rows : a.q_ext) + kLinSlab - 1) / kLinSlab;
  const int i0 = t.it * kCtaI;
  const int s0 = static_cast<int>(static_cast<long long>(t.slabs) * slice / S);          // this CTA's slabs [s0, s1),
  const int s1 = static_cast<int>(static_cast<long long>(t.slabs) * (slice + 1) / S);    // never empty (host)
  const uint32_t b_bytes = lin_b_bytes<MODE>(a, a.bj);
  const int stage = kLinABytes + static_cast<int>((b_bytes + 1023) & ~1023u);

  if (warp == 0) {
    int st = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int s = s0; s < s1; ++s) {
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(empty + st), ph ^ 1, a.status) && *abort_flag == 0);
      if (!ok) break;
      if (lane == 0) {
        const uint32_t sa = smem_u32(smem + st * stage), fb = smem_u32(full + st);
        mbar_arrive_expect_tx(fb, kLinABytes + b_bytes);
        lin_load_a<MODE, false>(a, &mapa, sa, t, i0, s * kLinSlab, fb);
        lin_load_b<MODE, false>(a, &mapb, sa + kLinABytes, t, t.j0, a.bj, s * kLinSlab, fb);
      }
      __syncwarp();
      if (++st == a.stages) {
        st = 0;
        ph ^= 1;
      }
    }
    if (!ok) {
      *abort_flag = 1;
      // let every copy issued into shared memory land before the CTA goes on
      for (int s = 0; s < a.stages; ++s) mbar_wait(smem_u32(full + s), s < st ? ph : (ph ^ 1), nullptr);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t id = lin_idesc(a.f16, kAMn, kBMn, kLinBI, static_cast<uint32_t>((t.ncols + kSplitStep - 1) & ~(kSplitStep - 1)));
      int st = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int s = s0; s < s1; ++s) {
        ok = mbar_wait(smem_u32(full + st), ph, a.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sa = smem_u32(smem + st * stage), sb = sa + kLinABytes;
#pragma unroll
        for (int k = 0; k < kLinSlab / 16; ++k)
          mma_bf16(tmem, lin_desc<kAMn>(sa + k * kLinStep<kAMn>), lin_desc<kBMn>(sb + k * kLinStep<kBMn>), id,
                   (s > s0 || k > 0) ? 1u : 0u);
        tc_commit(smem_u32(empty + st));
        if (++st == a.stages) {
          st = 0;
          ph ^= 1;
        }
      }
      if (ok)
        tc_commit(smem_u32(acc_full));
      else
        *abort_flag = 1;
    }
    __syncwarp();
  } else {
    const int q = warp & 3;
    bool ok = mbar_wait(smem_u32(acc_full), 0, a.status) && *abort_flag == 0;
    ok = named_barrier_and(1, 128, ok);
    tc_fence_after();
    if (!ok) {
      *abort_flag = 1;
    } else {
      const TmemSums mine{tmem + (static_cast<uint32_t>(q * 32) << 16)};
      if (S == 1) {
        lin_drain<MODE>(a, t, i0, 0, t.ncols, mine, q, lane);
      } else {
        // every MMA has read the ring: it takes this slice's sums, [column][128 lanes]
        float* part = reinterpret_cast<float*>(smem) + q * 32 + lane;
#pragma unroll 1
        for (int c0 = 0; c0 < t.ncols; c0 += 32) {
          float v[32];
          mine(c0, 32, v);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c0 + j < t.ncols) part[(c0 + j) * kLinBI] = v[j];
        }
      }
    }
  }
  __syncthreads();
  if (S > 1) {
    const bool ok = *abort_flag == 0;
    cluster_sync();
    if (warp >= 2 && ok) {
      const int q = warp & 3;
      const int w = (t.ncols + S - 1) / S, cb = min(slice * w, t.ncols), ce = min(cb + w, t.ncols);
      lin_drain<MODE>(a, t, i0, cb, ce,
                      ClusterSums{smem_u32(reinterpret_cast<float*>(smem) + q * 32 + lane), S}, q, lane);
    }
    cluster_sync();    // the slices stay until every CTA has read them
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kLinBJ);
  }
}

// ------------------------------------------------------------------------------------------

typedef CUresult (*EncodeTiledFnLin)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                     const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                     CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFnLin get_encode_lin() {
  static EncodeTiledFnLin fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &qr) == cudaSuccess &&
        qr == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFnLin>(p);
  }
  return fn;
}

// A map of 16-bit elements: extents d[0..n), strides (elements) s[1..n) of dimensions 1 .., box b[0..n).
bool lin_map(CUtensorMap* m, int f16, const void* p, int n, const long long* d, const long long* s, const int* b) {
  EncodeTiledFnLin enc = get_encode_lin();
  if (!enc) return false;
  cuuint64_t dims[5], strides[4];
  cuuint32_t box[5], es[5];
  for (int i = 0; i < n; ++i) {
    dims[i] = static_cast<cuuint64_t>(d[i]);
    box[i] = static_cast<cuuint32_t>(b[i]);
    es[i] = 1;
    if (i) strides[i - 1] = static_cast<cuuint64_t>(s[i]) * 2;
  }
  return enc(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(n),
             const_cast<void*>(p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [planes][rows][cols], contiguous along the sum: a copy takes box_rows rows of 64 columns.
bool map_k_major(CUtensorMap* m, int f16, const void* p, long long cols, long long rows, long long planes, long long ld,
                 int box_rows) {
  const long long d[4] = {cols, rows, planes, 1}, s[4] = {0, ld, ld * rows, ld * rows};
  const int b[4] = {kLinSlab, box_rows, 1, 1};
  return lin_map(m, f16, p, 4, d, s, b);
}

// [planes][rows][cols], summed over rows: a copy takes 64 rows of *blocks blocks of 64 columns, or
// (*blocks set to 0) of 64 columns from any column on where the matrix does not come in whole blocks.
bool map_mn_major(CUtensorMap* m, int f16, const void* p, long long cols, long long rows, long long planes, long long ld,
                  int* blocks) {
  if (cols % 64) *blocks = 0;
  if (*blocks) {
    const long long d[4] = {64, rows, cols / 64, planes}, s[4] = {0, ld, 64, ld * rows};
    const int b[4] = {64, kLinSlab, *blocks, 1};
    return lin_map(m, f16, p, 4, d, s, b);
  }
  const long long d[4] = {cols, rows, 1, planes}, s[4] = {0, ld, ld * rows, ld * rows};
  const int b[4] = {64, kLinSlab, 1, 1};
  return lin_map(m, f16, p, 4, d, s, b);
}

bool map_one_row(CUtensorMap* m, int f16, const void* p, long long cols, long long rows, long long ld) {
  const long long d[2] = {cols, rows}, s[2] = {0, ld};
  const int b[2] = {64, 1};
  return lin_map(m, f16, p, 2, d, s, b);
}

// How a problem runs.  j: rows of the output (dense) or of the row buffers (experts).
struct LinPlan {
  bool pair;
  int split, bj, stages, grid, b_box;
};

LinPlan lin_plan(bool dense, int i_cols, int cta_i, long long j, long long q, bool b_mn) {
  LinPlan p{};
  const int sms = num_sms(), pairs = sms / 2;
  const long long slabs = (q + kLinSlab - 1) / kLinSlab;
  p.bj = lin_tile_rows(static_cast<int>(j), kPairStep);
  const long long nj = (j + p.bj - 1) / p.bj;
  const long long tiles = (i_cols + 2 * cta_i - 1) / (2 * cta_i) * nj;
  p.pair = !dense || tiles * 2 > pairs;
  if (p.pair) {
    p.grid = 2 * static_cast<int>(dense && tiles < pairs ? tiles : pairs);
    p.split = 1;
    p.b_box = dense ? p.bj / 2 : 32;
    return p;
  }
  p.bj = lin_tile_rows(static_cast<int>(j), kSplitStep);
  const long long t1 = (i_cols + cta_i - 1) / cta_i * ((j + p.bj - 1) / p.bj);
  p.split = 1;
  while (p.split < 8 && t1 * p.split * 2 <= sms && slabs >= 4 * p.split) p.split *= 2;
  p.grid = static_cast<int>(t1) * p.split;
  p.b_box = p.bj;
  const int b_bytes = b_mn ? (p.bj + 63) / 64 * 8192 : p.bj * 128;
  const int stage = kLinABytes + (b_bytes + 1023) / 1024 * 1024;
  p.stages = kSplitRing / stage < kSplitMaxStages ? kSplitRing / stage : kSplitMaxStages;
  return p;
}

template <int MODE>
cudaError_t lin_launch(const LinPlan& p, const CUtensorMap (&m)[4], LinArgs a, cudaStream_t stream) {
  a.split = p.split;
  a.bj = p.bj;
  a.stages = p.stages;
  a.b_box = p.b_box;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = static_cast<unsigned>(p.pair ? 2 : p.split);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(p.grid);
  cfg.blockDim = dim3(kLinThreads);
  cfg.dynamicSmemBytes = p.pair ? kPairSmem : kSplitSmem;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (p.pair) {
    const cudaError_t err =
        cudaFuncSetAttribute(linear_pair_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem);
    if (err != cudaSuccess) return err;
    return cudaLaunchKernelEx(&cfg, linear_pair_kernel<MODE>, m[0], m[1], m[2], m[3], static_cast<const LinArgs>(a));
  }
  const cudaError_t err =
      cudaFuncSetAttribute(linear_split_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSplitSmem);
  if (err != cudaSuccess) return err;
  return cudaLaunchKernelEx(&cfg, linear_split_kernel<MODE>, m[0], m[1], static_cast<const LinArgs>(a));
}

LinArgs lin_args(const LinearShape& p, uint32_t* status) {
  LinArgs a{};
  a.counts = p.counts;
  a.E = p.counts ? p.E : 1;
  a.align = p.align;
  a.rows = p.rows;
  a.f16 = p.f16;
  a.act = kActNone;
  a.status = status;
  return a;
}

}  // namespace

cudaError_t launch_linear(const LinearShape& p, RowsView x, const uint16_t* w, const float* bias, RowsView res, int act,
                          RowsView y, RowsView z, uint32_t* status, cudaStream_t stream) {
  LinArgs a = lin_args(p, status);
  const bool gated = act == kActSwiglu;
  a.act = act;
  a.i_ext = gated ? p.N / 2 : p.N;
  a.q_ext = p.K;
  a.out = static_cast<uint16_t*>(y.ptr);
  a.ldo = y.ld;
  a.z = static_cast<uint16_t*>(z.ptr);
  a.ldz = z.ld;
  a.res = static_cast<const uint16_t*>(res.ptr);
  a.ldr = res.ld;
  a.bias = bias;
  const int cta_i = gated ? 64 : kLinBI;
  const LinPlan pl = lin_plan(!p.counts, a.i_ext, cta_i, p.rows, p.K, false);
  const int tile_i = pl.pair ? 2 * cta_i : cta_i;
  a.n_it = (a.i_ext + tile_i - 1) / tile_i;
  CUtensorMap m[4] = {};
  bool ok;
  if (gated) {
    // [E][N/2 / 8][2][8][K]: a copy takes, eight columns at a time, their gate rows and then their up rows
    const long long I = p.N / 2, K = p.K;
    const long long d[5] = {K, 8, 2, I / 8, a.E}, s[5] = {0, K, I * K, 8 * K, 2 * I * K};
    const int b[5] = {kLinSlab, 8, 2, 8, 1};
    ok = lin_map(&m[0], p.f16, w, 5, d, s, b);
  } else {
    ok = map_k_major(&m[0], p.f16, w, p.K, p.N, a.E, p.K, kLinBI);
  }
  if (!ok || !map_k_major(&m[1], p.f16, x.ptr, p.K, p.rows, 1, x.ld, pl.b_box)) return cudaErrorInvalidValue;
  return gated ? lin_launch<kLinFwdGated>(pl, m, a, stream) : lin_launch<kLinFwd>(pl, m, a, stream);
}

cudaError_t launch_linear_dx(const LinearShape& p, RowsView dz, const uint16_t* w, RowsView res, RowsView dx,
                             uint32_t* status, cudaStream_t stream) {
  LinArgs a = lin_args(p, status);
  a.i_ext = p.K;
  a.q_ext = p.N;
  a.out = static_cast<uint16_t*>(dx.ptr);
  a.ldo = dx.ld;
  a.res = static_cast<const uint16_t*>(res.ptr);
  a.ldr = res.ld;
  const LinPlan pl = lin_plan(!p.counts, p.K, kLinBI, p.rows, p.N, false);
  const int tile_i = pl.pair ? 2 * kLinBI : kLinBI;
  a.n_it = (p.K + tile_i - 1) / tile_i;
  CUtensorMap m[4] = {};
  a.a_blocks = 2;
  if (!map_mn_major(&m[0], p.f16, w, p.K, p.N, a.E, p.K, &a.a_blocks) ||
      !map_k_major(&m[1], p.f16, dz.ptr, p.N, p.rows, 1, dz.ld, pl.b_box))
    return cudaErrorInvalidValue;
  return lin_launch<kLinDx>(pl, m, a, stream);
}

cudaError_t launch_linear_dw(const LinearShape& p, RowsView dz, RowsView x, uint16_t* dw, uint32_t* status,
                             cudaStream_t stream) {
  LinArgs a = lin_args(p, status);
  a.i_ext = p.K;
  a.j_ext = p.N;
  a.out = dw;
  a.ldo = p.K;
  const LinPlan pl = lin_plan(!p.counts, p.K, kLinBI, p.N, p.rows, true);
  const int tile_i = pl.pair ? 2 * kLinBI : kLinBI;
  a.n_it = (p.K + tile_i - 1) / tile_i;
  CUtensorMap m[4] = {};
  a.a_blocks = 2;
  // B in one copy where every tile (over a pair: every half) starts on a block
  const int cta_j = pl.pair ? pl.bj / 2 : pl.bj;
  a.b_blocks = cta_j % 64 == 0 && (!pl.pair || p.N % pl.bj == 0) ? cta_j / 64 : 0;
  if (!map_mn_major(&m[0], p.f16, x.ptr, p.K, p.rows, 1, x.ld, &a.a_blocks) ||
      !map_mn_major(&m[1], p.f16, dz.ptr, p.N, p.rows, 1, dz.ld, &a.b_blocks) ||
      !map_one_row(&m[2], p.f16, x.ptr, p.K, p.rows, x.ld) || !map_one_row(&m[3], p.f16, dz.ptr, p.N, p.rows, dz.ld))
    return cudaErrorInvalidValue;
  return lin_launch<kLinDw>(pl, m, a, stream);
}

// ------------------------------------------------------------------------------------------
// dz = dy * act'(z) and the bias gradient's partial sums: thread = 8 columns, walking the rows
// s, s + S, ... of its expert (dense: all rows); CTA = 32 column groups x 8 rows.

namespace {

constexpr int kActRowLanes = 8;

__device__ __forceinline__ float silu_grad(float z, float& silu) {
  const float s = __fdividef(1.f, 1.f + __expf(-z));
  silu = z * s;
  return s * (1.f + z * (1.f - s));
}

template <class T>
__global__ void __launch_bounds__(32 * kActRowLanes)
    act_grad_kernel(const uint16_t* __restrict__ dy, long long lddy, const uint16_t* __restrict__ z, long long ldz, int act,
                    const int32_t* __restrict__ counts, int E, int align, int rows, int N, uint16_t* __restrict__ dz,
                    long long lddz, float* __restrict__ part, int S, uint32_t* status) {
  __shared__ unsigned long long s_seg;
  __shared__ float red[kActRowLanes][2][32 * 8 + 8];
  const int lane = threadIdx.x & 31, rl = threadIdx.x >> 5;
  const int e = blockIdx.y;
  int cnt = rows, seg = 0;
  if (counts) {
    if (threadIdx.x == 0) s_seg = 0;
    __syncthreads();
    int mine = 0;
    for (int i = threadIdx.x; i < e; i += blockDim.x) {
      const int c = min(max(__ldg(counts + i), 0), rows);
      mine = min(mine + (c + align - 1) / align * align, rows);
    }
    if (mine) atomicAdd(&s_seg, static_cast<unsigned long long>(mine));   // integers: the order does not matter
    __syncthreads();
    seg = s_seg < static_cast<unsigned long long>(rows) ? static_cast<int>(s_seg) : rows;
    cnt = min(max(__ldg(counts + e), 0), rows - seg);
  }
  const bool gated = act == kActSwiglu;
  const int cols = gated ? N / 2 : N;
  const int c = (blockIdx.x * 32 + lane) * 8;
  float acc[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[0][i] = acc[1][i] = 0.f;
  if (c < cols) {
    for (int r = blockIdx.z * kActRowLanes + rl; r < cnt; r += S * kActRowLanes) {
      const long long row = seg + r;
      const Pack<T, 8> g = load_pack<T, 8>(dy + row * lddy + c);
      Pack<T, 8> o, o2;
      if (gated) {
        const Pack<T, 8> a = load_pack<T, 8>(z + row * ldz + c), b = load_pack<T, 8>(z + row * ldz + cols + c);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float s;
          const float d = silu_grad(a.f(i), s);
          const float dg = g.f(i) * b.f(i) * d, du = g.f(i) * s;
          acc[0][i] += dg;
          acc[1][i] += du;
          o.set(i, dg);
          o2.set(i, du);
        }
        store_pack<T, 8>(dz + row * lddz + c, o);
        store_pack<T, 8>(dz + row * lddz + cols + c, o2);
      } else if (act == kActNone) {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[0][i] += g.f(i);
      } else {
        const Pack<T, 8> a = load_pack<T, 8>(z + row * ldz + c);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = a.f(i);
          float d;
          if (act == kActRelu) {
            d = v > 0.f ? g.f(i) : 0.f;
          } else if (act == kActSilu) {
            float s;
            d = g.f(i) * silu_grad(v, s);
          } else {
            d = g.f(i) * (0.5f * erfcf(v * -0.70710678118654752f) + v * 0.39894228040143268f * __expf(-0.5f * v * v));
          }
          acc[0][i] += d;
          o.set(i, d);
        }
        store_pack<T, 8>(dz + row * lddz + c, o);
      }
    }
  }
  if (!part) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    red[rl][0][lane * 8 + i] = acc[0][i];
    red[rl][1][lane * 8 + i] = acc[1][i];
  }
  __syncthreads();
  for (int h = 0; h < (gated ? 2 : 1); ++h) {
    const int col = blockIdx.x * 256 + threadIdx.x;
    if (col < cols) {
      float s = 0.f;
#pragma unroll
      for (int r = 0; r < kActRowLanes; ++r) s += red[r][h][threadIdx.x];
      part[(static_cast<size_t>(e) * S + blockIdx.z) * N + h * cols + col] = s;
    }
  }
}

__global__ void __launch_bounds__(256) bias_sum_kernel(const float* __restrict__ part, int S, int N, long long total,
                                                       float* __restrict__ db) {
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= total) return;
  const long long e = i / N, c = i - e * N;
  float s = 0.f;
  for (int k = 0; k < S; ++k) s += part[(e * S + k) * N + c];
  db[i] = s;
}

}  // namespace

// Row slices per expert: about eight CTAs per SM in all, at most 64.
int linear_bias_slices(int N, int E, int act) {
  const int cols = act == kActSwiglu ? N / 2 : N;
  const long long cta = static_cast<long long>((cols + 255) / 256) * (E > 0 ? E : 1);
  const long long s = (8LL * 152 + cta - 1) / cta;
  return static_cast<int>(s < 1 ? 1 : (s > 64 ? 64 : s));
}

cudaError_t launch_act_grad(const LinearShape& p, RowsView dy, RowsView z, int act, RowsView dz, float* part, float* db,
                            uint32_t* status, cudaStream_t stream) {
  const int E = p.counts ? p.E : 1, S = linear_bias_slices(p.N, E, act);
  const int cols = act == kActSwiglu ? p.N / 2 : p.N;
  const dim3 grid((cols + 255) / 256, E, S);
  float* pp = db ? part : nullptr;
  if (p.f16)
    act_grad_kernel<F16Elem><<<grid, 256, 0, stream>>>(static_cast<const uint16_t*>(dy.ptr), dy.ld,
                                                       static_cast<const uint16_t*>(z.ptr), z.ld, act, p.counts, E, p.align,
                                                       p.rows, p.N, static_cast<uint16_t*>(dz.ptr), dz.ld, pp, S, status);
  else
    act_grad_kernel<Bf16Elem><<<grid, 256, 0, stream>>>(static_cast<const uint16_t*>(dy.ptr), dy.ld,
                                                        static_cast<const uint16_t*>(z.ptr), z.ld, act, p.counts, E, p.align,
                                                        p.rows, p.N, static_cast<uint16_t*>(dz.ptr), dz.ld, pp, S, status);
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess || !db) return err;
  const long long total = static_cast<long long>(E) * p.N;
  bias_sum_kernel<<<static_cast<int>((total + 255) / 256), 256, 0, stream>>>(part, S, p.N, total, db);
  return cudaGetLastError();
}

}  // namespace moe
