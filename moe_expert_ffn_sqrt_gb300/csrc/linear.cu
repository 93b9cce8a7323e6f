// Matrix products with a fused epilogue, dense or with one weight per expert, and their gradients
// (bf16 or fp16 operands, fp32 accumulation), on tcgen05 (sm_103a).
//
//   forward   y[r, n]  = act( sum_k x[r, k] w[e, n, k] + bias[e, n] ) + residual[r, n]
//   input     dx[r, k] = sum_n dz[r, n] w[e, n, k] (+ residual[r, k])
//   weight    dw[e, n, k] = sum_r dz[r, n] x[r, k]        over expert e's rows
//
// All three are out[j, i] = sum_q A[i, q] B[j, q] with i the contiguous column of the output: i runs
// over the MMA's 128 M rows (accumulator lanes) and j over its N columns.  So the tokens are on N, where
// the MMA takes any multiple of 16: a ragged or short expert segment costs what it holds.  What
// changes is which operand is contiguous along the sum: w is (forward), w and x are not (gradients); the
// shared-memory descriptors take either order, so no operand is ever transposed in memory.
//
// Rows of experts: expert e's rows start at seg_e = sum_{e' < e} round_up(counts[e'], align) (the layout
// of moe_permute).  Padding rows are never read into a result nor written: in the forward and the input
// gradient a padding row is a column of the product that is not stored; in the weight gradient, where
// rows are summed over, the last partial slab of a segment is fetched row by row with the padding
// rows replaced by out-of-range ones, which read as zeros.
//
// One persistent CTA per SM: warp 0 loads (TMA, 128-byte swizzle), warp 1 issues the MMAs, warps 2..5
// drain the accumulators.  Two accumulators let one tile's epilogue run under the next tile's MMAs.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kernels.h"
#include "rows.cuh"

namespace moe {

namespace {

constexpr int kLinThreads = 192;
constexpr int kLinBI = 128;                 // output columns i per tile (MMA M)
constexpr int kLinBJ = 256;                 // output rows j per tile (MMA N), at most
constexpr int kLinSlab = 64;                // terms of the sum per pipeline stage
constexpr int kLinABytes = kLinBI * 128;
constexpr int kLinBBytes = kLinBJ * 128;
constexpr int kLinStage = kLinABytes + kLinBBytes;   // 48 KB
constexpr int kLinStages = 4;
constexpr int kLinMaxE = kLinearMaxExperts;
constexpr int kLinBars = 2 * kLinStages + 4;
constexpr int kLinSmem = 1024 + kLinStages * kLinStage + kLinBars * 8 + 16 + 2 * (kLinMaxE + 1) * 4;
static_assert(kLinSmem <= 227 * 1024, "shared memory budget");

enum LinMode { kLinFwd = 0, kLinFwdGated = 1, kLinDx = 2, kLinDw = 3 };

struct LinArgs {
  const int32_t* counts;      // [E] rows per expert; nullptr: one dense segment of `rows` rows
  int E, align, rows;         // rows: rows of the row buffers
  int n_it;                   // i tiles
  int i_ext;                  // output columns (gated forward: of y; z has twice as many)
  int j_ext;                  // weight gradient: N
  int q_ext;                  // forward: K, input gradient: N
  int act, f16;
  uint16_t* out;
  long long ldo;
  uint16_t* z;
  long long ldz;
  const uint16_t* res;
  long long ldr;
  const float* bias;          // [E, N]
  uint32_t* status;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_rows4(uint32_t dst, const CUtensorMap* map, int c0, int y0, int y1, int y2, int y3,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(y0), "r"(y1), "r"(y2), "r"(y3), "r"(bar)
      : "memory");
}

// Instruction descriptor of kind::f16 (bf16 or fp16 operands, fp32 accumulation); a_mn / b_mn: the
// operand's tile is contiguous along M / N instead of along the sum.
__device__ __forceinline__ uint32_t lin_idesc(int f16, int a_mn, int b_mn, uint32_t N) {
  const uint32_t fmt = f16 ? 0u : 1u;
  return (1u << 4) | (fmt << 7) | (fmt << 10) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
         ((N >> 3) << 17) | ((kLinBI >> 4) << 24);
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

struct LinTile {
  int e, it, row0, cnt, j0, ncols, slabs;
};

// Tiles in order of expert, then i tile, then j tile (the j tiles of one weight tile run side by side).
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
  const int u = t - pfx[lo];
  const int n = MODE == kLinDw ? a.j_ext : r.cnt;
  const int nj = (n + kLinBJ - 1) / kLinBJ;
  r.it = u / nj;
  r.j0 = (u - r.it * nj) * kLinBJ;
  r.ncols = min(kLinBJ, n - r.j0);
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

// Drains one accumulator (this warp's 32 lanes at TMEM address acc) of tile t.  acc = 0xffffffff: an
// empty sum (zeros).
template <int MODE>
__device__ __forceinline__ void lin_drain(const LinArgs& a, const LinTile& t, uint32_t acc, bool empty, int q, int lane) {
  // output column of this lane.  Gated forward: a warp's lanes 0..15 are gate rows, lanes 16..31 the
  // up rows of the same 16 columns.
  const int up = MODE == kLinFwdGated ? lane >> 4 : 0;
  const int i = MODE == kLinFwdGated ? t.it * 64 + q * 16 + (lane & 15) : t.it * kLinBI + q * 32 + lane;
  const bool live = (i & ~1) < a.i_ext;    // i_ext is even
  const int i2 = i & ~1, odd = lane & 1;
  const int zcol = MODE == kLinFwdGated ? i + up * a.i_ext : i;
  const int n_all = MODE == kLinFwdGated ? 2 * a.i_ext : a.i_ext;
  float bias = 0.f;
  if ((MODE == kLinFwd || MODE == kLinFwdGated) && a.bias && live)
    bias = __ldg(a.bias + static_cast<size_t>(t.e) * n_all + zcol);
  // output row of accumulator column 0
  const long long jr = MODE == kLinDw ? static_cast<long long>(t.e) * a.j_ext + t.j0 : static_cast<long long>(t.row0) + t.j0;
#pragma unroll 1
  for (int c0 = 0; c0 < t.ncols; c0 += 32) {
    float v[32];
    if (empty) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = 0.f;
    } else {
      uint32_t r[2][16];
      tc_ld_x16(acc + c0, r[0]);
      tc_ld_x16(acc + c0 + 16, r[1]);
      tc_wait_ld();
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j >> 4][j & 15]) + bias;
    }
    const int left = t.ncols - c0;
    float lo[16], hi[16];
    if (MODE == kLinFwd || MODE == kLinFwdGated) {
      if (a.z) {
        lin_pairs(v, lo, hi);
        uint16_t* zp = a.z + (jr + c0) * a.ldz + (zcol & ~1);
#pragma unroll
        for (int p = 0; p < 16; ++p) {
          const int j = 2 * p + odd;
          if (live && j < left) *reinterpret_cast<uint32_t*>(zp + j * a.ldz) = lin_pack(lo[p], hi[p], a.f16);
        }
      }
    }
    if (MODE == kLinFwdGated) {
      // gate and up meet: lanes 0..15 take column 2p, lanes 16..31 column 2p + 1
      float h[16];
#pragma unroll
      for (int p = 0; p < 16; ++p) {
        const float got = __shfl_xor_sync(0xffffffffu, up ? v[2 * p] : v[2 * p + 1], 16);
        h[p] = up ? lin_silu(got) * v[2 * p + 1] : lin_silu(v[2 * p]) * got;
      }
      uint16_t* op = a.out + (jr + c0) * a.ldo + i2;
      const uint16_t* rp = a.res ? a.res + (jr + c0) * a.ldr + i2 : nullptr;
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        const float got = __shfl_xor_sync(0xffffffffu, odd ? h[2 * p] : h[2 * p + 1], 1);
        float l0 = odd ? got : h[2 * p], h0 = odd ? h[2 * p + 1] : got;
        const int j = 2 * (2 * p + odd) + up;
        if (live && j < left) {
          if (rp) {
            const float2 x = lin_unpack(*reinterpret_cast<const uint32_t*>(rp + j * a.ldr), a.f16);
            l0 += x.x;
            h0 += x.y;
          }
          *reinterpret_cast<uint32_t*>(op + j * a.ldo) = lin_pack(l0, h0, a.f16);
        }
      }
      continue;
    }
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
    uint16_t* op = a.out + (jr + c0) * a.ldo + i2;
    if (MODE != kLinDw && a.res) {
      const uint16_t* rp = a.res + (jr + c0) * a.ldr + i2;
#pragma unroll
      for (int p = 0; p < 16; ++p) {
        const int j = 2 * p + odd;
        if (live && j < left) {
          const float2 x = lin_unpack(*reinterpret_cast<const uint32_t*>(rp + j * a.ldr), a.f16);
          lo[p] += x.x;
          hi[p] += x.y;
        }
      }
    }
#pragma unroll
    for (int p = 0; p < 16; ++p) {
      const int j = 2 * p + odd;
      if (live && j < left) *reinterpret_cast<uint32_t*>(op + j * a.ldo) = lin_pack(lo[p], hi[p], a.f16);
    }
  }
}

// mapa / mapb: 3-D maps of the operands (see launch); mapa4 / mapb4: one-row boxes of the same rows for
// the weight gradient's partial slabs.
template <int MODE>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_kernel(const __grid_constant__ CUtensorMap mapa, const __grid_constant__ CUtensorMap mapb,
                  const __grid_constant__ CUtensorMap mapa4, const __grid_constant__ CUtensorMap mapb4, const LinArgs a) {
  constexpr bool kAMn = MODE == kLinDx || MODE == kLinDw, kBMn = MODE == kLinDw;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kLinStages * kLinStage);
  uint64_t* empty = full + kLinStages;
  uint64_t* acc_full = empty + kLinStages;     // [2]
  uint64_t* acc_empty = acc_full + 2;          // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* seg = reinterpret_cast<int*>(tmem_slot + 4);   // [E + 1] first row of each expert
  int* pfx = seg + kLinMaxE + 1;                      // [E + 1] tiles before each expert

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kLinStages; ++s) {
      mbar_init(smem_u32(full + s), 1);
      mbar_init(smem_u32(empty + s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(acc_full + b), 1);
      mbar_init(smem_u32(acc_empty + b), 128);
    }
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&mapa);
    prefetch_tmap(&mapb);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 2 * kLinBJ);
    tmem_relinquish();
  }
  if (warp == 2) {
    // segment starts and tile counts; a segment that would leave the buffers is an error and is cut
    int srun = 0, prun = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      int c = 0;
      if (e < a.E) c = a.counts ? __ldg(a.counts + e) : a.rows;
      if (c < 0) {
        record_error(a.status, kDevErrIndex);
        c = 0;
      }
      if (c > a.rows) {
        record_error(a.status, kDevErrIndex);
        c = a.rows;
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
      int n = e < a.E ? a.n_it * (((MODE == kLinDw ? a.j_ext : c) + kLinBJ - 1) / kLinBJ) : 0;
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
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int n_tiles = pfx[a.E];

  if (warp == 0) {
    // ---------------- loads ----------------
    int st = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int ti = blockIdx.x; ok && ti < n_tiles; ti += gridDim.x) {
      const LinTile t = lin_tile<MODE>(a, seg, pfx, ti);
      for (int s = 0; s < t.slabs; ++s) {
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(empty + st), ph ^ 1, a.status)) && *abort_flag == 0;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t sa = smem_u32(smem + st * kLinStage), sb = sa + kLinABytes, fb = smem_u32(full + st);
        const int q0 = s * kLinSlab;
        if (lane == 0) mbar_arrive_expect_tx(fb, kLinStage);
        __syncwarp();
        if (MODE == kLinDw && a.counts && t.cnt - q0 < kLinSlab) {
          // partial slab: rows past the segment's end become row `rows`, which reads as zeros
          for (int u = lane; u < (kLinBI + kLinBJ) / 64 * 16; u += 32) {
            const int b = u >> 4, r4 = (u & 15) * 4;
            int y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = q0 + r4 + k < t.cnt ? t.row0 + q0 + r4 + k : a.rows;
            const uint32_t dst = sa + b * 8192 + r4 * 128;
            // a block of columns past the matrix: any rows do, it is never stored
            const int col = b < 2 ? t.it * kLinBI + b * 64 : t.j0 + (b - 2) * 64;
            if (b < 2)
              tma_rows4(dst, &mapa4, col < a.i_ext ? col : 0, y[0], y[1], y[2], y[3], fb);
            else
              tma_rows4(dst, &mapb4, col < a.j_ext ? col : 0, y[0], y[1], y[2], y[3], fb);
          }
        } else if (lane == 0) {
          if (MODE == kLinFwd) {
            tma_load_3d(sa, &mapa, q0, t.it * kLinBI, t.e, fb);
          } else if (MODE == kLinFwdGated) {
#pragma unroll
            for (int g = 0; g < 4; ++g) tma_load_3d(sa + g * 4096, &mapa, q0, t.it * 64 + g * 16, 2 * t.e, fb);
          } else if (MODE == kLinDx) {
#pragma unroll
            for (int b = 0; b < 2; ++b) tma_load_3d(sa + b * 8192, &mapa, t.it * kLinBI + b * 64, q0, t.e, fb);
          } else {
#pragma unroll
            for (int b = 0; b < 2; ++b) tma_load_3d(sa + b * 8192, &mapa, t.it * kLinBI + b * 64, t.row0 + q0, 0, fb);
          }
          if (MODE == kLinDw) {
#pragma unroll
            for (int b = 0; b < kLinBJ / 64; ++b) tma_load_3d(sb + b * 8192, &mapb, t.j0 + b * 64, t.row0 + q0, 0, fb);
          } else {
            tma_load_3d(sb, &mapb, q0, t.row0 + t.j0, 0, fb);
          }
        }
        __syncwarp();
        if (++st == kLinStages) {
          st = 0;
          ph ^= 1;
        }
      }
    }
    if (!ok) {
      *abort_flag = 1;
      // let every copy issued into shared memory land before the CTA exits
      for (int s = 0; s < kLinStages; ++s) mbar_wait(smem_u32(full + s), s < st ? ph : (ph ^ 1), nullptr);
    }
  } else if (warp == 1) {
    // ---------------- MMA issue ----------------
    int st = 0, b = 0;
    uint32_t ph = 0, aph = 0;
    bool ok = true;
    for (int ti = blockIdx.x; ok && ti < n_tiles; ti += gridDim.x) {
      const LinTile t = lin_tile<MODE>(a, seg, pfx, ti);
      if (t.slabs == 0) continue;
      const uint32_t id = lin_idesc(a.f16, kAMn, kBMn, static_cast<uint32_t>((t.ncols + 15) & ~15));
      ok = mbar_wait(smem_u32(acc_empty + b), ((aph >> b) & 1u) ^ 1u, a.status);
      ok = __all_sync(0xffffffffu, ok && *abort_flag == 0);
      if (!ok) break;
      tc_fence_after();
      for (int s = 0; s < t.slabs; ++s) {
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(full + st), ph, a.status) && *abort_flag == 0);
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          const uint32_t sa = smem_u32(smem + st * kLinStage), sb = sa + kLinABytes;
#pragma unroll
          for (int k = 0; k < kLinSlab / 16; ++k)
            mma_bf16(tmem + static_cast<uint32_t>(b * kLinBJ), lin_desc<kAMn>(sa + k * kLinStep<kAMn>),
                     lin_desc<kBMn>(sb + k * kLinStep<kBMn>), id, (s > 0 || k > 0) ? 1u : 0u);
          tc_commit(smem_u32(empty + st));
          if (s == t.slabs - 1) tc_commit(smem_u32(acc_full + b));
        }
        __syncwarp();
        if (++st == kLinStages) {
          st = 0;
          ph ^= 1;
        }
      }
      aph ^= 1u << b;
      b ^= 1;
    }
    if (!ok) *abort_flag = 1;
  } else {
    // ---------------- epilogue ----------------
    const int q = warp & 3;      // the TMEM lane quarter this warp may read
    int b = 0;
    uint32_t aph = 0;
    bool ok = true;
    for (int ti = blockIdx.x; ok && ti < n_tiles; ti += gridDim.x) {
      const LinTile t = lin_tile<MODE>(a, seg, pfx, ti);
      if (t.slabs == 0) {
        lin_drain<MODE>(a, t, 0, true, q, lane);
        continue;
      }
      ok = mbar_wait(smem_u32(acc_full + b), (aph >> b) & 1u, a.status) && *abort_flag == 0;
      ok = named_barrier_and(1, 128, ok);
      if (!ok) break;
      tc_fence_after();
      lin_drain<MODE>(a, t, tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(b * kLinBJ), false, q, lane);
      tc_fence_before();
      mbar_arrive(smem_u32(acc_empty + b));
      aph ^= 1u << b;
      b ^= 1;
    }
    if (!ok) *abort_flag = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * kLinBJ);
  }
}

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

// [planes][rows][cols] of 16-bit elements, box bp x br x 64.
bool lin_map(CUtensorMap* m, int f16, const void* p, long long cols, long long rows, long long planes, long long ld,
             long long plane, int br, int bp, int dims = 3) {
  EncodeTiledFnLin enc = get_encode_lin();
  if (!enc) return false;
  cuuint64_t d[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(planes)};
  cuuint64_t s[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(plane) * 2};
  cuuint32_t box[3] = {kLinSlab, static_cast<cuuint32_t>(br), static_cast<cuuint32_t>(bp)};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(dims),
             const_cast<void*>(p), d, s, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE>
cudaError_t lin_launch(const CUtensorMap (&m)[4], const LinArgs& a, cudaStream_t stream) {
  cudaError_t err = cudaFuncSetAttribute(linear_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kLinSmem);
  if (err != cudaSuccess) return err;
  // dense: the tile count is known here; experts: at most one CTA per SM, the kernel counts the tiles
  long long tiles = num_sms();
  if (!a.counts) tiles = static_cast<long long>(a.n_it) * (((MODE == kLinDw ? a.j_ext : a.rows) + kLinBJ - 1) / kLinBJ);
  const int grid = static_cast<int>(tiles < num_sms() ? tiles : num_sms());
  if (grid == 0) return cudaSuccess;
  linear_kernel<MODE><<<grid, kLinThreads, kLinSmem, stream>>>(m[0], m[1], m[2], m[3], a);
  return cudaGetLastError();
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
  a.n_it = gated ? (p.N / 2 + 63) / 64 : (p.N + kLinBI - 1) / kLinBI;
  a.q_ext = p.K;
  a.out = static_cast<uint16_t*>(y.ptr);
  a.ldo = y.ld;
  a.z = static_cast<uint16_t*>(z.ptr);
  a.ldz = z.ld;
  a.res = static_cast<const uint16_t*>(res.ptr);
  a.ldr = res.ld;
  a.bias = bias;
  CUtensorMap m[4] = {};
  // gated: [2E][N/2][K], a box takes 16 gate rows and the 16 up rows of the same columns
  const bool ok =
      gated ? lin_map(&m[0], p.f16, w, p.K, p.N / 2, 2LL * a.E, p.K, static_cast<long long>(p.N / 2) * p.K, 16, 2)
            : lin_map(&m[0], p.f16, w, p.K, p.N, a.E, p.K, static_cast<long long>(p.N) * p.K, kLinBI, 1);
  if (!ok || !lin_map(&m[1], p.f16, x.ptr, p.K, p.rows, 1, x.ld, x.ld * p.rows, kLinBJ, 1)) return cudaErrorInvalidValue;
  return gated ? lin_launch<kLinFwdGated>(m, a, stream) : lin_launch<kLinFwd>(m, a, stream);
}

cudaError_t launch_linear_dx(const LinearShape& p, RowsView dz, const uint16_t* w, RowsView res, RowsView dx,
                             uint32_t* status, cudaStream_t stream) {
  LinArgs a = lin_args(p, status);
  a.i_ext = p.K;
  a.n_it = (p.K + kLinBI - 1) / kLinBI;
  a.q_ext = p.N;
  a.out = static_cast<uint16_t*>(dx.ptr);
  a.ldo = dx.ld;
  a.res = static_cast<const uint16_t*>(res.ptr);
  a.ldr = res.ld;
  CUtensorMap m[4] = {};
  if (!lin_map(&m[0], p.f16, w, p.K, p.N, a.E, p.K, static_cast<long long>(p.N) * p.K, kLinSlab, 1) ||
      !lin_map(&m[1], p.f16, dz.ptr, p.N, p.rows, 1, dz.ld, dz.ld * p.rows, kLinBJ, 1))
    return cudaErrorInvalidValue;
  return lin_launch<kLinDx>(m, a, stream);
}

cudaError_t launch_linear_dw(const LinearShape& p, RowsView dz, RowsView x, uint16_t* dw, uint32_t* status,
                             cudaStream_t stream) {
  LinArgs a = lin_args(p, status);
  a.i_ext = p.K;
  a.n_it = (p.K + kLinBI - 1) / kLinBI;
  a.j_ext = p.N;
  a.out = dw;
  a.ldo = p.K;
  CUtensorMap m[4] = {};
  if (!lin_map(&m[0], p.f16, x.ptr, p.K, p.rows, 1, x.ld, x.ld * p.rows, kLinSlab, 1) ||
      !lin_map(&m[1], p.f16, dz.ptr, p.N, p.rows, 1, dz.ld, dz.ld * p.rows, kLinSlab, 1) ||
      !lin_map(&m[2], p.f16, x.ptr, p.K, p.rows, 1, x.ld, 0, 1, 1, 2) ||
      !lin_map(&m[3], p.f16, dz.ptr, p.N, p.rows, 1, dz.ld, 0, 1, 1, 2))
    return cudaErrorInvalidValue;
  return lin_launch<kLinDw>(m, a, stream);
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
