// Matrix products with a fused epilogue, dense or with one weight per expert, and their gradients
// (bf16 or fp16 operands, fp32 accumulation), on tcgen05 (sm_103a).
//
//   forward   y[r, n]  = act( sum_k x[r, k] w[e, n, k] + bias[e, n] ) + residual[r, n]
//   input     dx[r, k] = sum_n dz[r, n] w[e, n, k] (+ residual[r, k])
//   weight    dw[e, n, k] = sum_r dz[r, n] x[r, k]        over expert e's rows
//
// What changes between the three is which operand is contiguous along the sum: x, dz and (forward) w are, w
// and x in the gradients are not; the shared-memory descriptors take either order, so no operand is ever
// transposed in memory.
//
// The tensor core feeds its M side one row a cycle: an MMA of 128 rows of A per CTA takes 128 cycles however
// few columns N it has (measured; 256 columns fill them).  In the pair kernel's forward and input gradient the
// rows of x or dz are on M, 256 or 128 of them per tile, and 256 output columns on N: 8192^3 runs at 1.80 to
// 1.92 PFLOP/s, near what the copy of both operands into shared memory allows.  A segment's rest of up to 128
// rows takes a half tile, which its weights' way to shared memory keeps from half the time (19 experts of 384
// rows: 275 us, with whole tiles 303).  Both parts of a segment in one tile on both accumulators were slower (32
// experts of about 400 rows: 490 -> 568 us).  Weights on M and the rows on a trimmed N: the same 32 experts'
// forward, back to back, 545 us against 563, but their gradients 595 against 581 and a dense 4096 x 8192 x 2048
// product 84 against 81.
//
// Rows of experts: expert e's rows start at seg_e = sum_{e' < e} round_up(counts[e'], align) (the layout
// of moe_permute).  Padding rows are never read into a result nor written: in the forward and the input
// gradient a padding row is a row of the product that is not stored; in the weight gradient, where
// rows are summed over, each expert has tensor maps of its own whose rows end with its segment
// (expert_maps_kernel), so that what a copy takes past the end reads as zeros.  (Fetching the last partial
// slab row by row instead cost the 32-expert gradient 87 of 470 us.)
//
// Two kernels:
//  * linear_pair_kernel: a CTA pair per 256 x 256 tile (cta_group::2, each CTA half of either operand's rows in
//    shared memory), persistent, two accumulators so that one tile's epilogue runs under the next tile's MMAs.
//  * linear_split_kernel: for problems with too few tiles to fill the GPU: a cluster of up to four
//    CTAs per tile of 128 or 64 columns, each with a slice of the sum; the slices meet in shared memory.  Few
//    rows are the rule there, so the weights (or, for dw, x's columns) are on M and the rows on N.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "kernels.h"
#include "rows8.cuh"

namespace moe {

namespace {

constexpr int kLinEpiWarps = 12;            // three per TMEM lane quarter, each on every third piece of 32 columns
constexpr int kLinHop = 32 * kLinEpiWarps / 4;      // from one of a warp's pieces to its next
constexpr int kLinThreads = 64 + 32 * kLinEpiWarps;   // warp 0 loads, 1 MMA, the others drain
constexpr int kLinBI = 128;                 // rows of A per CTA (accumulator lanes)
constexpr int kLinBJ = 256;                 // rows of B per tile (MMA N, accumulator columns), at most
constexpr int kLinSlab = 64;                // terms of the sum per pipeline stage
constexpr int kLinABytes = kLinBI * 128;
constexpr int kLinMaxE = kLinearMaxExperts;
// pair kernel: a stage holds the CTA's 128 rows of A and up to 128 rows of B
constexpr int kPairB = 128 * 128;
constexpr int kPairStage = kLinABytes + kPairB;      // 32 KB
constexpr int kPairStages = 6;
constexpr int kPairSmem = 1024 + kPairStages * kPairStage + 512 + kLinEpiWarps * 2048 + 2 * kLinMaxE * 4;
// split kernel: stages of A and the tile's B rows, as many as fit
constexpr int kSplitRing = 208 * 1024;          // also: the slice's sums, then a piece per epilogue warp
constexpr int kSplitMaxStages = 12;
constexpr int kSplitSmem = 1024 + kSplitRing + 512;
static_assert(kPairSmem <= 227 * 1024 && kSplitSmem <= 227 * 1024, "shared memory budget");
static_assert(kSplitRing >= kLinBI * kLinBJ * 4 + kLinEpiWarps * 2048, "the slices' sums and the pieces fit the ring");

// The GELU forward is a mode of its own: its polynomial's registers cost the others 5% where the epilogue counts.
enum LinMode { kLinFwd = 0, kLinFwdGated = 1, kLinDx = 2, kLinDw = 3, kLinFwdGelu = 4 };

struct LinArgs {
  const int32_t* counts;      // [E] rows per expert; nullptr: one dense segment of `rows` rows
  int E, align, rows;         // rows: rows of the row buffers
  int n_it;                   // i tiles (i: output columns, j: output rows)
  int i_ext;                  // output columns (gated forward: of y; z has twice as many)
  int j_ext;                  // weight gradient: N
  int q_ext;                  // forward: K, input gradient: N
  int act, f16;
  int a_blocks, b_blocks;     // > 0: operand map with 64-column blocks as a dimension, blocks per copy
  int b_box;                  // split kernel: rows of B per copy (operands contiguous along the sum)
  int bj, stages;             // split kernel: rows j per tile, ring stages,
  int lanes;                  // rows of A per tile (the accumulator lanes in use): 128 or 64
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

// Rows j per tile where they are on N (split kernel, weight gradient) and n rows are cut into ceil(n / 256) tiles
// of equal height, a multiple of the MMA's step in N (16, over a pair 32).
constexpr int kPairStep = 32, kSplitStep = 16;
__host__ __device__ __forceinline__ int lin_tile_rows(int n, int step) {
  const int nj = (n + kLinBJ - 1) / kLinBJ;
  return nj ? ((n + nj - 1) / nj + step - 1) / step * step : step;
}

struct LinTile {
  int e, it, row0, cnt, j0, ncols, slabs;
};

// What a pair keeps about the experts' segments in shared memory.
struct LinSegs {
  int* row0;                  // [E] first row
  int* cnt;                   // [E] rows
};

// A pair's tiles: one of each round of `pairs` tiles, in order of expert, groups of 16 j tiles, i tile, j tile, so
// that the tiles that run at one time share their operands in L2 along both sides (all tall tiles before all short
// ones read every expert's weights from HBM twice: 371 against 282 us for 19 experts of 384 rows).  The pair's
// place in the round moves on by three each time: with a fixed place and experts of a tall and a short tile, an
// even number of pairs gives half of them nothing but tall ones.
// Every role walks the tiles by itself; a step costs a division and, on a new expert, a few shared-memory reads
// (a search per tile took up to half of a short tile's time).
template <int MODE>
struct LinWalk {
  const LinArgs& a;
  const LinSegs& g;
  int first, place, pairs, base, next, nj, bj;
  LinTile r;
  __device__ __forceinline__ LinWalk(const LinArgs& a_, const LinSegs& g_, int pair, int pairs_)
      : a(a_), g(g_), first(0), place(pair), pairs(pairs_), base(0), next(0), nj(1),
        bj(MODE == kLinDw ? lin_tile_rows(a_.j_ext, kPairStep) : kLinBJ) {
    r.e = -1;
  }
  __device__ __forceinline__ bool advance() {
    const int t = first + place;
    first += pairs;
    place += 3;
    if (place >= pairs) place -= pairs;
    if (t >= next) {
      int n;
      do {
        if (++r.e >= a.E) return false;
        n = MODE == kLinDw ? a.j_ext : g.cnt[r.e];
        nj = (n + bj - 1) / bj;
        base = next;
        next += a.n_it * nj;
      } while (t >= next);
      r.row0 = g.row0[r.e];
      r.cnt = g.cnt[r.e];
      r.slabs = ((MODE == kLinDw ? r.cnt : a.q_ext) + kLinSlab - 1) / kLinSlab;
    }
    unsigned u = static_cast<unsigned>(t - base);
    int j16 = 0, gj = nj;
    if (nj > 16) {
      j16 = static_cast<int>(u / (16u * a.n_it)) * 16;
      u -= static_cast<unsigned>(j16) * a.n_it;
      gj = min(16, nj - j16);
    }
    r.it = static_cast<int>(u / static_cast<unsigned>(gj));
    r.j0 = (j16 + static_cast<int>(u) - r.it * gj) * bj;
    r.ncols = min(bj, (MODE == kLinDw ? a.j_ext : r.cnt) - r.j0);
    return true;
  }
};

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

// Zero below v = -87.3, where the value's magnitude is below 1e-36: __fdividef gives 0 for a divisor past 2^126.  (Every
// other bf16 or fp16 value is within half a step of it.  With e^-|v|, whose divisor stays below 2, 16384 x 4096 gated
// outputs over 64 take 75 us instead of 71, and the gradients' pass 2.5% more.)
__device__ __forceinline__ float lin_silu(float v) { return __fdividef(v, 1.f + __expf(-v)); }
// Phi(-a), the normal distribution's tail, for 0 <= a <= 30, and e^(-a^2 / 2): Phi(-a) e^(a^2 / 2) is smooth in
// t = 1 / (1 + 0.36 a) and vanishes with it, so t times a polynomial of degree 6 in t, fitted for the least relative
// error (9e-7, for a up to 14; beyond it the exponential underflows).  (erfcf, which has more digits than a 16-bit
// result: 155 us for 16384 x 4096 outputs of a product over 64, so 82.)
__device__ __forceinline__ float normal_tail(float a, float& e) {
  const float t = __fdividef(1.f, fmaf(0.36f, a, 1.f));
  e = __expf(-0.5f * a * a);
  float q = fmaf(t, 0.047056060f, -0.179763914f);
  q = fmaf(t, q, 0.180952996f);
  q = fmaf(t, q, 0.026549993f);
  q = fmaf(t, q, 0.139719039f);
  q = fmaf(t, q, 0.141772494f);
  q = fmaf(t, q, 0.143713042f);
  return t * q * e;
}
// v Phi(v) = max(v, 0) - |v| Phi(-|v|), which cancels nowhere
__device__ __forceinline__ float lin_gelu(float v) {
  float e;
  const float a = fabsf(v) > 30.f ? 30.f : fabsf(v);   // (infinity times the tail's 0; keeps NaN)
  return (v < 0.f ? 0.f : v) - a * normal_tail(a, e);
}

// The epilogue works on pieces of 32 accumulator lanes x 32 columns per
// warp, held as four 8-column groups of 8x8 fragments: v[8n + 2h + k] of thread t is lane t/4 + 8h,
// column 8n + 2(t%4) + k of the piece (h, n, k: 0..3, 0..3, 0..1).  That is how tensor memory is read
// (16 lanes x 256 bits) and what stmatrix / ldmatrix move (transposed where the rows are on N) to and from rows
// of the output type in shared memory; from there each row's 32 columns leave (or the residual's arrive) 16 bytes per
// thread.
constexpr int kPiecePitch = 64;
constexpr int kPieceBytes = 32 * kPiecePitch;
// 16-byte unit u of row r: two neighbouring rows fill the banks, and four such pairs are turned against each other,
// so that neither eight rows' units (stmatrix) nor two rows' (the stores) share a bank.
__device__ __forceinline__ uint32_t piece_at(uint32_t stage, int r, int u) {
  return stage + static_cast<uint32_t>(r * kPiecePitch + ((u ^ ((r >> 1) & 3)) << 4));
}

// Where the sums come from: this CTA's tensor memory, or the slices that the cluster's CTAs keep in
// shared memory, added in slice order.
struct TmemSums {
  uint32_t acc;               // this warp's lane quarter, accumulator column 0
  __device__ __forceinline__ void operator()(int c0, int, float (&v)[32]) const {
    uint32_t r[2][16];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      asm volatile(
          "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
          : "=r"(r[h][0]), "=r"(r[h][1]), "=r"(r[h][2]), "=r"(r[h][3]), "=r"(r[h][4]), "=r"(r[h][5]), "=r"(r[h][6]),
            "=r"(r[h][7]), "=r"(r[h][8]), "=r"(r[h][9]), "=r"(r[h][10]), "=r"(r[h][11]), "=r"(r[h][12]), "=r"(r[h][13]),
            "=r"(r[h][14]), "=r"(r[h][15])
          : "r"(acc + c0 + (static_cast<uint32_t>(16 * h) << 16)));
    tc_wait_ld();
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[8 * n + k] = __uint_as_float(r[0][4 * n + k]);
        v[8 * n + 4 + k] = __uint_as_float(r[1][4 * n + k]);
      }
  }
};
struct ZeroSums {
  __device__ __forceinline__ void operator()(int, int, float (&v)[32]) const {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = 0.f;
  }
};
// A slice's sums in shared memory: value i of 8-column group g of epilogue thread t (of 128, one per lane) is
// float 4 * ((2g + i / 4) * 128 + t) + i % 4.  S slices, read from the CTA's own on round the cluster (so that
// they do not all read one CTA at a time) and added in that order, which is fixed by the column.
template <int S>
struct ClusterSums {
  uint32_t base;              // this thread's first value in its own shared memory
  int slice;
  __device__ __forceinline__ void operator()(int c0, int left, float (&v)[32]) const {
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      if (8 * n >= left) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[8 * n + j] = 0.f;
        continue;
      }
      const uint32_t off = base + static_cast<uint32_t>(c0 / 8 + n) * (2 * 128 * 16);
      float x[S][8];
#pragma unroll
      for (int s = 1; s < S; ++s) {
        const uint32_t p = mapa_shared(off, static_cast<uint32_t>((slice + s) & (S - 1)));
#pragma unroll
        for (int k = 0; k < 2; ++k)
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(x[s][4 * k]), "=f"(x[s][4 * k + 1]), "=f"(x[s][4 * k + 2]), "=f"(x[s][4 * k + 3])
                       : "r"(p + k * (128 * 16))
                       : "memory");
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(x[0][4 * k]), "=f"(x[0][4 * k + 1]), "=f"(x[0][4 * k + 2]), "=f"(x[0][4 * k + 3])
                     : "r"(off + k * (128 * 16))
                     : "memory");
#pragma unroll
      for (int j = 0; j < 8; ++j) v[8 * n + j] = x[0][j];
#pragma unroll
      for (int s = 1; s < S; ++s)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[8 * n + j] += x[s][j];
    }
  }
};

__device__ __forceinline__ void stmatrix_x4_t(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r0), "r"(r1),
               "r"(r2), "r"(r3)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void stmatrix_x4(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r0), "r"(r1), "r"(r2),
               "r"(r3)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts16(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// A whole piece (32 rows of 32 columns) to an output matrix by one tensor copy, whose 64-byte swizzle is
// piece_at's; rows and columns past the matrix are left out.  Called by the whole warp after its shared-memory
// writes; piece_free before the next ones.
__device__ __forceinline__ void piece_send(uint32_t stage, const CUtensorMap* map, int c0, int c1, int c2, int lane) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (lane == 0)
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];\n\t"
        "cp.async.bulk.commit_group;" ::"l"(map),
        "r"(c0), "r"(c1), "r"(c2), "r"(stage)
        : "memory");
}
__device__ __forceinline__ void piece_free(int lane) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
}

// Rows of 8 * U columns (U 16-byte units) between shared memory and the thread's share of global rows:
// unit lane % U of rows lane / U + (32 / U) s, s = 0 .. U-1.
template <int U>
struct PieceRows {
  int row, unit;
  __device__ __forceinline__ explicit PieceRows(int lane) : row(lane / U), unit(lane % U) {}
  __device__ __forceinline__ uint32_t at(uint32_t stage, int s) const {
    return piece_at(stage, row, unit) + static_cast<uint32_t>(32 / U * s * kPiecePitch);   // (whole turns further)
  }
  // p: this thread's unit of row 0 of the piece; live: its columns exist; left: rows of the piece
  __device__ __forceinline__ void store(uint32_t stage, uint16_t* p, long long ld, bool live, int left) const {
#pragma unroll
    for (int s = 0; s < U; ++s) {
      const int r = row + 32 / U * s;
      if (live && r < left) *reinterpret_cast<uint4*>(p + r * ld) = lds16(at(stage, s));
    }
  }
  __device__ __forceinline__ void fetch(uint4 (&v)[U], const uint16_t* p, long long ld, bool live, int left) const {
#pragma unroll
    for (int s = 0; s < U; ++s) {
      const int r = row + 32 / U * s;
      v[s] = live && r < left ? *reinterpret_cast<const uint4*>(p + r * ld) : make_uint4(0, 0, 0, 0);
    }
  }
};

// The forward's activation of a piece, but for the gated one.
template <int MODE>
__device__ __forceinline__ void lin_act(const LinArgs& a, const float (&v)[32], float (&o)[32]) {
#pragma unroll
  for (int j = 0; j < 32; ++j) o[j] = MODE == kLinFwdGelu ? lin_gelu(v[j]) : v[j];
  if (MODE == kLinFwd) {
    if (a.act == kActRelu) {
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = v[j] < 0.f ? 0.f : v[j];   // keeps NaN
    } else if (a.act == kActSilu) {
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = lin_silu(v[j]);
    }
  }
}

// Rows on M: the warp's 32 lanes are output rows [jw, jw + 32) of tile t, and accumulator columns [cb, ce)
// output columns from i0 + cb on (gated forward: columns 16m + 0..7 are the gate columns of y's columns
// i0 + 8m .., columns 16m + 8..15 their up columns).  Every third piece of columns from piece `par` on.
template <int MODE>
__device__ __forceinline__ void lin_drain_rows(const LinArgs& a, const LinTile& t, int i0, int jw, int cb, int ce,
                                               uint32_t acc, int par, int lane, uint32_t stage, const CUtensorMap* mapo) {
  constexpr bool kGated = MODE == kLinFwdGated, kFwd = MODE == kLinFwd || MODE == kLinFwdGelu || kGated;
  constexpr int kU = kGated ? 2 : 4;                  // 16-byte units per output row
  const int left = t.ncols - jw;
  if (left <= 0) return;
  const long long jr = static_cast<long long>(t.row0) + t.j0 + jw;
  const PieceRows<kU> rows(lane);
  const TmemSums sums{acc};
  // this thread's matrix row for stmatrix / ldmatrix: row `lane` of the piece, 16-byte unit n
  auto mat = [&](int n) { return piece_at(stage, lane, n); };
  auto col_of = [&](int c) { return i0 + (kGated ? c / 2 : c); };
  // the residual of the next piece is on its way while this one is worked on
  const bool has_res = a.res != nullptr;
  uint4 res[kU];
  auto fetch = [&](int c) {
    const int col = col_of(c) + rows.unit * 8;
    rows.fetch(res, a.res + jr * a.ldr + col, a.ldr, col < a.i_ext, left);
  };
  const int c_acc = cb;       // accumulator column 0
  cb += 32 * par;
  if (has_res && cb < ce) fetch(cb);
#pragma unroll 1
  for (int c0 = cb; c0 < ce; c0 += kLinHop) {
    const int col0 = col_of(c0);
    if (col0 >= a.i_ext) break;
    float v[32];
    sums(c0 - c_acc, 32, v);
    piece_free(lane);
    if (kFwd) {
      if (a.bias) {
        const float* b = a.bias + static_cast<size_t>(t.e) * (kGated ? 2 * a.i_ext : a.i_ext);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int col = col0 + (kGated ? (n >> 1) * 8 : n * 8) + 2 * (lane & 3);
          if (col >= a.i_ext) continue;               // i_ext is a multiple of 8
          const float2 x = __ldg(reinterpret_cast<const float2*>(b + col + (kGated && (n & 1) ? a.i_ext : 0)));
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            v[8 * n + 2 * h] += x.x;
            v[8 * n + 2 * h + 1] += x.y;
          }
        }
      }
      if (a.z) {
        const PieceRows<4> zr(lane);
        const int zc = kGated ? col0 + (zr.unit >> 1) * 8 : col0 + zr.unit * 8;
        __syncwarp();
#pragma unroll
        for (int n = 0; n < 4; ++n)
          stmatrix_x4(mat(n), lin_pack(v[8 * n], v[8 * n + 1], a.f16), lin_pack(v[8 * n + 2], v[8 * n + 3], a.f16),
                      lin_pack(v[8 * n + 4], v[8 * n + 5], a.f16), lin_pack(v[8 * n + 6], v[8 * n + 7], a.f16));
        __syncwarp();
        zr.store(stage, a.z + jr * a.ldz + zc + (kGated && (zr.unit & 1) ? a.i_ext : 0), a.ldz, zc < a.i_ext, left);
      }
    }
    float o[kGated ? 16 : 32];                        // o[8m + 2h + k]: column 8m + 2(t%4) + k, row t/4 + 8h
    if constexpr (kGated) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 8; ++i) o[8 * m + i] = lin_silu(v[16 * m + i]) * v[16 * m + 8 + i];
    } else {
      lin_act<MODE>(a, v, o);
    }
    __syncwarp();
    if (has_res) {
#pragma unroll
      for (int s = 0; s < kU; ++s) sts16(rows.at(stage, s), res[s]);
      __syncwarp();
#pragma unroll
      for (int m = 0; m < kU; ++m) {
        uint32_t r[4];
        ldmatrix_x4(mat(m), r);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const float2 x = lin_unpack(r[h], a.f16);
          o[8 * m + 2 * h] += x.x;
          o[8 * m + 2 * h + 1] += x.y;
        }
      }
      if (c0 + kLinHop < ce) fetch(c0 + kLinHop);
      __syncwarp();
    }
#pragma unroll
    for (int m = 0; m < kU; ++m)
      stmatrix_x4(mat(m), lin_pack(o[8 * m], o[8 * m + 1], a.f16), lin_pack(o[8 * m + 2], o[8 * m + 3], a.f16),
                  lin_pack(o[8 * m + 4], o[8 * m + 5], a.f16), lin_pack(o[8 * m + 6], o[8 * m + 7], a.f16));
    __syncwarp();
    if (!kGated && (left >= 32 || !a.counts)) {       // (an expert's rows end before the matrix does)
      piece_send(stage, mapo, col0, static_cast<int>(jr), 0, lane);
    } else {
      const int col = col0 + rows.unit * 8;
      rows.store(stage, a.out + jr * a.ldo + col, a.ldo, col < a.i_ext, left);
    }
  }
  __syncwarp();
}

// Rows on N: turns the sums of output rows [j0 + cb, j0 + ce) of tile t into outputs (cb a multiple of 8); this
// warp has lanes 32q .. of the CTA's output columns, which start at column i0 (gated forward: of y), and
// every third piece of rows from piece `par` on.  stage: the warp's piece in shared memory.
template <int MODE, class Sums>
__device__ __forceinline__ void lin_drain(const LinArgs& a, const LinTile& t, int i0, int cb, int ce, const Sums& sums, int q,
                                          int par, int lane, uint32_t stage, const CUtensorMap* mapo = nullptr) {
  constexpr bool kGated = MODE == kLinFwdGated, kFwd = MODE == kLinFwd || MODE == kLinFwdGelu || kGated;
  constexpr int kU = kGated ? 2 : 4;                  // 16-byte units per output row
  // accumulator lane l of the warp is output column iw + l; gated: lanes 16m + 0..7 are the gate rows of
  // columns iw + 8m .., lanes 16m + 8..15 their up rows
  const int iw = kGated ? i0 + q * 16 : i0 + q * 32;
  float bias[4] = {0.f, 0.f, 0.f, 0.f};
  if (kFwd && a.bias) {
    const float* b = a.bias + static_cast<size_t>(t.e) * (kGated ? 2 * a.i_ext : a.i_ext);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int col = kGated ? iw + (h >> 1) * 8 + (lane >> 2) : iw + 8 * h + (lane >> 2);
      if (col < a.i_ext) bias[h] = __ldg(b + col + (kGated && (h & 1) ? a.i_ext : 0));
    }
  }
  // output row of accumulator column 0
  const long long jr = MODE == kLinDw ? static_cast<long long>(t.e) * a.j_ext + t.j0 : static_cast<long long>(t.row0) + t.j0;
  const PieceRows<kU> rows(lane);
  const int col = iw + rows.unit * 8;
  const bool live = col < a.i_ext;                    // i_ext is a multiple of 8
  // this thread's matrix row for stmatrix / ldmatrix: row lane % 8 of matrix lane / 8
  const uint32_t mat = piece_at(stage, lane & 7, lane >> 3);
  // the residual of the next piece is on its way while this one is worked on
  const bool has_res = MODE != kLinDw && a.res != nullptr;
  uint4 res[kU];
  cb += 32 * par;
  if (has_res) rows.fetch(res, a.res + (jr + cb) * a.ldr + col, a.ldr, live, ce - cb);
#pragma unroll 1
  for (int c0 = cb; c0 < ce; c0 += kLinHop) {
    const int left = ce - c0;
    float v[32];
    sums(c0, left, v);
    if (mapo) piece_free(lane);
    if (kFwd) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] += bias[(j >> 1) & 3];
      if (a.z) {
        const PieceRows<4> zr(lane);
        const int zc = kGated ? iw + (zr.unit >> 1) * 8 : iw + zr.unit * 8;
        __syncwarp();
#pragma unroll
        for (int n = 0; n < 4; ++n)
          stmatrix_x4_t(mat + n * 8 * kPiecePitch, lin_pack(v[8 * n], v[8 * n + 1], a.f16),
                        lin_pack(v[8 * n + 2], v[8 * n + 3], a.f16), lin_pack(v[8 * n + 4], v[8 * n + 5], a.f16),
                        lin_pack(v[8 * n + 6], v[8 * n + 7], a.f16));
        __syncwarp();
        zr.store(stage, a.z + (jr + c0) * a.ldz + zc + (kGated && (zr.unit & 1) ? a.i_ext : 0), a.ldz, zc < a.i_ext, left);
      }
    }
    constexpr int kV = kGated ? 16 : 32;              // gated: o[4n + 2m + k] is column iw + 8m + t/4
    float o[kV];
    if constexpr (kGated) {
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          o[4 * n + k] = lin_silu(v[8 * n + k]) * v[8 * n + 2 + k];
          o[4 * n + 2 + k] = lin_silu(v[8 * n + 4 + k]) * v[8 * n + 6 + k];
        }
    } else {
      lin_act<MODE>(a, v, o);
    }
    // gated: two 8-column groups of rows make one x4 (matrix m: columns 8 (m & 1), rows 8 (m >> 1))
    const uint32_t om = kGated ? piece_at(stage, (lane >> 4) * 8 + (lane & 7), (lane >> 3) & 1) : mat;
    constexpr int kSteps = kGated ? 2 : 4, kStepRows = 32 / kSteps;
    __syncwarp();
    if (has_res) {
#pragma unroll
      for (int s = 0; s < kU; ++s) sts16(rows.at(stage, s), res[s]);
      __syncwarp();
#pragma unroll
      for (int n = 0; n < kSteps; ++n) {
        uint32_t r[4];
        ldmatrix_x4_t(om + n * kStepRows * kPiecePitch, r);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float2 x = lin_unpack(r[m], a.f16);
          o[8 * n + 2 * m] += x.x;
          o[8 * n + 2 * m + 1] += x.y;
        }
      }
      if (c0 + kLinHop < ce) rows.fetch(res, a.res + (jr + c0 + kLinHop) * a.ldr + col, a.ldr, live, left - kLinHop);
      __syncwarp();
    }
#pragma unroll
    for (int n = 0; n < kSteps; ++n)
      stmatrix_x4_t(om + n * kStepRows * kPiecePitch, lin_pack(o[8 * n], o[8 * n + 1], a.f16),
                    lin_pack(o[8 * n + 2], o[8 * n + 3], a.f16), lin_pack(o[8 * n + 4], o[8 * n + 5], a.f16),
                    lin_pack(o[8 * n + 6], o[8 * n + 7], a.f16));
    __syncwarp();
    if (mapo)       // weight gradient of the pair kernel
      piece_send(stage, mapo, iw, t.j0 + c0, t.e, lane);
    else
      rows.store(stage, a.out + (jr + c0) * a.ldo + col, a.ldo, live, left);
  }
  __syncwarp();
}

// Loads the operand of the output's columns, from column i0 on (gated: i0 of y), and q0 .. of the sum: w, in the
// weight gradient x.
template <int MODE, bool PAIR>
__device__ __forceinline__ void lin_load_a(const LinArgs& a, const CUtensorMap* map, uint32_t dst, const LinTile& t, int i0,
                                           int q0, uint32_t bar) {
  if (MODE == kLinFwd || MODE == kLinFwdGelu) {
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
      if (PAIR || a.lanes > 64) tma_load_4d<PAIR>(dst + 8192, map, i0 + 64, row, 0, plane, bar);
    }
  }
}

// Maps of the operand of the output's rows (x or dz).  Pair kernel: [0] copies 128 rows at a time, [1] 64; split
// kernel and weight gradient: [0].
struct LinMapsB {
  CUtensorMap m[2];
};

// Loads that operand's rows j .. j + n (n a multiple of 8), q0 .. of the sum: lin_b_bytes in all.
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
    tma_load_4d<PAIR>(dst, map, q0, t.row0 + j, 0, 0, bar);
  }
}
template <int MODE>
__device__ __forceinline__ uint32_t lin_b_bytes(const LinArgs& a, int n) {
  if (MODE == kLinDw) return static_cast<uint32_t>(a.b_blocks ? a.b_blocks : (n + 63) / 64) * 8192u;
  return static_cast<uint32_t>(a.b_box) * 128u;
}

// ------------------------------------------------------------------------------------------

__device__ __forceinline__ void tensormap_acquire(const CUtensorMap* m) {
  asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(m) : "memory");
}

// Copies of two maps (the weight gradient's of x and dz, else the rows operand's for 128 and 64 rows) for each
// expert, their rows (dimension 1) ending with the expert's segment.  One CTA, thread = expert.
__global__ void __launch_bounds__(kLinMaxE) expert_maps_kernel(const __grid_constant__ CUtensorMap mapa,
                                                               const __grid_constant__ CUtensorMap mapb,
                                                               const int32_t* __restrict__ counts, int E, int align, int rows,
                                                               CUtensorMap* emaps) {
  __shared__ int sums[kLinMaxE / 32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int e = threadIdx.x, warp = e / 32, lane = e % 32;
  const int c = e < E ? min(max(__ldg(counts + e), 0), rows) : 0;
  const int padded = (c + align - 1) / align * align;
  int s = padded;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s = min(s + o, 0x3fffffff);
  }
  if (lane == 31) sums[warp] = s;
  __syncthreads();
  for (int w = 0; w < warp; ++w) s = min(s + sums[w], 0x3fffffff);
  if (e >= E) return;
  const int end = max(min(s - padded + c, rows), 1);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    CUtensorMap* m = emaps + 2 * e + k;
    const uint4* src = reinterpret_cast<const uint4*>(k ? &mapb : &mapa);
#pragma unroll
    for (int i = 0; i < 8; ++i) reinterpret_cast<uint4*>(m)[i] = src[i];
    asm volatile("tensormap.replace.tile.global_dim.global.b1024.b32 [%0], 1, %1;" ::"l"(m), "r"(end) : "memory");
  }
  asm volatile("fence.proxy.tensormap::generic.release.gpu;" ::: "memory");
}

// Bound by the tensor core and shared memory alike: a slab of 64 terms takes 512 cycles of MMAs, in which either CTA's
// 32 KB of it are copied in and read by the MMAs, 128 bytes a cycle, all that an SM's shared memory moves (measured:
// 546 to 590 cycles a slab).  An epilogue's pieces go through it too, 128 KB a tile: with six slabs to a tile (experts'
// weight gradients) a slab takes 750.  8192^3 bf16 597 us (1.84
// PFLOP/s, 97% of the measured rate of library products); 4096^3 82 us (1.68; 256 tiles on 76 pairs leave 16% of the
// last round empty, and the tensor core is busy for 86% of the SMs' active cycles); 4096 x 7168 over 2048 with bias and
// residual 73 us, 82 under the power limit (1705 MHz instead of 2070); 12288 rows of 32 experts, 4096 x 7168, SwiGLU 490 to 590 us by the box's power limit, 16% of it for
// the rows that fill their tiles up.
// Tried and not kept: tiles claimed from a counter instead of dealt out (both gradients of the 32 experts 585 -> 607 us);
// two pieces per epilogue warp in turn (within 2% either way); pieces of two warps as one copy of 128-byte rows
// (16384 x 4096 over 64 36 -> 41 us); the last round's dense tiles in halves (1 to 4%, lost in the noise).
// With sums below about 512 terms the epilogue is the longest way, 500 cycles a piece: 16384 x 4096 outputs over 64
// 34.6 us, with a residual 74, SiLU 54, GELU 82 (with two warps per quarter 36, 84, 60 and 86; experts'
// products over long sums are 1% faster with two).
// mapa: map of the operand of the output's columns (w, in the weight gradient x), mapsb: of its rows, mapo: of the
// output, 32 x 32 pieces.  emaps: expert e's maps at 2e and 2e + 1 (see expert_maps_kernel), or null.
template <int MODE>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap mapa, const __grid_constant__ LinMapsB mapsb,
                       const __grid_constant__ CUtensorMap mapo, const CUtensorMap* __restrict__ emaps, const LinArgs a) {
  constexpr bool kRowsM = MODE != kLinDw;                       // A: rows of x or dz, B: weights; else A: x, B: dz
  constexpr bool kAMn = MODE == kLinDw, kBMn = MODE == kLinDx || MODE == kLinDw;
  constexpr int kCtaI = MODE == kLinFwdGated ? 64 : kLinBI;     // output columns per CTA
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kPairStages * kPairStage);   // even CTA: both CTAs' tiles landed
  uint64_t* empty = full + kPairStages;        // each CTA: the pair's MMAs have read the stage
  uint64_t* acc_full = empty + kPairStages;    // [2] each CTA: accumulator written
  uint64_t* acc_empty = acc_full + 2;          // [2] even CTA: drained by both CTAs
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint8_t* pieces = smem + kPairStages * kPairStage + 512;                    // one per epilogue warp
  LinSegs segs;
  segs.row0 = reinterpret_cast<int*>(pieces + kLinEpiWarps * kPieceBytes);
  segs.cnt = segs.row0 + kLinMaxE;

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
      mbar_init(smem_u32(acc_empty + b), 2 * kLinEpiWarps);
    }
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&mapa);
    prefetch_tmap(&mapsb.m[0]);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 2 * kLinBJ);
    tmem_relinquish_pair();
  }
  grid_dependency_wait();        // everything below reads what the stream's previous kernels wrote
  grid_launch_dependents();
  if (warp == 2) {
    // segment starts; a segment that would leave the buffers is an error and is cut
    int srun = 0;
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
      if (e < a.E) {
        segs.row0[e] = start;
        segs.cnt[e] = c;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();      // both CTAs' barriers exist before any cross-CTA arrival
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ---------------- loads: this CTA's half of A and of B ----------------
    const uint32_t full0 = mapa_shared(smem_u32(full), 0);
    int st = 0;
    uint32_t ph = 0;
    int e_maps = -1;
    bool ok = true;
    LinWalk<MODE> walk(a, segs, pair, pairs);
    while (ok && walk.advance()) {
      const LinTile& t = walk.r;
      const int half = ((t.ncols + kPairStep - 1) & ~(kPairStep - 1)) / 2;
      const int mrows = t.ncols <= 128 ? 64 : 128;
      const CUtensorMap *ma = &mapa, *mb = &mapsb.m[0], *mr = &mapsb.m[mrows == 64];
      if (emaps != nullptr) {
        const CUtensorMap* em = emaps + 2 * t.e;
        if (e_maps != t.e && t.slabs) {      // written by the launch before this one
          e_maps = t.e;
          tensormap_acquire(em);
          tensormap_acquire(em + 1);
        }
        if (kRowsM) {
          mr = em + (mrows == 64);
        } else {
          ma = em;
          mb = em + 1;
        }
      }
      const int i0 = (t.it * 2 + rank) * kCtaI, j0 = t.j0 + rank * half;
      const uint32_t bytes = kPairB + (kRowsM ? static_cast<uint32_t>(mrows) * 128u : lin_b_bytes<MODE>(a, half));
      for (int s = 0; s < t.slabs; ++s) {
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(empty + st), ph ^ 1, a.status) && *abort_flag == 0);
        if (!ok) break;
        const uint32_t sa = smem_u32(smem + st * kPairStage), sb = sa + kLinABytes, fb = full0 + st * 8;
        const int q0 = s * kLinSlab;
        if (rank == 0 && lane == 0) mbar_arrive_expect_tx(smem_u32(full + st), 2 * bytes);
        __syncwarp();
        if (lane == 0) {
          if (kRowsM) {
            tma_load_4d<true>(sa, mr, q0, t.row0 + t.j0 + rank * mrows, 0, 0, fb);
            lin_load_a<MODE, true>(a, ma, sb, t, i0, q0, fb);
          } else {
            lin_load_a<MODE, true>(a, ma, sa, t, i0, q0, fb);
            lin_load_b<MODE, true>(a, mb, sb, t, j0, half, q0, fb);
          }
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
      LinWalk<MODE> walk(a, segs, pair, pairs);
      while (ok && walk.advance()) {
        const LinTile& t = walk.r;
        if (t.slabs == 0) continue;
        const uint32_t id =
            kRowsM ? lin_idesc(a.f16, kAMn, kBMn, t.ncols <= 128 ? kLinBI : 2 * kLinBI, kLinBJ)
                   : lin_idesc(a.f16, kAMn, kBMn, 2 * kLinBI, static_cast<uint32_t>((t.ncols + kPairStep - 1) & ~(kPairStep - 1)));
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
    // ---------------- epilogue: this CTA's accumulator lanes ----------------
    const int q = warp & 3, par = (warp - 2) >> 2;   // the TMEM lane quarter this warp may read
    const uint32_t acc_empty0 = mapa_shared(smem_u32(acc_empty), 0), stage = smem_u32(pieces + (warp - 2) * kPieceBytes);
    int b = 0;
    uint32_t aph = 0;
    bool ok = true;
    LinWalk<MODE> walk(a, segs, pair, pairs);
    while (ok && walk.advance()) {
      const LinTile& t = walk.r;
      const int i0 = (t.it * 2 + rank) * kCtaI;
      if (MODE == kLinDw && t.slabs == 0) {
        lin_drain<MODE>(a, t, i0, 0, t.ncols, ZeroSums{}, q, par, lane, stage, &mapo);
        continue;
      }
      ok = mbar_wait(smem_u32(acc_full + b), (aph >> b) & 1u, a.status) && *abort_flag == 0;
      ok = named_barrier_and(1, 32 * kLinEpiWarps, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(b * kLinBJ);
      if constexpr (!kRowsM) {
        lin_drain<MODE>(a, t, i0, 0, t.ncols, TmemSums{acc}, q, par, lane, stage, &mapo);
      } else if (t.ncols > 128) {
        // M = 256: this CTA's 128 rows, all 256 columns
        lin_drain_rows<MODE>(a, t, t.it * 2 * kCtaI, rank * 128 + q * 32, 0, kLinBJ, acc, par, lane, stage, &mapo);
      } else {
        // M = 128: this CTA's 64 rows twice, columns 0..127 in lanes 0..63 and 128..255 in lanes 64..127
        lin_drain_rows<MODE>(a, t, t.it * 2 * kCtaI, rank * 64 + (q & 1) * 32, (q >> 1) * 128, (q >> 1) * 128 + 128, acc, par,
                             lane, stage, &mapo);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(acc_empty0 + b * 8);
      aph ^= 1u << b;
      b ^= 1;
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
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

// The expert, its segment and the first row of tile tj of all experts' tiles of a.bj rows.  One warp; false: there are
// not that many.  A segment that would leave the buffers is an error and is cut.
__device__ __forceinline__ bool lin_find_tile(const LinArgs& a, int tj, int lane, LinTile& t) {
  int row = 0, tiles = 0;
  for (int e0 = 0; e0 < a.E; e0 += 32) {
    const int e = e0 + lane;
    int c = e < a.E ? __ldg(a.counts + e) : 0;
    if (c < 0 || c > a.rows) {
      record_error(a.status, kDevErrIndex);
      c = c < 0 ? 0 : a.rows;
    }
    const int padded = (c + a.align - 1) / a.align * a.align, nt = (c + a.bj - 1) / a.bj;
    int s = padded, n = nt;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int os = __shfl_up_sync(0xffffffffu, s, d), on = __shfl_up_sync(0xffffffffu, n, d);
      if (lane >= d) {
        s = min(s + os, 0x3fffffff);
        n = min(n + on, 0x3fffffff);
      }
    }
    const int start = min(row + s - padded, 0x3fffffff), first = min(tiles + n - nt, 0x3fffffff);
    if (c > 0 && start + c > a.rows) {
      record_error(a.status, kDevErrIndex);
      c = max(a.rows - start, 0);
    }
    const unsigned hit = __ballot_sync(0xffffffffu, tj >= first && tj - first < nt);
    if (hit) {
      const int src = __ffs(static_cast<int>(hit)) - 1;
      t.e = e0 + src;
      t.row0 = __shfl_sync(0xffffffffu, start, src);
      t.cnt = __shfl_sync(0xffffffffu, c, src);
      t.j0 = (tj - __shfl_sync(0xffffffffu, first, src)) * a.bj;
      return t.j0 < t.cnt;
    }
    row = min(row + __shfl_sync(0xffffffffu, s, 31), 0x3fffffff);
    tiles = min(tiles + __shfl_sync(0xffffffffu, n, 31), 0x3fffffff);
  }
  return false;
}

// One token, 4096 x 7168 gated (58.7 MB of weights) 13.8 us, 4.3 TB/s: 5 us of launch, first loads and the slices'
// meeting, then the weights at 6.6 TB/s.  256 x 7168 over 2048 15.4 us.
// Few tiles: cluster c computes tile c, its CTA r the r-th of S slices of the sum.  A tile may use 64 of the MMA's
// 128 lanes: the others multiply what the ring happens to hold and are not read.  Experts (forward and input
// gradient): tiles of a.bj rows, as many clusters as there can be tiles; rows past an expert's end are other
// columns of the product, which are not stored.
template <int MODE, int S>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_split_kernel(const __grid_constant__ CUtensorMap mapa, const __grid_constant__ CUtensorMap mapb, const LinArgs a) {
  constexpr bool kAMn = MODE == kLinDx || MODE == kLinDw, kBMn = MODE == kLinDw;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kSplitRing);
  uint64_t* empty = full + kSplitMaxStages;
  uint64_t* acc_full = empty + kSplitMaxStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int slice = static_cast<int>(blockIdx.x) % S, tile = static_cast<int>(blockIdx.x) / S;
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
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t tmem = *tmem_slot;

  LinTile t;
  t.e = 0;
  t.row0 = 0;
  t.cnt = MODE == kLinDw ? a.j_ext : a.rows;
  t.it = tile % a.n_it;
  t.j0 = tile / a.n_it * a.bj;
  if (MODE != kLinDw && a.counts != nullptr) {
    __shared__ LinTile found;
    if (warp == 2) {
      if (!lin_find_tile(a, tile / a.n_it, lane, t)) t.cnt = t.j0 = 0;
      if (lane == 0) found = t;
    }
    __syncthreads();
    t.e = found.e;
    t.row0 = found.row0;
    t.cnt = found.cnt;
    t.j0 = found.j0;
  }
  t.ncols = min(a.bj, t.cnt - t.j0);          // 0 (experts): no tile for this cluster
  t.slabs = ((MODE == kLinDw ? a.rows : a.q_ext) + kLinSlab - 1) / kLinSlab;
  const int i0 = t.it * (MODE == kLinFwdGated ? a.lanes / 2 : a.lanes);
  const int s0 = static_cast<int>(static_cast<long long>(t.slabs) * slice / S);          // this CTA's slabs [s0, s1),
  const int s1 = static_cast<int>(static_cast<long long>(t.slabs) * (slice + 1) / S);    // never empty (host)
  const uint32_t b_bytes = lin_b_bytes<MODE>(a, a.bj);
  const uint32_t a_bytes = static_cast<uint32_t>(a.lanes) * 128;
  const int stage = static_cast<int>(a_bytes + ((b_bytes + 1023) & ~1023u));
  const uint32_t piece = smem_u32(smem) + kLinBI * kLinBJ * 4 + static_cast<uint32_t>(warp >= 2 ? warp - 2 : 0) * kPieceBytes;

  if (t.ncols <= 0) {
    // nothing to do but meet the cluster below
  } else if (warp == 0) {
    int st = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int s = s0; s < s1; ++s) {
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(empty + st), ph ^ 1, a.status) && *abort_flag == 0);
      if (!ok) break;
      if (lane == 0) {
        const uint32_t sa = smem_u32(smem + st * stage), fb = smem_u32(full + st);
        mbar_arrive_expect_tx(fb, a_bytes + b_bytes);
        lin_load_a<MODE, false>(a, &mapa, sa, t, i0, s * kLinSlab, fb);
        lin_load_b<MODE, false>(a, &mapb, sa + a_bytes, t, t.j0, a.bj, s * kLinSlab, fb);
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
        const uint32_t sa = smem_u32(smem + st * stage), sb = sa + a_bytes;
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
    const int q = warp & 3, par = (warp - 2) >> 2;
    bool ok = mbar_wait(smem_u32(acc_full), 0, a.status) && *abort_flag == 0;
    ok = named_barrier_and(1, 32 * kLinEpiWarps, ok);
    tc_fence_after();
    if (!ok) {
      *abort_flag = 1;
    } else {
      const bool used = q * 32 < a.lanes;
      const TmemSums mine{tmem + (static_cast<uint32_t>(q * 32) << 16)};
      if (S == 1) {
        if (used) lin_drain<MODE>(a, t, i0, 0, t.ncols, mine, q, par, lane, piece);
      } else {
        // every MMA has read the ring: it takes this slice's sums, as ClusterSums reads them
        float4* part = reinterpret_cast<float4*>(smem) + q * 32 + lane;
#pragma unroll 1
        for (int c0 = 32 * par; used && c0 < t.ncols; c0 += kLinHop) {
          float v[32];
          mine(c0, 32, v);
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            if (c0 + (j & ~7) < t.ncols) part[(c0 + j) / 4 * 128] = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
      }
    }
  }
  __syncthreads();
  if (S > 1) {
    const bool ok = *abort_flag == 0;
    cluster_sync();
    if (t.ncols > 0 && warp >= 2 && ok && (warp & 3) * 32 < a.lanes) {
      const int q = warp & 3, par = (warp - 2) >> 2;
      const int w = ((t.ncols + S - 1) / S + 7) & ~7, cb = min(slice * w, t.ncols), ce = min(cb + w, t.ncols);
      lin_drain<MODE>(a, t, i0, cb, ce, ClusterSums<S>{smem_u32(reinterpret_cast<float4*>(smem) + q * 32 + lane), slice},
                      q, par, lane, piece);
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
bool lin_map(CUtensorMap* m, int f16, const void* p, int n, const long long* d, const long long* s, const int* b,
             CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
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
             const_cast<void*>(p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
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

// How a problem runs.
struct LinPlan {
  bool pair;
  int lanes;
  int split, bj, stages, grid, b_box;
};

// The cheapest way to run a problem by a count of cycles that was fitted to measurements of every
// way (pair; split with 128 or 64 lanes and 1, 2 or 4 slices) over 132 dense shapes of 1 to 4096 rows, 256 to 7168
// columns and terms: the way it picks is on average 0.2% off the fastest one, 4% at most.
//  * pair: 76 tiles at a time, 420 a slab, 1000 and 16 per row j of the epilogue at the end;
//  * split: 590 a slab (the MMA feeds its 128 rows of A at one a cycle, so short tiles are no cheaper), 5200 for each
//    further round of CTAs; slices halve or quarter that for a meeting of 1900 + 250 S and 27 per row j and 128
//    lanes for the partial sums over the cluster.
// (Clusters of eight do not fill the GPU: 16 of them took two rounds.)
// Experts' rows are not known here: taken are those of buffers that the experts' padding fills up, about evenly
// spread, in split tiles of twice an expert's share.  Fitted to 89 shapes of 2 to 64 experts and 1 to 7000 rows (1.8%
// from the fastest way on average, 24% faster than the pair kernel alone): pair 590 a slab, 6000 at the start and 300
// an expert, whose segments every CTA lays out; split 10000 for a further round and 3000 for each round of clusters that
// there might be tiles for.
// i_cols: output columns, gated: of y; j: rows of the output (dense) or of the row buffers; whole: the pair kernel in
// any case (experts' weight gradient).
LinPlan lin_plan(const LinearShape& s, int i_cols, bool gated, long long j, long long q, bool b_mn, bool whole) {
  LinPlan p{};
  const int sms = num_sms(), pairs = sms > 1 ? sms / 2 : 1, E = s.counts ? s.E : 0;      // (no device: one SM)
  const long long slabs = (q + kLinSlab - 1) / kLinSlab;
  p.lanes = kLinBI;
  p.split = 1;
  p.pair = true;
  const int pair_i = gated ? kLinBI : 2 * kLinBI;
  const long long n_it = (i_cols + pair_i - 1) / pair_i;
  long long rows = j, live = 1, tiles, most = 0;       // live experts, tiles of rows of all of them, at most
  int bj = lin_tile_rows(static_cast<int>(j), kSplitStep);
  if (E) {
    p.bj = kLinBJ;                                     // (the weight gradient's goes by N, as for a dense problem)
    if (whole) p.bj = lin_tile_rows(static_cast<int>(j), kPairStep);
    p.grid = 2 * pairs;
    if (whole) return p;
    rows = j - static_cast<long long>(E) * (s.align - 1);
    if (rows < 1) rows = 1;
    live = rows < E ? rows : E;
    const long long twice = (2 * rows + live - 1) / live;
    bj = twice >= kLinBJ ? kLinBJ : static_cast<int>((twice + kSplitStep - 1) / kSplitStep * kSplitStep);
    if (bj < 2 * kSplitStep) bj = 2 * kSplitStep;
    const long long mean = (rows + kLinBJ / 2 * live) / kLinBJ;   // of sum_e ceil(rows_e / 256)
    tiles = n_it * (mean > live ? mean : live);
    most = j / bj + (j < E ? j : E);
  } else {
    p.bj = lin_tile_rows(static_cast<int>(j), kPairStep);
    tiles = n_it * ((j + p.bj - 1) / p.bj);
    p.grid = 2 * static_cast<int>(tiles < pairs ? tiles : pairs);
  }
  const long long slab = E ? 590 : 420, more = E ? 10000 : 5200;
  long long best = (tiles + pairs - 1) / pairs * slabs * slab + (E ? 6000 + 300 * E : 1000 + 16 * p.bj);
  long long nj = E ? (2 * rows + live * bj) / (2 * bj) : (j + bj - 1) / bj;
  if (nj < live) nj = live;
  for (int lanes = 128; lanes >= 64; lanes /= 2) {
    const int tile_i = gated ? lanes / 2 : lanes;
    const long long it = (i_cols + tile_i - 1) / tile_i, t1 = it * nj, all = E ? it * most : t1;
    for (int S = 1; S <= 4 && slabs >= 2 * S; S *= 2) {
      if (all * S > 0x3fffffff) continue;
      const long long rounds = (t1 * S + sms - 1) / sms, spare = ((all - t1) * S + sms - 1) / sms;
      long long cost = rounds * ((slabs + S - 1) / S * 590 + 2 * bj / S) + more * (rounds - 1) + (spare > 0 ? 3000 * spare : 0);
      if (S > 1) cost += rounds * (1900 + 250 * S + 27LL * bj * lanes / 128 * (S - 1) / S);
      if (cost >= best) continue;
      best = cost;
      p.pair = false;
      p.lanes = lanes;
      p.split = S;
      p.grid = static_cast<int>(all) * S;
    }
  }
  if (p.pair) return p;
  p.bj = bj;
  p.b_box = bj;
  const int b_bytes = b_mn ? (bj + 63) / 64 * 8192 : bj * 128;
  const int stage = p.lanes * 128 + (b_bytes + 1023) / 1024 * 1024;
  // (64 lanes: the MMA reads 8 KB past a stage's A, which stays inside the ring)
  p.stages = (kSplitRing - 8192) / stage < kSplitMaxStages ? (kSplitRing - 8192) / stage : kSplitMaxStages;
  return p;
}

// Output columns per tile (of a pair: both CTAs').
int lin_tile_i(const LinPlan& p, bool gated) { return (p.pair ? 2 * p.lanes : p.lanes) / (gated ? 2 : 1); }

template <int MODE>
cudaError_t lin_launch(const LinPlan& p, const CUtensorMap& ma, const LinMapsB& mb, const CUtensorMap* emaps, LinArgs a,
                       cudaStream_t stream) {
  CUtensorMap mo = {};
  if (p.pair) {
    // the output (weight gradient: [E][N][K]) in pieces of 32 rows of 32 columns
    const long long rows = MODE == kLinDw ? a.j_ext : a.rows;
    const long long d[3] = {a.i_ext, rows, MODE == kLinDw ? a.E : 1}, st[3] = {0, a.ldo, a.ldo * rows};
    const int b[3] = {32, 32, 1};
    if (!lin_map(&mo, a.f16, a.out, 3, d, st, b, CU_TENSOR_MAP_SWIZZLE_64B)) return cudaErrorInvalidValue;
  }
  static std::atomic<unsigned long long> pair_done{0}, split_done[3] = {};
  a.bj = p.bj;
  a.stages = p.stages;
  a.lanes = p.lanes;
  a.b_box = p.b_box;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = static_cast<unsigned>(p.pair ? 2 : p.split);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(p.grid);
  cfg.blockDim = dim3(kLinThreads);
  cfg.dynamicSmemBytes = p.pair ? kPairSmem : kSplitSmem;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  if (p.pair) {
    const cudaError_t err = allow_smem(reinterpret_cast<const void*>(&linear_pair_kernel<MODE>), kPairSmem, pair_done);
    if (err != cudaSuccess) return err;
    return cudaLaunchKernelEx(&cfg, linear_pair_kernel<MODE>, ma, mb, mo, emaps, static_cast<const LinArgs>(a));
  }
  const auto kernel = p.split == 1   ? linear_split_kernel<MODE, 1>
                      : p.split == 2 ? linear_split_kernel<MODE, 2>
                                     : linear_split_kernel<MODE, 4>;
  const cudaError_t err = allow_smem(reinterpret_cast<const void*>(kernel), kSplitSmem, split_done[p.split / 2]);
  if (err != cudaSuccess) return err;
  return cudaLaunchKernelEx(&cfg, kernel, ma, mb.m[0], static_cast<const LinArgs>(a));
}

// The rows operand of the forward and the input gradient.
bool map_rows(LinMapsB& mb, const LinPlan& p, int f16, RowsView x, long long cols, long long rows) {
  if (!p.pair) return map_k_major(&mb.m[0], f16, x.ptr, cols, rows, 1, x.ld, p.b_box);
  return map_k_major(&mb.m[0], f16, x.ptr, cols, rows, 1, x.ld, 128) && map_k_major(&mb.m[1], f16, x.ptr, cols, rows, 1, x.ld, 64);
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

namespace {

// Experts' maps (see expert_maps_kernel) into `emaps`, *out = emaps.
cudaError_t expert_maps(const LinearShape& p, const CUtensorMap& m0, const CUtensorMap& m1, void* maps, const CUtensorMap** out,
                        cudaStream_t stream) {
  CUtensorMap* emaps = static_cast<CUtensorMap*>(maps);
  *out = emaps;
  return launch_pdl(expert_maps_kernel, dim3(1), dim3(kLinMaxE), 0, stream, m0, m1, p.counts, p.E, p.align, p.rows, emaps);
}

// Forward and input gradient in the pair kernel: whether a tile's rows past its expert's end are to read as zeros
// instead of the next expert's rows.  The result is the same; zeros are not fetched and cost the tensor core less
// power, which a long run is bound by (32 experts of about 400 rows, back to back: forward 571 -> 563 us, both
// gradients 597 -> 581).  The maps' launch adds 2 us (and 3 on the host), so only where the product takes about 100 us
// at least and it is not the weights' way from HBM that does.
bool expert_rows_apart(const LinearShape& p, const LinPlan& pl) {
  return p.counts && pl.pair && p.rows >= 64LL * p.E && static_cast<double>(p.rows) * p.N * p.K >= 1e11;
}

}  // namespace

cudaError_t launch_linear(const LinearShape& p, RowsView x, const uint16_t* w, const float* bias, RowsView res, int act,
                          RowsView y, RowsView z, void* maps, uint32_t* status, cudaStream_t stream) {
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
  const LinPlan pl = lin_plan(p, a.i_ext, gated, p.rows, p.K, false, false);
  const int tile_i = lin_tile_i(pl, gated);
  a.n_it = (a.i_ext + tile_i - 1) / tile_i;
  CUtensorMap ma = {};
  LinMapsB mb = {};
  bool ok;
  if (gated) {
    // [E][N/2 / 8][2][8][K]: a copy takes, eight columns at a time, their gate rows and then their up rows
    const long long I = p.N / 2, K = p.K;
    const long long d[5] = {K, 8, 2, I / 8, a.E}, s[5] = {0, K, I * K, 8 * K, 2 * I * K};
    const int b[5] = {kLinSlab, 8, 2, pl.lanes / 16, 1};
    ok = lin_map(&ma, p.f16, w, 5, d, s, b);
  } else {
    ok = map_k_major(&ma, p.f16, w, p.K, p.N, a.E, p.K, pl.lanes);
  }
  if (!ok || !map_rows(mb, pl, p.f16, x, p.K, p.rows)) return cudaErrorInvalidValue;
  const CUtensorMap* emaps = nullptr;
  if (expert_rows_apart(p, pl)) {
    const cudaError_t err = expert_maps(p, mb.m[0], mb.m[1], maps, &emaps, stream);
    if (err != cudaSuccess) return err;
  }
  if (gated) return lin_launch<kLinFwdGated>(pl, ma, mb, emaps, a, stream);
  if (act == kActGelu) return lin_launch<kLinFwdGelu>(pl, ma, mb, emaps, a, stream);
  return lin_launch<kLinFwd>(pl, ma, mb, emaps, a, stream);
}

cudaError_t launch_linear_dx(const LinearShape& p, RowsView dz, const uint16_t* w, RowsView res, RowsView dx, void* maps,
                             uint32_t* status, cudaStream_t stream) {
  LinArgs a = lin_args(p, status);
  a.i_ext = p.K;
  a.q_ext = p.N;
  a.out = static_cast<uint16_t*>(dx.ptr);
  a.ldo = dx.ld;
  a.res = static_cast<const uint16_t*>(res.ptr);
  a.ldr = res.ld;
  const LinPlan pl = lin_plan(p, p.K, false, p.rows, p.N, false, false);
  const int tile_i = lin_tile_i(pl, false);
  a.n_it = (p.K + tile_i - 1) / tile_i;
  CUtensorMap ma = {};
  LinMapsB mb = {};
  a.a_blocks = pl.lanes / 64;
  if (!map_mn_major(&ma, p.f16, w, p.K, p.N, a.E, p.K, &a.a_blocks) ||
      !map_rows(mb, pl, p.f16, dz, p.N, p.rows))
    return cudaErrorInvalidValue;
  const CUtensorMap* emaps = nullptr;
  if (expert_rows_apart(p, pl)) {
    const cudaError_t err = expert_maps(p, mb.m[0], mb.m[1], maps, &emaps, stream);
    if (err != cudaSuccess) return err;
  }
  return lin_launch<kLinDx>(pl, ma, mb, emaps, a, stream);
}

cudaError_t launch_linear_dw(const LinearShape& p, RowsView dz, RowsView x, uint16_t* dw, void* maps, uint32_t* status,
                             cudaStream_t stream) {
  LinArgs a = lin_args(p, status);
  a.i_ext = p.K;
  a.j_ext = p.N;
  a.out = dw;
  a.ldo = p.K;
  const LinPlan pl = lin_plan(p, p.K, false, p.N, p.rows, true, p.counts != nullptr);
  const int tile_i = lin_tile_i(pl, false);
  a.n_it = (p.K + tile_i - 1) / tile_i;
  CUtensorMap ma = {};
  LinMapsB mb = {};
  a.a_blocks = pl.lanes / 64;
  // B in one copy where every tile (over a pair: every half) starts on a block
  const int cta_j = pl.pair ? pl.bj / 2 : pl.bj;
  a.b_blocks = cta_j % 64 == 0 && (!pl.pair || p.N % pl.bj == 0) ? cta_j / 64 : 0;
  if (!map_mn_major(&ma, p.f16, x.ptr, p.K, p.rows, 1, x.ld, &a.a_blocks) ||
      !map_mn_major(&mb.m[0], p.f16, dz.ptr, p.N, p.rows, 1, dz.ld, &a.b_blocks))
    return cudaErrorInvalidValue;
  const CUtensorMap* emaps = nullptr;
  if (p.counts) {
    const cudaError_t err = expert_maps(p, ma, mb.m[0], maps, &emaps, stream);
    if (err != cudaSuccess) return err;
  }
  return lin_launch<kLinDw>(pl, ma, mb, emaps, a, stream);
}

// ------------------------------------------------------------------------------------------
// dz = dy * act'(z), rounded to 16 bits since it is an operand of both products (at most 2^-8 of a value in bf16, 2^-11
// in fp16, where it is infinite past 65504), and the bias gradient's partial sums, of values before that rounding:
// thread = 8 columns, walking the rows s, s + S, ... of its expert (dense: all rows); CTA = 32 column groups x 8 rows.
// Memory bounds it where rows are many: SiLU, 16384 x 7168, 705 MB in 113 us (93% of a plain copy's rate; with four CTAs
// per SM instead of six 147, two rows of a thread at a time 152).  4096 x 2048 with the bias' second launch 15 us of
// 7.5 for the bytes, GELU 19, no activation 8.7 of 2.5: a thread has one row's loads on their way, and the launch.

namespace {

constexpr int kActRowLanes = 8;

__device__ __forceinline__ float silu_grad(float z, float& silu) {
  const float s = __fdividef(1.f, 1.f + __expf(-z));
  silu = z * s;
  return s * (1.f + z * (1.f - s));
}

// (v Phi(v))' = Phi(v) + v phi(v).  (With erfcf the pass is bound by its instructions: 25 us for 4096 x 2048 values.)
__device__ __forceinline__ float gelu_grad(float v) {
  float e;
  const float a = fabsf(v) > 30.f ? 30.f : fabsf(v), tail = normal_tail(a, e), vphi = a * 0.39894228040143268f * e;
  return v < 0.f ? tail - vphi : 1.f - tail + vphi;
}

// Eight values of z, kept in the rows' type or in 8 bits (codes in whole words; the same values as unpacked ones).
template <class T, bool Z8>
struct ZRows {
  const uint16_t* z;
  const uint8_t *q, *sf;
  long long ld, ldsf;
  int words;
  __device__ __forceinline__ auto get(long long row, int c) const {
    if constexpr (!Z8) {
      return load_pack<T>(z + row * ld + c);
    } else {
      Codes8<T> v;
      load_codes8<8>(q + row * ld + c, v.w, 8, words);
      v.set_scale(__ldg(sf + row * ldsf + c / kGroup8));
      return v;
    }
  }
};

// With a bias gradient.  (Z8 with more registers and fewer CTAs: 4096 x 4096 SwiGLU gradients 283 us of the whole call, with
// six CTAs 295.)
template <class T, bool Z8>
__global__ void __launch_bounds__(32 * kActRowLanes, Z8 ? 4 : 6)
    act_grad_kernel(const uint16_t* __restrict__ dy, long long lddy, const ZRows<T, Z8> z, int act,
                    const int32_t* __restrict__ counts, int E, int align, int rows, int N, uint16_t* __restrict__ dz,
                    long long lddz, float* __restrict__ part, int S, uint32_t* status) {
  __shared__ float red[kActRowLanes][2][32 * 8 + 8];
  const int lane = threadIdx.x & 31, rl = threadIdx.x >> 5;
  const int e = blockIdx.y;
  grid_dependency_wait();
  grid_launch_dependents();
  // (alone, this pass is what reports a segment that would leave the buffers)
  int cnt, seg;
  expert_segment(counts, e, align, rows, blockIdx.x == 0 && blockIdx.z == 0, seg, cnt, status);
  const bool gated = act == kActSwiglu;
  const int cols = gated ? N / 2 : N;
  const int c = (blockIdx.x * 32 + lane) * 8;
  float acc[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[0][i] = acc[1][i] = 0.f;
  if (c < cols) {
    for (int r = blockIdx.z * kActRowLanes + rl; r < cnt; r += S * kActRowLanes) {
      const long long row = seg + r;
      const Pack<T> g = load_pack<T>(dy + row * lddy + c);
      Pack<T> o, o2;
      if (gated) {
        const auto a = z.get(row, c), b = z.get(row, cols + c);
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
        store_pack<T>(dz + row * lddz + c, o);
        store_pack<T>(dz + row * lddz + cols + c, o2);
      } else if (act == kActNone) {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[0][i] += g.f(i);
      } else {
        const auto a = z.get(row, c);
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
            d = g.f(i) * gelu_grad(v);
          }
          acc[0][i] += d;
          o.set(i, d);
        }
        store_pack<T>(dz + row * lddz + c, o);
      }
    }
  }
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

// Where the experts' rows lie: expert e's segment starts at row[e] and has cnt[e] rows; end[e]: the chunks of `chunk` rows of
// experts 0 to e.  CTAs that walk over all experts' chunks share the work evenly, however the rows are spread.
struct LiveChunks {
  int row[kLinearMaxExperts], cnt[kLinearMaxExperts], end[kLinearMaxExperts];
};

// What the threads before this one of a CTA of 256 have in all, no more than `most` (sums: a warp's, one array per call).
__device__ __forceinline__ int sum_before(int mine, int most, int (&sums)[8]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int all = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, all, d);
    if (lane >= d) all = min(all + o, most);
  }
  int before = __shfl_up_sync(0xffffffffu, all, 1);
  if (lane == 0) before = 0;
  if (lane == 31) sums[warp] = all;
  __syncthreads();
  for (int w = 0; w < warp; ++w) before = min(before + sums[w], most);
  return before;
}

// Called by the whole CTA of 256 threads; where `report`, segments that would leave the buffers are recorded; they are cut in
// any case, as in expert_segment.
__device__ __forceinline__ void live_chunks(const int32_t* counts, int E, int align, int rows, int chunk, bool report,
                                            LiveChunks& s, uint32_t* status) {
  __shared__ int s_sums[2][8];
  const int q = (E + 255) / 256, e0 = threadIdx.x * q;
  int padded = 0, chunks = 0;
  for (int e = e0; e < min(e0 + q, E); ++e) {
    const int c = min(max(__ldg(counts + e), 0), rows);
    padded = min(padded + (c + align - 1) / align * align, rows);
  }
  int seg = sum_before(padded, rows, s_sums[0]);
  for (int e = e0; e < min(e0 + q, E); ++e) {
    const int all = __ldg(counts + e), cnt = min(max(all, 0), rows - seg);
    if (report && (all < 0 || all > cnt)) record_error(status, kDevErrIndex);
    s.row[e] = seg;
    s.cnt[e] = cnt;
    chunks += (cnt + chunk - 1) / chunk;
    seg = min(seg + (min(max(all, 0), rows) + align - 1) / align * align, rows);
  }
  int end = sum_before(chunks, 0x7fffffff, s_sums[1]);
  for (int e = e0; e < min(e0 + q, E); ++e) {
    end += (s.cnt[e] + chunk - 1) / chunk;
    s.end[e] = end;
  }
  __syncthreads();
}

// The same values without the bias gradient's sums: `lanes` threads to a row (fewer than a CTA's where rows are narrow), two
// rows of a thread on their way together (experts: CTAs walk over chunks of `chunk` rows, act_walk); blockIdx.x: which `lanes`
// groups of eight columns, so that neighbouring CTAs read one row.  Beside act_grad_kernel, with the dx product of K = 64 behind
// both: 4096 x 2048 SiLU 18.3 us of 21.1 and GELU 21.7 of 28.7, 128 x 4096 SwiGLU 11.0 of 13.1, 16384 x 7168 SiLU 163.2 of 162.2
// and GELU 180.6 of 185.7, 1000 x 4096 ReLU 14.9 of 14.5, 4096 rows of 8 experts, 2048 columns, all alike, GELU 26.4 of 24.2;
// from 8 bits, 6971 x 80 ReLU 4 of 17 and 7 experts of 288 columns 6 of 14 (a warp of act_grad_kernel takes 256 columns of one
// row).  With one row at a time and six CTAs per SM the SiLU case of 16384 x 7168 is 174, with CTAs of one column group side by
// side 163.6.
template <class T, bool Z8, bool EXPERTS>
__global__ void __launch_bounds__(256, 4)
    act_grad_rows_kernel(const uint16_t* __restrict__ dy, long long lddy, const ZRows<T, Z8> z, int act,
                         const int32_t* __restrict__ counts, int E, int align, int rows, int N, uint16_t* __restrict__ dz,
                         long long lddz, int lanes, int chunk, uint32_t* status) {
  constexpr int kAhead = 2;
  grid_dependency_wait();
  grid_launch_dependents();
  const bool gated = act == kActSwiglu;
  const int cols = gated ? N / 2 : N, per = 256 / lanes;
  const int c = (blockIdx.x * lanes + threadIdx.x % lanes) * 8, mine = threadIdx.x / lanes;
  // rows r and r + step, below past
  const auto two_rows = [&](long long r, long long step, long long past) {
    Pack<T> g[kAhead];
    decltype(z.get(0, 0)) a[kAhead], b[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const long long row = r + k * step < past ? r + k * step : r;
      g[k] = load_pack<T>(dy + row * lddy + c);
      a[k] = z.get(row, c);
      if (gated) b[k] = z.get(row, cols + c);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (r + k * step >= past) break;
      uint16_t* out = dz + (r + k * step) * lddz + c;
      Pack<T> o;
      if (gated) {
        Pack<T> o2;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float s;
          const float d = silu_grad(a[k].f(i), s);
          o.set(i, g[k].f(i) * b[k].f(i) * d);
          o2.set(i, g[k].f(i) * s);
        }
        store_pack<T>(out + cols, o2);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = a[k].f(i);
          float s;
          o.set(i, act == kActRelu   ? (v > 0.f ? g[k].f(i) : 0.f)
                   : act == kActSilu ? g[k].f(i) * silu_grad(v, s)
                                     : g[k].f(i) * gelu_grad(v));
        }
      }
      store_pack<T>(out, o);
    }
  };
  if constexpr (EXPERTS) {
    __shared__ LiveChunks live;
    live_chunks(counts, E, align, rows, chunk, blockIdx.x == 0 && blockIdx.z == 0, live, status);
    if (c >= cols) return;
    const int all = live.end[E - 1];
    int e = -1, end = 0, base = 0, past = 0;        // the expert, where its chunks end, its rows' place less its chunks', its end
    for (int j = blockIdx.z; j < all; j += gridDim.z) {
      if (j >= end) {                               // the first expert whose chunks reach past j
        int lo = e + 1, hi = E - 1;
        while (lo < hi) {
          const int mid = (lo + hi) / 2;
          if (j >= live.end[mid]) lo = mid + 1;
          else hi = mid;
        }
        e = lo;
        end = live.end[e];
        base = live.row[e] - (e ? live.end[e - 1] : 0) * chunk;
        past = live.row[e] + live.cnt[e];
      }
      const int first = base + j * chunk, last = min(past, first + chunk);
      for (int r = first + mine; r < last; r += kAhead * per) two_rows(r, per, last);
    }
  } else {
    if (c >= cols) return;
    const int step = gridDim.z * per;
    for (long long r = static_cast<long long>(blockIdx.z) * per + mine; r < rows; r += kAhead * step) two_rows(r, step, rows);
  }
}

// CTAs along the rows of act_grad_rows_kernel (`per` rows a CTA at a time, two such steps on their way together): 8 per SM at
// most, 16 where each has five steps or more all the same (16384 x 7168 SiLU 164.4 us with 8, 163.2 with 16, GELU 183.4 and
// 180.5; but 4096 x 2048, 1.7 steps with 16, GELU 21.5 and 22.4), and no more than give a CTA two steps while that leaves two
// CTAs per SM or so (1000 x 1408 SiLU 10.8 us with a step each, so 10.1; 2000 x 1408 ReLU 12.0, 11.3).
unsigned act_row_blocks(long long rows, int per, int nz) {
  const long long steps = (rows + per) / per, most = 16LL * num_sms() / nz;
  long long n = steps >= 5 * most ? most : steps < most / 2 ? steps : most / 2;
  if (n * nz >= 2 * num_sms() && n > (steps + 1) / 2) n = (steps + 1) / 2;
  return static_cast<unsigned>(n < 1 ? 1 : n);
}

// The same for experts with `rows` rows in all, and the rows of a chunk.  CTAs that each had an expert took as long as the
// largest one: 12288 rows of 256 experts, SwiGLU, 4096 columns, routed at random with uneven shares 145 us, so 103; all alike 114
// and 101; half of the rows one expert's, a quarter the next one's, .. 783 and 77.  Chunks of eight steps where a CTA has 16
// or more (12288 rows of 32 experts, GELU, 4096 columns 97 us, with two 104.6; but 4096 of 8, 2048 columns, three steps to a CTA,
// SwiGLU 22.4 with eight, 18.3 with two), and then 8 CTAs per SM, 4 otherwise (that case 19.0 with 8).
struct ActWalk {
  unsigned ctas;
  int chunk;
};
ActWalk act_walk(long long rows, int E, int per, int nz) {
  const long long most = 8LL * num_sms() / nz;
  if (rows >= 16 * most * per) return {static_cast<unsigned>(most < 1 ? 1 : most), 8 * per};
  long long n = rows / (2 * per) + E;               // (an expert's last chunk may be short)
  if (n > rows) n = rows;
  if (n > most / 2) n = most / 2;
  return {static_cast<unsigned>(n < 1 ? 1 : n), 2 * per};
}

__global__ void __launch_bounds__(256) bias_sum_kernel(const float* __restrict__ part, int S, int N, long long total,
                                                       float* __restrict__ db) {
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  grid_dependency_wait();
  grid_launch_dependents();
  if (i >= total) return;
  const long long e = i / N, c = i - e * N;
  float s = 0.f;
  for (int k = 0; k < S; ++k) s += part[(e * S + k) * N + c];
  db[i] = s;
}

}  // namespace

// Row slices per expert: about sixteen CTAs per SM in all, at most 64, none with less than 32 rows on average
// (with one slice the bias gradient is the slice's sum and needs no second launch).
int linear_bias_slices(int rows, int N, int E, int act) {
  const int cols = act == kActSwiglu ? N / 2 : N, n = E > 0 ? E : 1;
  const long long cta = static_cast<long long>((cols + 255) / 256) * n;
  long long s = (16LL * 152 + cta - 1) / cta;
  const long long most = static_cast<long long>(rows) / n / 32;
  if (s > most) s = most;
  return static_cast<int>(s < 1 ? 1 : (s > 64 ? 64 : s));
}

cudaError_t launch_act_grad(const LinearShape& p, RowsView dy, RowsView z, Rows8View z8, int act, RowsView dz, float* part,
                            float* db, uint32_t* status, cudaStream_t stream) {
  const int E = p.counts ? p.E : 1;
  // with the experts' padding known, the rows that are likely there; never more slices than the workspace holds
  const long long live = p.counts ? p.rows - static_cast<long long>(E) * (p.align - 1) : p.rows;
  const int most = linear_bias_slices(p.rows, p.N, E, act), few = linear_bias_slices(live > 0 ? static_cast<int>(live) : 0, p.N, E, act);
  const int S = few < most ? few : most;
  const int cols = act == kActSwiglu ? p.N / 2 : p.N;
  const dim3 grid((cols + 255) / 256, E, S);
  float* pp = S == 1 ? db : part;
  const auto run = [&](auto type, auto kept8) {
    using T = decltype(type);
    constexpr bool Z8 = decltype(kept8)::value;
    ZRows<T, Z8> zr{};
    zr.z = static_cast<const uint16_t*>(z.ptr);
    zr.ld = Z8 ? z8.ldq : z.ld;
    zr.q = z8.q;
    zr.sf = z8.sf;
    zr.ldsf = z8.lds;
    zr.words = codes_aligned(z8, p.rows, 8);
    if (!db) {
      // threads per row: the most (of 256, 128, ..) that leave at most an eighth of a row's last round idle
      const int packs = cols / 8;
      int lanes = 256;
      while (lanes > 8 && (packs + lanes - 1) / lanes * lanes - packs > packs / 8) lanes /= 2;
      const int nz = (packs + lanes - 1) / lanes, per = 256 / lanes;
      // (rows that are likely there: at least one in each aligned block of them)
      const ActWalk walk = p.counts ? act_walk(live > p.rows / p.align ? live : p.rows / p.align, E, per, nz)
                                    : ActWalk{act_row_blocks(p.rows, per, nz), 0};
      const auto kernel = p.counts ? act_grad_rows_kernel<T, Z8, true> : act_grad_rows_kernel<T, Z8, false>;
      return launch_pdl(kernel, dim3(static_cast<unsigned>(nz), 1, walk.ctas), dim3(256), 0, stream,
                        static_cast<const uint16_t*>(dy.ptr), dy.ld, zr, act, p.counts, E, p.align, p.rows, p.N,
                        static_cast<uint16_t*>(dz.ptr), dz.ld, lanes, walk.chunk, status);
    }
    return launch_pdl(act_grad_kernel<T, Z8>, grid, dim3(32 * kActRowLanes), 0, stream, static_cast<const uint16_t*>(dy.ptr),
                      dy.ld, zr, act, p.counts, E, p.align, p.rows, p.N, static_cast<uint16_t*>(dz.ptr), dz.ld, pp, S, status);
  };
  const cudaError_t err = z8.q ? (p.f16 ? run(F16Elem{}, std::true_type{}) : run(Bf16Elem{}, std::true_type{}))
                               : (p.f16 ? run(F16Elem{}, std::false_type{}) : run(Bf16Elem{}, std::false_type{}));
  if (err != cudaSuccess || !db || S == 1) return err;
  const long long total = static_cast<long long>(E) * p.N;
  return launch_pdl(bias_sum_kernel, dim3(static_cast<int>((total + 255) / 256)), dim3(256), 0, stream,
                    static_cast<const float*>(part), S, p.N, total, db);
}

}  // namespace moe
