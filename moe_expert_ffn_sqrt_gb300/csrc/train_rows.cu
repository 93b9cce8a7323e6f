// Rows sorted by expert and back, for training: the gather of token rows into the expert-contiguous
// layout, the weighted sum back, and both gradients, on bf16, fp16 or fp32 rows.
//
//   dispatch           x_perm[inv[t,k]] = x[t]
//   its gradient       dx[t] = sum_k dx_perm[inv[t,k]] (+ residual[t])            (sum_rows_kernel, no weights)
//   combine            out[t] = sum_k w[t,k] y[inv[t,k]] (+ residual[t])          (sum_rows_kernel)
//   its gradients      dy[inv[t,k]] = w[t,k] dout[t],  dw[t,k] = <dout[t], y[inv[t,k]]>
//
// Every kernel walks the tokens: a token's own row is read once and its K sorted rows are read or
// written once, so each byte crosses HBM once; memory bandwidth bounds all of them.  16384 tokens of 7168 bf16
// columns, K = 6, against a plain copy's rate: dispatch 267 us (92%), combine 242 (102%), combine's gradients 470
// (97%); 4096 tokens in fp32, dispatch's gradient 141 (99%).  Sums are fp32 in
// slot order k = 0..K-1 (the order of moe_unpermute_reduce) and are rounded once on the store, and
// no atomics are used: equal inputs give equal bits (dw's order goes by the rows' alignment).
//
// A row is walked in 16-byte packs where every row of the call starts on a 16-byte boundary and holds
// whole packs.  Else a thread's pack begins on a boundary of the row that is written, what it takes of other rows is
// shifted out of aligned words, and the row's two ends are written element by element.  A CTA of 256 threads takes one token, or several when a row
// has fewer packs than that (64-column rows one token per CTA leave 248 threads idle), and a call with
// few tokens cuts their rows (or their slots) over more CTAs.
//
// Every launch may begin while the stream's previous kernel ends (programmatic dependent launch): the
// kernels wait for it before they touch memory.
//
// inv_perm entries of -1 are pairs that a full BatchedExperts slot dropped: they add nothing and get a
// zero weight gradient.  Any other entry outside [0, U) records MOE_ERR_DEVICE_INDEX and is skipped.
#include <initializer_list>
#include <type_traits>

#include "kernels.h"
#include "permute_small.cuh"
#include "rows.cuh"

namespace moe {

namespace {

constexpr int kRowThreads = 256;
constexpr int kMaxSlots = 32;                       // K at most
constexpr int kMinLanes = 8;                        // threads per token at least
constexpr int kMaxTokens = kRowThreads / kMinLanes;

// The K sorted rows (and weights) of the CTA's tokens, checked once: -1 where there is none.
struct SlotTable {
  int row[kMaxTokens * kMaxSlots];
  float w[kMaxTokens * kMaxSlots];
};

__device__ __forceinline__ void load_slots(SlotTable& s, const int32_t* inv, const float* w, int t0, int tokens, int T, int K,
                                           int U, uint32_t* status) {
  for (int i = threadIdx.x; i < tokens * K; i += kRowThreads) {
    const long long p = static_cast<long long>(t0) * K + i;
    int r = -1;
    float wk = 1.f;
    if (p < static_cast<long long>(T) * K) {
      r = __ldg(inv + p);
      if (w) wk = __ldg(w + p);
      if (r < 0 || r >= U) {
        if (r != -1) record_error(status, kDevErrIndex);
        r = -1;
      }
    }
    s.row[i] = r;
    s.w[i] = wk;
  }
  __syncthreads();
}

// Moves rows of n 16-byte units unchanged.
__global__ void __launch_bounds__(kRowThreads) scatter_rows_kernel(const uint4* __restrict__ x, long long ldx,
                                                                   const int32_t* __restrict__ inv, int T, int K, int n,
                                                                   int U, uint4* __restrict__ out, long long ldo, int lanes,
                                                                   uint32_t* status) {
  __shared__ SlotTable slots;
  const int tokens = kRowThreads / lanes, slot = threadIdx.x / lanes;
  const int t0 = blockIdx.x * tokens, t = t0 + slot;
  grid_dependency_wait();
  grid_launch_dependents();
  load_slots(slots, inv, nullptr, t0, tokens, T, K, U, status);
  if (t >= T) return;
  const int* rows = slots.row + slot * K;
  const int step = gridDim.y * lanes;
  for (int c = blockIdx.y * lanes + threadIdx.x % lanes; c < n; c += 2 * step) {     // two units on their way
    uint4 v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (c + i * step < n) v[i] = x[t * ldx + c + i * step];
    for (int k = 0; k < K; ++k) {
      const int r = rows[k];
      if (r < 0) continue;
      uint4* o = out + r * ldo + c;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (c + i * step < n) o[i * step] = v[i];
    }
  }
}

// The packs of a row that is written: its columns c .. c + N-1 from a 16-byte boundary on, of which [from, to) exist.
template <class T>
struct RowParts {
  static constexpr int N = Pack<T>::N;
  int mis, H;                                       // columns of the first pack that are before the row
  __device__ __forceinline__ RowParts(const typename T::raw* row, int H_)
      : mis(static_cast<int>(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(typename T::raw))), H(H_) {}
  __device__ __forceinline__ int count() const { return (H + mis + N - 1) / N; }
  __device__ __forceinline__ int col(int j) const { return j * N - mis; }
  __device__ __forceinline__ int from(int c) const { return max(-c, 0); }
  __device__ __forceinline__ int to(int c) const { return min(H - c, N); }
};

// scatter_rows_kernel for rows of any width and alignment.  (2049 columns of 16 bits, 16384 tokens, K = 4: dispatch
// with rows moved element by element 91 us, so 72.)
template <class T>
__global__ void __launch_bounds__(kRowThreads) scatter_any_rows_kernel(const typename T::raw* __restrict__ x, long long ldx,
                                                                       const int32_t* __restrict__ inv, int T_, int K, int H,
                                                                       int U, typename T::raw* __restrict__ out,
                                                                       long long ldo, int lanes, uint32_t* status) {
  __shared__ SlotTable slots;
  const int tokens = kRowThreads / lanes, slot = threadIdx.x / lanes;
  const int t0 = blockIdx.x * tokens, t = t0 + slot;
  grid_dependency_wait();
  grid_launch_dependents();
  load_slots(slots, inv, nullptr, t0, tokens, T_, K, U, status);
  if (t >= T_) return;
  const int* rows = slots.row + slot * K;
  const typename T::raw *row = x + t * ldx, *end = x + (T_ - 1) * ldx + H;
  for (int k = 0; k < K; ++k) {
    if (rows[k] < 0) continue;
    typename T::raw* o = out + rows[k] * ldo;
    const RowParts<T> part(o, H);
    for (int j = blockIdx.y * lanes + threadIdx.x % lanes; j < part.count(); j += gridDim.y * lanes) {
      const int c = part.col(j);
      ShiftedPack<T> v;
      v.load(row + c, x, end);
      store_part<T>(o + c, v.get(), part.from(c), part.to(c));
    }
  }
}

// (Four CTAs per SM: with the registers for six the loads no longer go out together, 301 -> 452 us for 16384 x 7168,
// K = 6; unaligned without a limit 144 us instead of 109 for 16384 x 2049, K = 4, and element by element 133.)
// G packs of a token's row per thread and pass, 8 / G of its sorted rows at a time: with few rows per token more packs
// keep as many loads on their way.  (Four packs do not fit the registers: K = 1, 63 us with two, 73 with four.)
template <class T, bool ALIGNED, int G>
__global__ void __launch_bounds__(kRowThreads, 4)
    sum_rows_kernel(const typename T::raw* __restrict__ y, long long ldy, const int32_t* __restrict__ inv,
                    const float* __restrict__ w, const typename T::raw* res, long long ldr, int T_, int K, int H, int U,
                    typename T::raw* out, long long ldo, int lanes, uint32_t* status) {
  constexpr int N = Pack<T>::N;
  constexpr int kBatch = ALIGNED ? 8 / G : 2;        // rows on their way at a time
  __shared__ SlotTable slots;
  const int tokens = kRowThreads / lanes, slot = threadIdx.x / lanes;
  const int t0 = blockIdx.x * tokens, t = t0 + slot;
  grid_dependency_wait();
  grid_launch_dependents();
  load_slots(slots, inv, w, t0, tokens, T_, K, U, status);
  if (t >= T_) return;
  const int* rows = slots.row + slot * K;
  const float* ws = slots.w + slot * K;
  typename T::raw* o_row = out + t * ldo;
  if constexpr (ALIGNED) {
    const int step = gridDim.y * lanes * N;
    for (int c = (blockIdx.y * lanes + threadIdx.x % lanes) * N; c < H; c += G * step) {
      float acc[G][N];
      Pack<T> rv[G];
#pragma unroll
      for (int g = 0; g < G; ++g) {
#pragma unroll
        for (int i = 0; i < N; ++i) acc[g][i] = 0.f;
        if (res && c + g * step < H) rv[g] = load_pack<T>(res + t * ldr + c + g * step);
      }
      for (int k0 = 0; k0 < K; k0 += kBatch) {
        Pack<T> v[kBatch][G];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          if (k0 + k >= K || rows[k0 + k] < 0) continue;
          const typename T::raw* p = y + rows[k0 + k] * ldy + c;
#pragma unroll
          for (int g = 0; g < G; ++g)
            if (c + g * step < H) v[k][g] = load_pack<T>(p + g * step);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          if (k0 + k >= K || rows[k0 + k] < 0) continue;
          const float wk = ws[k0 + k];
#pragma unroll
          for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = 0; i < N; ++i) acc[g][i] = fmaf(wk, v[k][g].f(i), acc[g][i]);
        }
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (c + g * step >= H) continue;
        Pack<T> o;
#pragma unroll
        for (int i = 0; i < N; ++i) o.set(i, res ? acc[g][i] + rv[g].f(i) : acc[g][i]);
        store_pack<T>(o_row + c + g * step, o);
      }
    }
  } else {
    const typename T::raw* y_end = y + static_cast<long long>(U - 1) * ldy + H;
    const RowParts<T> part(o_row, H);
    for (int j = blockIdx.y * lanes + threadIdx.x % lanes; j < part.count(); j += gridDim.y * lanes) {
      const int c = part.col(j);
      float acc[N];
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = 0.f;
      ShiftedPack<T> rv;
      if (res) rv.load(res + t * ldr + c, res, res + static_cast<long long>(T_ - 1) * ldr + H);
      for (int k0 = 0; k0 < K; k0 += kBatch) {
        ShiftedPack<T> v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (k0 + k < K && rows[k0 + k] >= 0) v[k].load(y + rows[k0 + k] * ldy + c, y, y_end);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          if (k0 + k < K && rows[k0 + k] >= 0) {
            const float wk = ws[k0 + k];
            const Pack<T> p = v[k].get();
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = fmaf(wk, p.f(i), acc[i]);
          }
        }
      }
      Pack<T> o, r;
      if (res) r = rv.get();
#pragma unroll
      for (int i = 0; i < N; ++i) o.set(i, res ? acc[i] + r.f(i) : acc[i]);
      store_part<T>(o_row + c, o, part.from(c), part.to(c));
    }
  }
}

// Slots [blockIdx.y * per, ...) of the CTA's tokens.  dout's row is read per slot (from L1 after the
// first); a slot's partial dot products meet in warp shuffles, then in shared memory, in a fixed order.
// (What counts is threads: 16384 x 7168 rows of 16 bits, K = 6, with 8 CTAs per SM 470 us, with 6 505, with 5 546.)
template <class T, bool ALIGNED>
__global__ void __launch_bounds__(kRowThreads, ALIGNED && sizeof(typename T::raw) == 2 ? 8 : 4)
    combine_grad_kernel(const typename T::raw* __restrict__ dout, long long ldd, const typename T::raw* y, long long ldy,
                        const int32_t* __restrict__ inv, const float* __restrict__ w, int T_, int K, int H, int U,
                        typename T::raw* dy, long long lddy, float* __restrict__ dw, int lanes, int per, uint32_t* status) {
  constexpr int N = Pack<T>::N;
  __shared__ SlotTable slots;
  __shared__ float part[kMaxSlots][kRowThreads / 32];
  const int tokens = kRowThreads / lanes, slot = threadIdx.x / lanes, lane = threadIdx.x % lanes;
  const int t0 = blockIdx.x * tokens, t = t0 + slot;
  grid_dependency_wait();
  grid_launch_dependents();
  load_slots(slots, inv, w, t0, tokens, T_, K, U, status);
  const int k_end = min(K, static_cast<int>(blockIdx.y + 1) * per);
  for (int k = blockIdx.y * per; k < k_end; ++k) {
    const int r = t < T_ ? slots.row[slot * K + k] : -1;
    float dot = 0.f;
    if (r >= 0) {
      const float wk = slots.w[slot * K + k];
      const typename T::raw* dp = dout + t * ldd;
      const typename T::raw* yp = dw ? y + r * ldy : nullptr;
      typename T::raw* op = dy + r * lddy;
      if constexpr (ALIGNED) {
        for (int c = lane * N; c < H; c += lanes * N) {
          const Pack<T> d = load_pack<T>(dp + c);
          Pack<T> v, o;
          if (dw) v = load_pack<T>(yp + c);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            if (dw) dot = fmaf(d.f(i), v.f(i), dot);
            o.set(i, wk * d.f(i));
          }
          store_pack<T>(op + c, o);
        }
      } else {
        const typename T::raw* d_end = dout + static_cast<long long>(T_ - 1) * ldd + H;
        const typename T::raw* y_end = y + static_cast<long long>(U - 1) * ldy + H;
        const RowParts<T> rp(op, H);
        for (int j = lane; j < rp.count(); j += lanes) {
          const int c = rp.col(j), from = rp.from(c), to = rp.to(c);
          ShiftedPack<T> ds, vs;
          ds.load(dp + c, dout, d_end);
          if (dw) vs.load(yp + c, y, y_end);
          const Pack<T> d = ds.get();
          Pack<T> v, o;
          if (dw) v = vs.get();
#pragma unroll
          for (int i = 0; i < N; ++i) {
            if (dw && i >= from && i < to) dot = fmaf(d.f(i), v.f(i), dot);
            o.set(i, wk * d.f(i));
          }
          store_part<T>(op + c, o, from, to);
        }
      }
    }
    if (!dw) continue;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
      if (off < lanes) dot += __shfl_xor_sync(0xffffffffu, dot, off);
    if (lanes <= 32) {
      if (lane == 0 && t < T_) dw[static_cast<size_t>(t) * K + k] = dot;
    } else if (threadIdx.x % 32 == 0) {
      part[k][threadIdx.x / 32] = dot;
    }
  }
  if (!dw || lanes <= 32) return;
  __syncthreads();
  const int warps = lanes / 32;
  for (int i = threadIdx.x; i < tokens * (k_end - static_cast<int>(blockIdx.y) * per); i += kRowThreads) {
    const int s = i % tokens, k = blockIdx.y * per + i / tokens;
    if (t0 + s >= T_) continue;
    float v = 0.f;
    for (int j = 0; j < warps; ++j) v += part[k][s * warps + j];
    dw[static_cast<size_t>(t0 + s) * K + k] = v;
  }
}

// ------------------------------------------------------------------------------------------
// Few tokens: index arrays and rows in one launch.  Every CTA derives the whole layout from the ids while its first
// piece of a row is on its way: each 32 pairs' experts are counted by a warp's matches (hist[chunk][expert], 16
// bits), then summed over the chunks before, so that a pair's rank is its chunk's sum and its place among the
// chunk's matches.  The index arrays are written by the first CTA, padding entries by all.  One warp per (pair,
// 1 KB of its row).  8 tokens of 7168 bf16 columns, 256 experts, K = 6: 3.0 us, 42 tokens 4.1.  (Index arrays by
// launches of their own: 10 us for 384 pairs, 20 for 1020.)
// From 257 to 2048 pairs the same kernel, with more threads and no rows to move, only writes the index arrays
// (every CTA of a copy that fills the GPU working them out would take longer than a launch).  Of 64 experts, with the
// copy of 64 columns: 1200 pairs 7.1 us, by the layer's own permute 8.6, 2048 pairs 8.6 and 8.7, 4096 12.9 and 8.8.
constexpr int kFewPairs = 256, kLayoutPairs = 2048;
constexpr int kFewHist = 32768;                     // entries of hist at most
constexpr int kFewUnits = 2;                        // copy units per lane and piece

inline int few_chunks(int pairs) { return (pairs + 31) / 32; }
// hist, then counts, segment starts and pairs' rows.
inline size_t few_smem(int pairs, int E) {
  return (static_cast<size_t>(few_chunks(pairs)) * E * 2 + 15) / 16 * 16 + (2 * static_cast<size_t>(E) + pairs) * 4;
}
constexpr int kFewExperts = 1024;
constexpr int kLayoutSmem = kFewHist * 2 + (2 * kFewExperts + kLayoutPairs) * 4;    // few_smem at most (80 KB)

template <class V, int kFewThreads>
__global__ void __launch_bounds__(kFewThreads) dispatch_few_kernel(const PermuteArgs a, const V* __restrict__ x, long long ldx,
                                                                   int n, V* __restrict__ out, long long ldo) {
  constexpr int kFewWarps = kFewThreads / 32;
  extern __shared__ __align__(16) uint16_t hist[];  // [chunks][E]
  const int N = a.T * a.K, E = a.E, chunks = (N + 31) / 32;
  int32_t* cnt = reinterpret_cast<int32_t*>(hist + (static_cast<size_t>(chunks) * E + 7) / 8 * 8);   // [E]
  int32_t* seg = cnt + E;                           // [E]
  int32_t* s_pos = seg + E;                         // [N]
  __shared__ int32_t s_scan[kFewWarps];
  __shared__ int32_t s_total;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int pieces = (n + 32 * kFewUnits - 1) / (32 * kFewUnits);
  const long long units = static_cast<long long>(N) * pieces;
  const long long u0 = static_cast<long long>(blockIdx.x) * kFewWarps + warp;
  for (int i = tid; i < (chunks * E + 7) / 8; i += kFewThreads) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
  grid_dependency_wait();
  grid_launch_dependents();
  // the first piece of a row
  V v[kFewUnits];
  if (u0 < units) {
    const int p = static_cast<int>(u0 / pieces), c = static_cast<int>(u0 % pieces) * 32 * kFewUnits + lane;
#pragma unroll
    for (int i = 0; i < kFewUnits; ++i)
      if (c + 32 * i < n) v[i] = x[p / a.K * ldx + c + 32 * i];
  }
  __syncthreads();
  // 1. matches within each chunk
  for (int ch = warp; ch < chunks; ch += kFewWarps) {
    const int p = ch * 32 + lane;
    int e = p < N ? __ldg(a.topk_ids + p) : -1;
    if (p < N && (e < 0 || e >= E)) {
      if (blockIdx.x == 0) record_error(a.status, kDevErrIndex);
      e = -1;
    }
    const unsigned peers = __match_any_sync(0xffffffffu, e >= 0 ? e : -1 - lane);
    const int rank = __popc(peers & ((1u << lane) - 1u));
    if (e >= 0 && rank == 0) hist[ch * E + e] = static_cast<uint16_t>(__popc(peers));
    if (p < N) s_pos[p] = e < 0 ? -1 : e << 5 | rank;
  }
  __syncthreads();
  // 2. per expert: sums over the chunks before, counts; then the scan of the aligned segment sizes (expert order:
  // thread t has experts t * per ..)
  const int per = (E + kFewThreads - 1) / kFewThreads;
  int local = 0;
  for (int j = 0; j < per; ++j) {
    const int e = tid * per + j;
    if (e >= E) break;
    int run = 0;
    for (int c8 = 0; c8 < chunks; c8 += 8) {        // eight reads before the first write
      int h[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = c8 + i < chunks ? hist[(c8 + i) * E + e] : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (c8 + i < chunks) hist[(c8 + i) * E + e] = static_cast<uint16_t>(run);
        run += h[i];
      }
    }
    cnt[e] = run;
    local += round_up_pow2(run, a.align);
  }
  int incl = local;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < warp; ++w) before += s_scan[w];
  int run = before + incl - local;
  for (int j = 0; j < per; ++j) {
    const int e = tid * per + j;
    if (e >= E) break;
    seg[e] = run;
    run += round_up_pow2(cnt[e], a.align);
  }
  if (tid == kFewThreads - 1) s_total = before + incl;
  __syncthreads();
  // 3. rows of the pairs
  for (int p = tid; p < N; p += kFewThreads) {
    const int m = s_pos[p];
    if (m < 0) continue;
    const int e = m >> 5, pos = seg[e] + hist[(p >> 5) * E + e] + (m & 31);
    s_pos[p] = pos;
    if (blockIdx.x == 0) {
      a.inv_perm[p] = pos;
      a.sorted_ids[pos] = p;
      a.expert_ids[pos] = e;
    }
  }
  if (blockIdx.x == 0) {
    if (a.counts)
      for (int i = tid; i < E; i += kFewThreads) a.counts[i] = cnt[i];
    if (tid == 0) *a.m_sum = s_total;
  }
  __syncthreads();
  for (long long u = u0; u < units; u += static_cast<long long>(gridDim.x) * kFewWarps) {
    const int p = static_cast<int>(u / pieces), c = static_cast<int>(u % pieces) * 32 * kFewUnits + lane;
    const int r = s_pos[p];
#pragma unroll
    for (int i = 0; i < kFewUnits; ++i) {
      if (c + 32 * i >= n) continue;
      if (u != u0) v[i] = x[p / a.K * ldx + c + 32 * i];
      if (r >= 0) out[r * ldo + c + 32 * i] = v[i];
    }
  }
  // padding entries: of the segments, then the rows [M_sum, U)
  for (int i = blockIdx.x * kFewWarps + warp; i < E; i += gridDim.x * kFewWarps) {
    const int padded = round_up_pow2(cnt[i], a.align);
    for (int r = cnt[i] + lane; r < padded; r += 32) {
      a.sorted_ids[seg[i] + r] = N;
      a.expert_ids[seg[i] + r] = -1;
    }
  }
  for (int r = s_total + blockIdx.x * kFewThreads + tid; r < a.U; r += gridDim.x * kFewThreads) {
    a.sorted_ids[r] = N;
    a.expert_ids[r] = -1;
  }
}

// ------------------------------------------------------------------------------------------

inline bool vec_ok(const RowsView& m, int dt) {
  return !m.ptr || (reinterpret_cast<uintptr_t>(m.ptr) % 16 == 0 && m.ld * static_cast<long long>(dtype_bytes(dt)) % 16 == 0);
}
inline bool rows_vec(int dt, int H, std::initializer_list<RowsView> ms) {
  bool v = H * static_cast<long long>(dtype_bytes(dt)) % 16 == 0;
  for (const RowsView& m : ms) v = v && vec_ok(m, dt);
  return v;
}

// Calls f(element type, whether rows are whole aligned packs) for the row type.
template <class F>
cudaError_t by_type(int dt, bool vec, F f) {
  switch (dt) {
    case kBf16: return vec ? f(Bf16Elem{}, std::true_type{}) : f(Bf16Elem{}, std::false_type{});
    case kF16: return vec ? f(F16Elem{}, std::true_type{}) : f(F16Elem{}, std::false_type{});
    default: return vec ? f(F32Elem{}, std::true_type{}) : f(F32Elem{}, std::false_type{});
  }
}
// Calls f(copy unit, units per 16 bytes or per element, as an element size) for rows that are only moved.
template <class F>
cudaError_t by_unit(int dt, bool vec, F f) {
  if (vec) return f(uint4{}, 16);
  return dt == kF32 ? f(uint32_t{}, 4) : f(uint16_t{}, 2);
}

// 16-byte packs of a row (one more where it need not start on a boundary).
int row_packs(int dt, int H, bool vec) {
  const int N = static_cast<int>(16 / dtype_bytes(dt));
  return (H + N - 1) / N + (vec ? 0 : 1);
}
// Threads per token for rows of n packs: the largest power of two that leaves each `packs` of them, as far as that
// goes.  Several passes per thread hide what a CTA needs before its first one: sums of 4 rows of 2048 16-bit columns
// for 16384 tokens, a pack at a time: 4 passes 73 us, one 87; rows just past a power of two (2064 columns) 79 instead of 105.
int row_lanes(int n, int packs) {
  int l = kMinLanes;
  while (2 * l <= kRowThreads && 2 * l * packs <= n) l *= 2;
  return l;
}
// CTAs per row, so that a call with few tokens still has two CTAs per SM.
int row_cuts(int T, int lanes, int n) {
  const int tokens = kRowThreads / lanes, ctas = (T + tokens - 1) / tokens, most = (n + lanes - 1) / lanes;
  const int want = (2 * num_sms() + ctas - 1) / ctas;
  return want < most ? want : most;
}

}  // namespace

cudaError_t launch_scatter_rows(int dt, RowsView x, const int32_t* inv, int T, int K, int H, int U, RowsView out,
                                uint32_t* status, cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  const bool vec = rows_vec(dt, H, {x, out});
  const int n = row_packs(dt, H, vec), lanes = row_lanes(n, 2), tokens = kRowThreads / lanes;
  const dim3 grid((T + tokens - 1) / tokens, row_cuts(T, lanes, n));
  if (vec) {
    const int es = static_cast<int>(dtype_bytes(dt));
    return launch_pdl(scatter_rows_kernel, grid, dim3(kRowThreads), 0, stream, static_cast<const uint4*>(x.ptr), x.ld * es / 16,
                      inv, T, K, n, U, static_cast<uint4*>(out.ptr), out.ld * es / 16, lanes, status);
  }
  const auto any = [&](auto e) {       // the bits are moved, whatever the type of that size
    using E = decltype(e);
    return launch_pdl(scatter_any_rows_kernel<E>, grid, dim3(kRowThreads), 0, stream,
                      static_cast<const typename E::raw*>(x.ptr), x.ld, inv, T, K, H, U,
                      static_cast<typename E::raw*>(out.ptr), out.ld, lanes, status);
  };
  return dt == kF32 ? any(F32Elem{}) : any(Bf16Elem{});
}

bool dispatch_layout_supported(int T, int K, int E) {
  const long long pairs = static_cast<long long>(T) * K;
  return pairs <= kLayoutPairs && E <= kFewExperts && static_cast<long long>(few_chunks(static_cast<int>(pairs))) * E <= kFewHist;
}

cudaError_t launch_dispatch_layout(int dt, const int32_t* topk_ids, RowsView x, int T, int H, int E, int K, int align, int U,
                                   RowsView out, int32_t* sorted_ids, int32_t* expert_ids, int32_t* inv_perm, int32_t* m_sum,
                                   int32_t* counts, uint32_t* status, cudaStream_t stream) {
  const PermuteArgs a{topk_ids, T, K, E, align, U, sorted_ids, expert_ids, inv_perm, m_sum, counts, status, 0};
  const size_t smem = few_smem(T * K, E);
  if (T * K <= kFewPairs) {
    return by_unit(dt, rows_vec(dt, H, {x, out}), [&](auto unit, int bytes) {
      using V = decltype(unit);
      const int es = static_cast<int>(dtype_bytes(dt)), n = static_cast<int>(static_cast<long long>(H) * es / bytes);
      const long long units = static_cast<long long>(T) * K * ((n + 32 * kFewUnits - 1) / (32 * kFewUnits));
      const long long want = (units + 7) / 8;
      const int grid = static_cast<int>(want < 1 ? 1 : want > 4 * num_sms() ? 4 * num_sms() : want);
      return launch_pdl(dispatch_few_kernel<V, 256>, dim3(grid), dim3(256), smem, stream, a, static_cast<const V*>(x.ptr),
                        x.ld * es / bytes, n, static_cast<V*>(out.ptr), out.ld * es / bytes);
    });
  }
  const auto kernel = dispatch_few_kernel<uint4, 1024>;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t err = allow_smem(reinterpret_cast<const void*>(kernel), kLayoutSmem, done);
  if (err != cudaSuccess) return err;
  const int grid = U > 4096 ? 16 : 4;                // shares of the padding entries
  const cudaError_t err2 = launch_pdl(kernel, dim3(grid), dim3(1024), smem, stream, a, static_cast<const uint4*>(nullptr), 0, 0,
                                      static_cast<uint4*>(nullptr), 0);
  if (err2 != cudaSuccess) return err2;
  return launch_scatter_rows(dt, x, inv_perm, T, K, H, U, out, status, stream);
}

cudaError_t launch_sum_rows(int dt, RowsView y, const int32_t* inv, const float* w, RowsView res, int T, int K, int H,
                            int U, RowsView out, uint32_t* status, cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  const bool vec = rows_vec(dt, H, {y, res, out});
  const int n = row_packs(dt, H, vec);
  int lanes = row_lanes(n, 4);
  // few tokens: more threads for each before their rows are cut
  while (lanes < n && lanes < kRowThreads && 2LL * T * lanes < 3LL * kRowThreads * num_sms()) lanes *= 2;
  const int tokens = kRowThreads / lanes;
  const dim3 grid((T + tokens - 1) / tokens, row_cuts(T, lanes, n));
  return by_type(dt, vec, [&](auto e, auto aligned) {
    using E = decltype(e);
    constexpr bool kVec = decltype(aligned)::value;
    // two packs at a time for up to four rows (16384 x 4096 bf16 with a residual, K = 1: 103 -> 84 us,
    // K = 4: 141 -> 128; K = 6 has rows enough), where a thread has two (72 columns, K = 4: 4.3 us, with two 5.3)
    const auto kernel = kVec && K <= 4 && n >= 2 * lanes ? sum_rows_kernel<E, kVec, kVec ? 2 : 1> : sum_rows_kernel<E, kVec, 1>;
    return launch_pdl(kernel, grid, dim3(kRowThreads), 0, stream, static_cast<const typename E::raw*>(y.ptr),
                      y.ld, inv, w, static_cast<const typename E::raw*>(res.ptr), res.ld, T, K, H, U,
                      static_cast<typename E::raw*>(out.ptr), out.ld, lanes, status);
  });
}

cudaError_t launch_combine_grad(int dt, RowsView dout, RowsView y, const int32_t* inv, const float* w, int T, int K,
                                int H, int U, RowsView dy, float* dw, uint32_t* status, cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  const bool vec = rows_vec(dt, H, {dout, y, dy});
  // (a pass more would take dout's rows out of L1 before the last slot: 16384 x 7168, K = 6, with 7 for each thread
  // 558 us instead of 470)
  const int lanes = row_lanes(row_packs(dt, H, vec), 3), tokens = kRowThreads / lanes, ctas = (T + tokens - 1) / tokens;
  const int per = ctas >= 4 * num_sms() ? K : 1;     // few tokens: a CTA per slot
  return by_type(dt, vec, [&](auto e, auto aligned) {
    using E = decltype(e);
    return launch_pdl(combine_grad_kernel<E, decltype(aligned)::value>, dim3(ctas, (K + per - 1) / per), dim3(kRowThreads), 0, stream,
                      static_cast<const typename E::raw*>(dout.ptr), dout.ld, static_cast<const typename E::raw*>(y.ptr), y.ld,
                      inv, w, T, K, H, U, static_cast<typename E::raw*>(dy.ptr), dy.ld, dw, lanes, per, status);
  });
}

}  // namespace moe
