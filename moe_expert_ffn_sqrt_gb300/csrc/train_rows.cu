// Rows sorted by expert and back, for training: the gather of token rows into the expert-contiguous
// layout, the weighted sum back, and both gradients, on bf16, fp16 or fp32 rows.
//
//   dispatch           x_perm[inv[t,k]] = x[t]
//   its gradient       dx[t] = sum_k dx_perm[inv[t,k]] (+ residual[t])            (sum_rows_kernel, no weights)
//   combine            out[t] = sum_k w[t,k] y[inv[t,k]] (+ residual[t])          (sum_rows_kernel)
//   its gradients      dy[inv[t,k]] = w[t,k] dout[t],  dw[t,k] = <dout[t], y[inv[t,k]]>
//
// Every kernel walks the tokens: a token's own row is read once and its K sorted rows are read or
// written once, so each byte crosses HBM once; memory bandwidth bounds all of them.  Sums are fp32 in
// slot order k = 0..K-1 (the order of moe_unpermute_reduce) and are rounded once on the store, and
// no atomics are used: equal inputs give equal bits.
//
// A row is walked in 16-byte packs where every row of the call starts on a 16-byte boundary and holds
// whole packs, else element by element.  A CTA of 256 threads takes one token, or several when a row
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

// Moves rows unchanged: V is the unit of the copy (16 bytes, or one element).
template <class V>
__global__ void __launch_bounds__(kRowThreads) scatter_rows_kernel(const V* __restrict__ x, long long ldx,
                                                                   const int32_t* __restrict__ inv, int T, int K, int n,
                                                                   int U, V* __restrict__ out, long long ldo, int lanes,
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
  // several units of the row on their way at a time: 16-byte ones two, single elements eight
  constexpr int G = sizeof(V) == 16 ? 2 : 8;
  for (int c = blockIdx.y * lanes + threadIdx.x % lanes; c < n; c += G * step) {
    V v[G];
#pragma unroll
    for (int i = 0; i < G; ++i)
      if (c + i * step < n) v[i] = x[t * ldx + c + i * step];
    for (int k = 0; k < K; ++k) {
      const int r = rows[k];
      if (r < 0) continue;
      V* o = out + r * ldo + c;
#pragma unroll
      for (int i = 0; i < G; ++i)
        if (c + i * step < n) o[i * step] = v[i];
    }
  }
}

template <class T, int N>
__global__ void __launch_bounds__(kRowThreads) sum_rows_kernel(const typename T::raw* __restrict__ y, long long ldy,
                                                               const int32_t* __restrict__ inv,
                                                               const float* __restrict__ w, const typename T::raw* res,
                                                               long long ldr, int T_, int K, int H, int U,
                                                               typename T::raw* out, long long ldo, int lanes,
                                                               uint32_t* status) {
  constexpr int kBatch = N == 1 ? 4 : 8;             // rows on their way at a time
  __shared__ SlotTable slots;
  const int tokens = kRowThreads / lanes, slot = threadIdx.x / lanes;
  const int t0 = blockIdx.x * tokens, t = t0 + slot;
  grid_dependency_wait();
  grid_launch_dependents();
  load_slots(slots, inv, w, t0, tokens, T_, K, U, status);
  if (t >= T_) return;
  const int* rows = slots.row + slot * K;
  const float* ws = slots.w + slot * K;
  // G packs per thread and pass, `step` apart: single elements eight, so that a slot's row is looked up once for them
  constexpr int G = N == 1 ? 8 : 1;
  const int step = gridDim.y * lanes * N;
  for (int c = (blockIdx.y * lanes + threadIdx.x % lanes) * N; c < H; c += G * step) {
    float acc[G][N];
    Pack<T, N> rv[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
#pragma unroll
      for (int i = 0; i < N; ++i) acc[g][i] = 0.f;
      if (res && c + g * step < H) rv[g] = load_pack<T, N>(res + t * ldr + c + g * step);
    }
    for (int k0 = 0; k0 < K; k0 += kBatch) {
      Pack<T, N> v[kBatch][G];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (k0 + k < K && rows[k0 + k] >= 0) {
          const typename T::raw* p = y + rows[k0 + k] * ldy + c;
#pragma unroll
          for (int g = 0; g < G; ++g)
            if (c + g * step < H) v[k][g] = load_pack<T, N>(p + g * step);
        }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (k0 + k < K && rows[k0 + k] >= 0) {
          const float wk = ws[k0 + k];
#pragma unroll
          for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = 0; i < N; ++i) acc[g][i] = fmaf(wk, v[k][g].f(i), acc[g][i]);
        }
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (c + g * step >= H) continue;
      Pack<T, N> o;
#pragma unroll
      for (int i = 0; i < N; ++i) o.set(i, res ? acc[g][i] + rv[g].f(i) : acc[g][i]);
      store_pack<T, N>(out + t * ldo + c + g * step, o);
    }
  }
}

// Slots [blockIdx.y * per, ...) of the CTA's tokens.  dout's row is read per slot (from L1 after the
// first); a slot's partial dot products meet in warp shuffles, then in shared memory, in a fixed order.
template <class T, int N>
__global__ void __launch_bounds__(kRowThreads) combine_grad_kernel(const typename T::raw* __restrict__ dout, long long ldd,
                                                                   const typename T::raw* y, long long ldy,
                                                                   const int32_t* __restrict__ inv,
                                                                   const float* __restrict__ w, int T_, int K, int H, int U,
                                                                   typename T::raw* dy, long long lddy, float* __restrict__ dw,
                                                                   int lanes, int per, uint32_t* status) {
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
      constexpr int G = N == 1 ? 8 : 1;                // packs per thread and pass, as in sum_rows_kernel
      const typename T::raw* dp = dout + t * ldd;
      const typename T::raw* yp = dw ? y + r * ldy : nullptr;
      typename T::raw* op = dy + r * lddy;
      const int step = lanes * N;
      for (int c = lane * N; c < H; c += G * step) {
        Pack<T, N> d[G], v[G];
#pragma unroll
        for (int g = 0; g < G; ++g)
          if (c + g * step < H) {
            d[g] = load_pack<T, N>(dp + c + g * step);
            if (dw) v[g] = load_pack<T, N>(yp + c + g * step);
          }
#pragma unroll
        for (int g = 0; g < G; ++g) {
          if (c + g * step >= H) continue;
          Pack<T, N> o;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            if (dw) dot = fmaf(d[g].f(i), v[g].f(i), dot);
            o.set(i, wk * d[g].f(i));
          }
          store_pack<T, N>(op + c + g * step, o);
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
// 1 KB of its row).  (Index arrays by launches of their own: 10 us for 384 pairs, 20 for 1020.)
// From 257 to 1024 pairs the same kernel, with more threads and no rows to move, only writes the index arrays
// (every CTA of a copy that fills the GPU working them out would take longer than a launch).
constexpr int kFewPairs = 256, kLayoutPairs = 1024;
constexpr int kFewHist = 32768;                     // entries of hist at most
constexpr int kFewUnits = 2;                        // copy units per lane and piece

inline int few_chunks(int pairs) { return (pairs + 31) / 32; }
// hist, then counts, segment starts and pairs' rows.
inline size_t few_smem(int pairs, int E) {
  return (static_cast<size_t>(few_chunks(pairs)) * E * 2 + 15) / 16 * 16 + (2 * static_cast<size_t>(E) + pairs) * 4;
}

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

// Calls f(element type, pack width) for the row type.
template <class F>
cudaError_t by_type(int dt, bool vec, F f) {
  switch (dt) {
    case kBf16: return vec ? f(Bf16Elem{}, std::integral_constant<int, 8>{}) : f(Bf16Elem{}, std::integral_constant<int, 1>{});
    case kF16: return vec ? f(F16Elem{}, std::integral_constant<int, 8>{}) : f(F16Elem{}, std::integral_constant<int, 1>{});
    default: return vec ? f(F32Elem{}, std::integral_constant<int, 4>{}) : f(F32Elem{}, std::integral_constant<int, 1>{});
  }
}
// Calls f(copy unit, units per 16 bytes or per element, as an element size) for rows that are only moved.
template <class F>
cudaError_t by_unit(int dt, bool vec, F f) {
  if (vec) return f(uint4{}, 16);
  return dt == kF32 ? f(uint32_t{}, 4) : f(uint16_t{}, 2);
}

// Threads per token for rows of n units (a power of two), and CTAs per row so that a call with few
// tokens still has two CTAs per SM.
// Single elements (vec false): sixteen per thread, or a CTA would have too little to do for its start.
int row_lanes(int n, bool vec) {
  if (!vec) n = (n + 15) / 16;
  int l = kMinLanes;
  while (l < kRowThreads && l < n) l *= 2;
  return l;
}
int row_cuts(int T, int lanes, int n) {
  const int tokens = kRowThreads / lanes, ctas = (T + tokens - 1) / tokens, most = (n + lanes - 1) / lanes;
  const int want = (2 * num_sms() + ctas - 1) / ctas;
  return want < most ? want : most;
}

}  // namespace

cudaError_t launch_scatter_rows(int dt, RowsView x, const int32_t* inv, int T, int K, int H, int U, RowsView out,
                                uint32_t* status, cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  return by_unit(dt, rows_vec(dt, H, {x, out}), [&](auto unit, int bytes) {
    using V = decltype(unit);
    const int es = static_cast<int>(dtype_bytes(dt)), n = static_cast<int>(static_cast<long long>(H) * es / bytes);
    const int lanes = row_lanes(n, bytes == 16), tokens = kRowThreads / lanes;
    const dim3 grid((T + tokens - 1) / tokens, row_cuts(T, lanes, n));
    return launch_pdl(scatter_rows_kernel<V>, grid, dim3(kRowThreads), 0, stream, static_cast<const V*>(x.ptr),
                      x.ld * es / bytes, inv, T, K, n, U, static_cast<V*>(out.ptr), out.ld * es / bytes, lanes, status);
  });
}

bool dispatch_layout_supported(int T, int K, int E) {
  const long long pairs = static_cast<long long>(T) * K;
  return pairs <= kLayoutPairs && E <= 1024 && static_cast<long long>(few_chunks(static_cast<int>(pairs))) * E <= kFewHist;
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
  const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
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
  return by_type(dt, rows_vec(dt, H, {y, res, out}), [&](auto e, auto width) {
    using E = decltype(e);
    constexpr int N = decltype(width)::value;
    const int n = (H + N - 1) / N, lanes = row_lanes(n, N > 1), tokens = kRowThreads / lanes;
    const dim3 grid((T + tokens - 1) / tokens, row_cuts(T, lanes, n));
    return launch_pdl(sum_rows_kernel<E, N>, grid, dim3(kRowThreads), 0, stream, static_cast<const typename E::raw*>(y.ptr),
                      y.ld, inv, w, static_cast<const typename E::raw*>(res.ptr), res.ld, T, K, H, U,
                      static_cast<typename E::raw*>(out.ptr), out.ld, lanes, status);
  });
}

cudaError_t launch_combine_grad(int dt, RowsView dout, RowsView y, const int32_t* inv, const float* w, int T, int K,
                                int H, int U, RowsView dy, float* dw, uint32_t* status, cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  return by_type(dt, rows_vec(dt, H, {dout, y, dy}), [&](auto e, auto width) {
    using E = decltype(e);
    constexpr int N = decltype(width)::value;
    const int lanes = row_lanes((H + N - 1) / N, N > 1), tokens = kRowThreads / lanes, ctas = (T + tokens - 1) / tokens;
    const int per = ctas >= 4 * num_sms() ? K : 1;   // few tokens: a CTA per slot
    return launch_pdl(combine_grad_kernel<E, N>, dim3(ctas, (K + per - 1) / per), dim3(kRowThreads), 0, stream,
                      static_cast<const typename E::raw*>(dout.ptr), dout.ld, static_cast<const typename E::raw*>(y.ptr), y.ld,
                      inv, w, T, K, H, U, static_cast<typename E::raw*>(dy.ptr), dy.ld, dw, lanes, per, status);
  });
}

}  // namespace moe
