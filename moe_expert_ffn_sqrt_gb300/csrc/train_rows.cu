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
  // two units of the row on their way at a time
  for (int c = blockIdx.y * lanes + threadIdx.x % lanes; c < n; c += 2 * step) {
    const bool two = c + step < n;
    const V v = x[t * ldx + c];
    const V u = two ? x[t * ldx + c + step] : V{};
    for (int k = 0; k < K; ++k) {
      const int r = rows[k];
      if (r < 0) continue;
      out[r * ldo + c] = v;
      if (two) out[r * ldo + c + step] = u;
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
  constexpr int kBatch = 8;                          // rows on their way at a time
  __shared__ SlotTable slots;
  const int tokens = kRowThreads / lanes, slot = threadIdx.x / lanes;
  const int t0 = blockIdx.x * tokens, t = t0 + slot;
  grid_dependency_wait();
  grid_launch_dependents();
  load_slots(slots, inv, w, t0, tokens, T_, K, U, status);
  if (t >= T_) return;
  const int* rows = slots.row + slot * K;
  const float* ws = slots.w + slot * K;
  for (int c = (blockIdx.y * lanes + threadIdx.x % lanes) * N; c < H; c += gridDim.y * lanes * N) {
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
    Pack<T, N> rv;
    if (res) rv = load_pack<T, N>(res + t * ldr + c);
    for (int k0 = 0; k0 < K; k0 += kBatch) {
      Pack<T, N> v[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (k0 + k < K && rows[k0 + k] >= 0) v[k] = load_pack<T, N>(y + rows[k0 + k] * ldy + c);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (k0 + k < K && rows[k0 + k] >= 0) {
          const float wk = ws[k0 + k];
#pragma unroll
          for (int i = 0; i < N; ++i) acc[i] = fmaf(wk, v[k].f(i), acc[i]);
        }
      }
    }
    Pack<T, N> o;
#pragma unroll
    for (int i = 0; i < N; ++i) o.set(i, res ? acc[i] + rv.f(i) : acc[i]);
    store_pack<T, N>(out + t * ldo + c, o);
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
      for (int c = lane * N; c < H; c += lanes * N) {
        const Pack<T, N> d = load_pack<T, N>(dout + t * ldd + c);
        if (dw) {
          const Pack<T, N> v = load_pack<T, N>(y + r * ldy + c);
#pragma unroll
          for (int i = 0; i < N; ++i) dot = fmaf(d.f(i), v.f(i), dot);
        }
        Pack<T, N> o;
#pragma unroll
        for (int i = 0; i < N; ++i) o.set(i, wk * d.f(i));
        store_pack<T, N>(dy + r * lddy + c, o);
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
// Few tokens: index arrays and rows in one launch.  Every CTA derives the whole layout (counts, segment
// starts, ranks) from the ids while its first piece of a row is on its way; the index arrays are written
// by the first CTAs, padding entries by all.  One warp per (pair, 1 KB of its row).
constexpr int kFewPairs = 256;
constexpr int kFewThreads = 256;
constexpr int kFewUnits = 2;                        // copy units per lane and piece

template <class V>
__global__ void __launch_bounds__(kFewThreads) dispatch_few_kernel(const PermuteArgs a, const V* __restrict__ x, long long ldx,
                                                                   int n, V* __restrict__ out, long long ldo) {
  extern __shared__ int32_t sh[];
  int32_t* cnt = sh;                                // [E]
  int32_t* seg = sh + a.E;                          // [E]
  __shared__ __align__(16) int32_t s_ids[kFewPairs];
  __shared__ int32_t s_pos[kFewPairs];
  __shared__ int32_t s_total;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int N = a.T * a.K;
  const int pieces = (n + 32 * kFewUnits - 1) / (32 * kFewUnits);
  const long long units = static_cast<long long>(N) * pieces;
  const long long u0 = static_cast<long long>(blockIdx.x) * (kFewThreads / 32) + warp;
  for (int i = tid; i < a.E; i += kFewThreads) cnt[i] = 0;
  grid_dependency_wait();
  grid_launch_dependents();
  // the first piece, and the ids
  V v[kFewUnits];
  if (u0 < units) {
    const int p = static_cast<int>(u0 / pieces), c = static_cast<int>(u0 % pieces) * 32 * kFewUnits + lane;
#pragma unroll
    for (int i = 0; i < kFewUnits; ++i)
      if (c + 32 * i < n) v[i] = x[p / a.K * ldx + c + 32 * i];
  }
  int e = -1;
  if (tid < N) {
    e = a.topk_ids[tid];
    if (e < 0 || e >= a.E) {
      if (blockIdx.x == 0) record_error(a.status, kDevErrIndex);
      e = -1;
    }
  }
  s_ids[tid] = e;
  __syncthreads();
  int rank = 0;
  if (e >= 0) {
    atomicAdd(&cnt[e], 1);
    const int4* ids4 = reinterpret_cast<const int4*>(s_ids);
    for (int j = 0; j < tid / 4; ++j) {
      const int4 q = ids4[j];
      rank += (q.x == e) + (q.y == e) + (q.z == e) + (q.w == e);
    }
    for (int j = tid & ~3; j < tid; ++j) rank += s_ids[j] == e;
  }
  __syncthreads();
  if (warp == 0) {                                  // exclusive scan of the aligned segment sizes
    const int per = (a.E + 31) / 32;
    int local = 0;
    for (int j = 0; j < per; ++j)
      if (lane * per + j < a.E) local += round_up_pow2(cnt[lane * per + j], a.align);
    int incl = local;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += o;
    }
    int run = incl - local;
    for (int j = 0; j < per; ++j) {
      const int i = lane * per + j;
      if (i < a.E) {
        seg[i] = run;
        run += round_up_pow2(cnt[i], a.align);
      }
    }
    if (lane == 31) s_total = incl;
  }
  __syncthreads();
  const int pos = e >= 0 ? seg[e] + rank : -1;
  s_pos[tid] = pos;
  if (blockIdx.x == 0) {
    if (e >= 0) {
      a.inv_perm[tid] = pos;
      a.sorted_ids[pos] = tid;
      a.expert_ids[pos] = e;
    }
    if (a.counts)
      for (int i = tid; i < a.E; i += kFewThreads) a.counts[i] = cnt[i];
    if (tid == 0) *a.m_sum = s_total;
  }
  __syncthreads();
  for (long long u = u0; u < units; u += static_cast<long long>(gridDim.x) * (kFewThreads / 32)) {
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
  for (int i = blockIdx.x * (kFewThreads / 32) + warp; i < a.E; i += gridDim.x * (kFewThreads / 32)) {
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
int row_lanes(int n) {
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
    const int lanes = row_lanes(n), tokens = kRowThreads / lanes;
    const dim3 grid((T + tokens - 1) / tokens, row_cuts(T, lanes, n));
    return launch_pdl(scatter_rows_kernel<V>, grid, dim3(kRowThreads), 0, stream, static_cast<const V*>(x.ptr),
                      x.ld * es / bytes, inv, T, K, n, U, static_cast<V*>(out.ptr), out.ld * es / bytes, lanes, status);
  });
}

bool dispatch_few_supported(int T, int K, int E) { return static_cast<long long>(T) * K <= kFewPairs && E <= 1024; }

cudaError_t launch_dispatch_few(int dt, const int32_t* topk_ids, RowsView x, int T, int H, int E, int K, int align, int U,
                                RowsView out, int32_t* sorted_ids, int32_t* expert_ids, int32_t* inv_perm, int32_t* m_sum,
                                int32_t* counts, uint32_t* status, cudaStream_t stream) {
  const PermuteArgs a{topk_ids, T, K, E, align, U, sorted_ids, expert_ids, inv_perm, m_sum, counts, status, 0};
  return by_unit(dt, rows_vec(dt, H, {x, out}), [&](auto unit, int bytes) {
    using V = decltype(unit);
    const int es = static_cast<int>(dtype_bytes(dt)), n = static_cast<int>(static_cast<long long>(H) * es / bytes);
    const long long units = static_cast<long long>(T) * K * ((n + 32 * kFewUnits - 1) / (32 * kFewUnits));
    const long long want = (units + kFewThreads / 32 - 1) / (kFewThreads / 32);
    const int grid = static_cast<int>(want < 1 ? 1 : want > 4 * num_sms() ? 4 * num_sms() : want);
    return launch_pdl(dispatch_few_kernel<V>, dim3(grid), dim3(kFewThreads), 2 * E * sizeof(int32_t), stream, a,
                      static_cast<const V*>(x.ptr), x.ld * es / bytes, n, static_cast<V*>(out.ptr), out.ld * es / bytes);
  });
}

cudaError_t launch_sum_rows(int dt, RowsView y, const int32_t* inv, const float* w, RowsView res, int T, int K, int H,
                            int U, RowsView out, uint32_t* status, cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  return by_type(dt, rows_vec(dt, H, {y, res, out}), [&](auto e, auto width) {
    using E = decltype(e);
    constexpr int N = decltype(width)::value;
    const int n = (H + N - 1) / N, lanes = row_lanes(n), tokens = kRowThreads / lanes;
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
    const int lanes = row_lanes((H + N - 1) / N), tokens = kRowThreads / lanes, ctas = (T + tokens - 1) / tokens;
    const int per = ctas >= 4 * num_sms() ? K : 1;   // few tokens: a CTA per slot
    return launch_pdl(combine_grad_kernel<E, N>, dim3(ctas, (K + per - 1) / per), dim3(kRowThreads), 0, stream,
                      static_cast<const typename E::raw*>(dout.ptr), dout.ld, static_cast<const typename E::raw*>(y.ptr), y.ld,
                      inv, w, T, K, H, U, static_cast<typename E::raw*>(dy.ptr), dy.ld, dw, lanes, per, status);
  });
}

}  // namespace moe
