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
// inv_perm entries of -1 are pairs that a full BatchedExperts slot dropped: they add nothing and get a
// zero weight gradient.  Any other entry outside [0, U) records MOE_ERR_DEVICE_INDEX and is skipped.
#include <initializer_list>
#include <type_traits>

#include "kernels.h"
#include "rows.cuh"

namespace moe {

namespace {

__device__ __forceinline__ bool row_ok(int r, int U, uint32_t* status) {
  if (r >= 0 && r < U) return true;
  if (r != -1) record_error(status, kDevErrIndex);
  return false;
}

template <class T, int N>
__global__ void __launch_bounds__(256) scatter_rows_kernel(const typename T::raw* __restrict__ x, long long ldx,
                                                           const int32_t* __restrict__ inv, int T_, int K, int H, int U,
                                                           typename T::raw* __restrict__ out, long long ldo,
                                                           uint32_t* status) {
  const int t = blockIdx.x;
  for (int c = (blockIdx.y * blockDim.x + threadIdx.x) * N; c < H; c += gridDim.y * blockDim.x * N) {
    const Pack<T, N> v = load_pack<T, N>(x + t * ldx + c);
    for (int k = 0; k < K; ++k) {
      const int r = __ldg(inv + static_cast<size_t>(t) * K + k);
      if (row_ok(r, U, status)) store_pack<T, N>(out + r * ldo + c, v);
    }
  }
}

template <class T, int N>
__global__ void __launch_bounds__(256) sum_rows_kernel(const typename T::raw* __restrict__ y, long long ldy,
                                                       const int32_t* __restrict__ inv, const float* __restrict__ w,
                                                       const typename T::raw* res, long long ldr, int K, int H, int U,
                                                       typename T::raw* out, long long ldo, uint32_t* status) {
  const int t = blockIdx.x;
  for (int c = (blockIdx.y * blockDim.x + threadIdx.x) * N; c < H; c += gridDim.y * blockDim.x * N) {
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
    for (int k = 0; k < K; ++k) {
      const int r = __ldg(inv + static_cast<size_t>(t) * K + k);
      if (!row_ok(r, U, status)) continue;
      const float wk = w ? __ldg(w + static_cast<size_t>(t) * K + k) : 1.f;
      const Pack<T, N> v = load_pack<T, N>(y + r * ldy + c);
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = fmaf(wk, v.f(i), acc[i]);
    }
    if (res) {
      const Pack<T, N> v = load_pack<T, N>(res + t * ldr + c);
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] += v.f(i);
    }
    Pack<T, N> o;
#pragma unroll
    for (int i = 0; i < N; ++i) o.set(i, acc[i]);
    store_pack<T, N>(out + t * ldo + c, o);
  }
}

template <class T, int N>
__global__ void __launch_bounds__(256) combine_grad_kernel(const typename T::raw* __restrict__ dout, long long ldd,
                                                           const typename T::raw* y, long long ldy,
                                                           const int32_t* __restrict__ inv, const float* __restrict__ w,
                                                           int K, int H, int U, typename T::raw* dy,
                                                           long long lddy, float* __restrict__ dw,
                                                           uint32_t* status) {
  __shared__ float part[8];
  const int t = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int k = 0; k < K; ++k) {
    const int r = __ldg(inv + static_cast<size_t>(t) * K + k);
    const bool ok = row_ok(r, U, status);
    float dot = 0.f;
    if (ok) {
      const float wk = w ? __ldg(w + static_cast<size_t>(t) * K + k) : 1.f;
      for (int c = threadIdx.x * N; c < H; c += blockDim.x * N) {
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
    for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
    if (lane == 0) part[warp] = dot;
    __syncthreads();
    if (threadIdx.x == 0) {
      float s = 0.f;
      for (int i = 0; i < static_cast<int>(blockDim.x) / 32; ++i) s += part[i];
      dw[static_cast<size_t>(t) * K + k] = s;
    }
    __syncthreads();
  }
}

inline bool vec_ok(const RowsView& m, int dt) {
  return !m.ptr || (reinterpret_cast<uintptr_t>(m.ptr) % 16 == 0 && m.ld * static_cast<long long>(dtype_bytes(dt)) % 16 == 0);
}

// Calls f(element type, pack width) for the row type: 16-byte packs when every row starts on a 16-byte
// boundary and holds whole packs, else single elements.
template <class F>
cudaError_t by_type(int dt, bool vec, F f) {
  switch (dt) {
    case kBf16: return vec ? f(Bf16Elem{}, std::integral_constant<int, 8>{}) : f(Bf16Elem{}, std::integral_constant<int, 1>{});
    case kF16: return vec ? f(F16Elem{}, std::integral_constant<int, 8>{}) : f(F16Elem{}, std::integral_constant<int, 1>{});
    default: return vec ? f(F32Elem{}, std::integral_constant<int, 4>{}) : f(F32Elem{}, std::integral_constant<int, 1>{});
  }
}

inline bool rows_vec(int dt, int H, std::initializer_list<RowsView> ms) {
  bool v = H * dtype_bytes(dt) % 16 == 0;
  for (const RowsView& m : ms) v = v && vec_ok(m, dt);
  return v;
}

}  // namespace

cudaError_t launch_scatter_rows(int dt, RowsView x, const int32_t* inv, int T, int K, int H, int U, RowsView out,
                                uint32_t* status, cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  return by_type(dt, rows_vec(dt, H, {x, out}), [&](auto e, auto n) {
    using E = decltype(e);
    constexpr int N = decltype(n)::value;
    scatter_rows_kernel<E, N><<<dim3(T, 1), 256, 0, stream>>>(static_cast<const typename E::raw*>(x.ptr), x.ld, inv, T, K,
                                                              H, U, static_cast<typename E::raw*>(out.ptr), out.ld, status);
    return cudaGetLastError();
  });
}

cudaError_t launch_sum_rows(int dt, RowsView y, const int32_t* inv, const float* w, RowsView res, int T, int K, int H,
                            int U, RowsView out, uint32_t* status, cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  return by_type(dt, rows_vec(dt, H, {y, res, out}), [&](auto e, auto n) {
    using E = decltype(e);
    constexpr int N = decltype(n)::value;
    sum_rows_kernel<E, N><<<dim3(T, 1), 256, 0, stream>>>(
        static_cast<const typename E::raw*>(y.ptr), y.ld, inv, w, static_cast<const typename E::raw*>(res.ptr), res.ld, K,
        H, U, static_cast<typename E::raw*>(out.ptr), out.ld, status);
    return cudaGetLastError();
  });
}

cudaError_t launch_combine_grad(int dt, RowsView dout, RowsView y, const int32_t* inv, const float* w, int T, int K,
                                int H, int U, RowsView dy, float* dw, uint32_t* status, cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  return by_type(dt, rows_vec(dt, H, {dout, y, dy}), [&](auto e, auto n) {
    using E = decltype(e);
    constexpr int N = decltype(n)::value;
    combine_grad_kernel<E, N><<<T, 256, 0, stream>>>(
        static_cast<const typename E::raw*>(dout.ptr), dout.ld, static_cast<const typename E::raw*>(y.ptr), y.ld, inv, w, K,
        H, U, static_cast<typename E::raw*>(dy.ptr), dy.ld, dw, status);
    return cudaGetLastError();
  });
}

}  // namespace moe
