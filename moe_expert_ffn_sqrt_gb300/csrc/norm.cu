// Root-mean-square norm of rows, with the residual's addition before it and 8-bit output rows, and its gradients.
//
//   s = x + residual (rounded to the rows' type, as it is stored: forward and backward then see the same stream)
//   r = (mean(s^2) + eps)^(-1/2);   y_i = s_i r w_i
//   g_i = dy_i w_i:   dx_i = r g_i - s_i r^3 mean(s g) + dsum_i;   dw_i = sum over rows of dy_i s_i r
// Both are taken in fp32; each output is rounded once, the 8-bit rows (rows8.cuh) from the fp32 y.  One pass over a
// row gives both of the backward's sums (s^2 and s g), so nothing but s is kept from the forward.
#include "rows8.cuh"

namespace moe {

namespace {

constexpr int kNormThreads = 256;

struct NormArgs {
  const void *x, *res;
  void *sum, *y;
  const float* w;
  uint8_t *q, *sf;
  long long ldx, ldr, lds, ldy, ldq, ldsf;
  float eps;
  int T, H;
  int q_words;                // codes in whole words
};

// Sum over the block of K values per thread, in a fixed order; every thread gets it.
template <int K>
__device__ __forceinline__ void block_sum(float (&v)[K], float (*sh)[K]) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], d);
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) sh[warp][k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = lane < warps ? sh[lane][k] : 0.f;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], d);
}

// A matrix of rows of H columns.  AL: every row on a 16-byte boundary and H in whole packs.
template <class T>
struct Mat {
  using raw = typename T::raw;
  raw *lo, *hi;               // its first element and the end of its last row
  long long ld;
  __device__ __forceinline__ Mat(const void* p, long long l, int rows, int H)
      : lo(static_cast<raw*>(const_cast<void*>(p))), hi(lo + (rows - 1) * l + H), ld(l) {}
  // columns [c, c + N) of a row; zeros past its end
  template <bool AL>
  __device__ __forceinline__ Pack<T> get(long long row, int c, int H) const {
    const raw* p = lo + row * ld + c;
    if constexpr (AL) {
      return load_pack<T>(p);
    } else {
      ShiftedPack<T> s;
      s.load(p, lo, hi);
      Pack<T> v = s.get();
#pragma unroll
      for (int i = 0; i < Pack<T>::N; ++i)
        if (c + i >= H) v.v[i] = T::from_f(0.f);
      return v;
    }
  }
  template <bool AL>
  __device__ __forceinline__ void put(long long row, int c, int H, const Pack<T>& v) const {
    raw* p = lo + row * ld + c;
    if constexpr (AL) {
      store_pack<T>(p, v);
    } else {
#pragma unroll
      for (int i = 0; i < Pack<T>::N; ++i)
        if (c + i < H) p[i] = v.v[i];
    }
  }
};

// One CTA per row.
template <class T, bool AL>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const NormArgs a) {
  constexpr int N = Pack<T>::N;
  __shared__ float sh[32][1];
  grid_dependency_wait();
  grid_launch_dependents();
  const long long t = blockIdx.x;
  const int H = a.H;
  const Mat<T> x(a.x, a.ldx, a.T, H), r(a.res, a.ldr, a.T, H), s(a.sum, a.lds, a.T, H), y(a.y, a.ldy, a.T, H);
  float ss[1] = {0.f};
  for (int c = threadIdx.x * N; c < H; c += kNormThreads * N) {
    Pack<T> p = x.template get<AL>(t, c, H);
    if (a.res) {
      const Pack<T> q = r.template get<AL>(t, c, H);
#pragma unroll
      for (int i = 0; i < N; ++i) p.set(i, p.f(i) + q.f(i));
    }
    if (a.sum) s.template put<AL>(t, c, H, p);
#pragma unroll
    for (int i = 0; i < N; ++i) ss[0] = fmaf(p.f(i), p.f(i), ss[0]);
  }
  block_sum<1>(ss, sh);
  const float rs = rsqrtf(ss[0] / H + a.eps);
  const int whole = groups8(H) * kGroup8;      // (a group's lanes meet in group_max)
  for (int c0 = 0; c0 < whole; c0 += kNormThreads * N) {
    const int c = c0 + threadIdx.x * N;
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
    if (c < H) {
      Pack<T> p;
      if (a.sum) {
        p = s.template get<AL>(t, c, H);
      } else {
        p = x.template get<AL>(t, c, H);
        if (a.res) {
          const Pack<T> q = r.template get<AL>(t, c, H);
#pragma unroll
          for (int i = 0; i < N; ++i) p.set(i, p.f(i) + q.f(i));
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (AL || c + i < H) v[i] = p.f(i) * rs * __ldg(a.w + c + i);
      if (a.y) {
#pragma unroll
        for (int i = 0; i < N; ++i) p.set(i, v[i]);
        y.template put<AL>(t, c, H, p);
      }
    }
    if (a.q) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) m = fmaxf(m, finite_abs(v[i]));
      const int e = ue8m0_exponent(group_max<N>(m));
      if (c < H) {
        uint32_t w[N / 4];
        codes8<N>(v, pow2_neg(e), w);
        store_codes8<N>(a.q + t * a.ldq + c, w, H - c, a.q_words);
        if (c % kGroup8 == 0) a.sf[t * a.ldsf + c / kGroup8] = static_cast<uint8_t>(e + 127);
      }
    }
  }
}

struct NormGradArgs {
  const void *dy, *x, *dsum;
  void* dx;
  const float* w;
  float *rs, *part;           // [T], [S, H]
  long long lddy, ldx, lddsum, lddx;
  float eps;
  int T, H;
};

template <class T, bool AL>
__global__ void __launch_bounds__(kNormThreads) norm_grad_kernel(const NormGradArgs a) {
  constexpr int N = Pack<T>::N;
  __shared__ float sh[32][2];
  grid_dependency_wait();
  grid_launch_dependents();
  const long long t = blockIdx.x;
  const int H = a.H;
  const Mat<T> dy(a.dy, a.lddy, a.T, H), x(a.x, a.ldx, a.T, H), ds(a.dsum, a.lddsum, a.T, H), dx(a.dx, a.lddx, a.T, H);
  float m[2] = {0.f, 0.f};
  for (int c = threadIdx.x * N; c < H; c += kNormThreads * N) {
    const Pack<T> p = x.template get<AL>(t, c, H), d = dy.template get<AL>(t, c, H);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (AL || c + i < H) {
        m[0] = fmaf(p.f(i), p.f(i), m[0]);
        m[1] = fmaf(p.f(i), d.f(i) * __ldg(a.w + c + i), m[1]);
      }
  }
  block_sum<2>(m, sh);
  const float rs = rsqrtf(m[0] / H + a.eps), k = m[1] / H * rs * rs;
  if (threadIdx.x == 0) a.rs[t] = rs;
  if (!a.dx) return;
  for (int c = threadIdx.x * N; c < H; c += kNormThreads * N) {
    const Pack<T> p = x.template get<AL>(t, c, H), d = dy.template get<AL>(t, c, H);
    Pack<T> o, u;
    if (a.dsum) u = ds.template get<AL>(t, c, H);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float v = 0.f;
      if (AL || c + i < H) v = (d.f(i) * __ldg(a.w + c + i) - p.f(i) * k) * rs;
      if (a.dsum) v += u.f(i);
      o.set(i, v);
    }
    dx.template put<AL>(t, c, H, o);
  }
}

// Partial sums of dw over rows blockIdx.y, + gridDim.y, ...; thread = column.
template <class T>
__global__ void __launch_bounds__(256) norm_dw_kernel(const NormGradArgs a) {
  using raw = typename T::raw;
  grid_dependency_wait();
  grid_launch_dependents();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.H) return;
  float s = 0.f;
  for (long long t = blockIdx.y; t < a.T; t += gridDim.y)
    s = fmaf(T::to_f(static_cast<const raw*>(a.dy)[t * a.lddy + c]),
             T::to_f(static_cast<const raw*>(a.x)[t * a.ldx + c]) * a.rs[t], s);
  a.part[static_cast<size_t>(blockIdx.y) * a.H + c] = s;
}

__global__ void __launch_bounds__(256) norm_dw_sum_kernel(const float* __restrict__ part, int S, int H, float* __restrict__ dw) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= H) return;
  float s = 0.f;
  for (int k = 0; k < S; ++k) s += part[static_cast<size_t>(k) * H + c];
  dw[c] = s;
}

template <class T>
cudaError_t norm_launch(const NormArgs& a, bool al, cudaStream_t stream) {
  return launch_pdl(al ? norm_kernel<T, true> : norm_kernel<T, false>, dim3(a.T), dim3(kNormThreads), 0, stream, a);
}

int norm_slices(int T) { return T < 64 ? (T < 1 ? 1 : T) : 64; }

// The gradient of w first: dx may take the place of what it reads.
template <class T>
cudaError_t norm_grad_launch(NormGradArgs a, bool al, float* dw, cudaStream_t stream) {
  const auto kernel = al ? norm_grad_kernel<T, true> : norm_grad_kernel<T, false>;
  void* dx = a.dx;
  if (dw) {
    a.dx = nullptr;
    cudaError_t err = launch_pdl(kernel, dim3(a.T), dim3(kNormThreads), 0, stream, a);
    if (err != cudaSuccess) return err;
    const int S = norm_slices(a.T), blocks = (a.H + 255) / 256;
    err = launch_pdl(norm_dw_kernel<T>, dim3(blocks, S), dim3(256), 0, stream, a);
    if (err != cudaSuccess) return err;
    err = launch_pdl(norm_dw_sum_kernel, dim3(blocks), dim3(256), 0, stream, static_cast<const float*>(a.part), S, a.H, dw);
    if (err != cudaSuccess) return err;
  }
  a.dx = dx;
  return dx ? launch_pdl(kernel, dim3(a.T), dim3(kNormThreads), 0, stream, a) : cudaSuccess;
}

}  // namespace

cudaError_t launch_norm(int dt, RowsView x, RowsView res, const float* w, float eps, int T, int H, RowsView sum, RowsView y,
                        Rows8View y8, cudaStream_t stream) {
  NormArgs a{};
  a.x = x.ptr;
  a.res = res.ptr;
  a.sum = sum.ptr;
  a.y = y.ptr;
  a.w = w;
  a.q = y8.q;
  a.sf = y8.sf;
  a.ldx = x.ld;
  a.ldr = res.ld;
  a.lds = sum.ld;
  a.ldy = y.ld;
  a.ldq = y8.ldq;
  a.ldsf = y8.lds;
  a.eps = eps;
  a.T = T;
  a.H = H;
  const int n = static_cast<int>(16 / dtype_bytes(dt));
  a.q_words = codes_aligned(y8, T, n);
  const bool al = H % n == 0 && rows_aligned(x, T, dt) && rows_aligned(res, T, dt) && rows_aligned(sum, T, dt) &&
                  rows_aligned(y, T, dt);
  if (dt == kBf16) return norm_launch<Bf16Elem>(a, al, stream);
  if (dt == kF16) return norm_launch<F16Elem>(a, al, stream);
  return norm_launch<F32Elem>(a, al, stream);
}

size_t norm_scratch_bytes(int T, int H) {
  return (static_cast<size_t>(T) * 4 + 255) / 256 * 256 + static_cast<size_t>(norm_slices(T)) * H * 4;
}

cudaError_t launch_norm_grad(int dt, RowsView dy, RowsView x, const float* w, float eps, RowsView dsum, int T, int H,
                             RowsView dx, float* dw, void* scratch, cudaStream_t stream) {
  NormGradArgs a{};
  a.dy = dy.ptr;
  a.x = x.ptr;
  a.dsum = dsum.ptr;
  a.dx = dx.ptr;
  a.w = w;
  a.rs = static_cast<float*>(scratch);
  a.part = reinterpret_cast<float*>(static_cast<char*>(scratch) + (static_cast<size_t>(T) * 4 + 255) / 256 * 256);
  a.lddy = dy.ld;
  a.ldx = x.ld;
  a.lddsum = dsum.ld;
  a.lddx = dx.ld;
  a.eps = eps;
  a.T = T;
  a.H = H;
  const int n = static_cast<int>(16 / dtype_bytes(dt));
  const bool al = H % n == 0 && rows_aligned(dy, T, dt) && rows_aligned(x, T, dt) && rows_aligned(dsum, T, dt) &&
                  rows_aligned(dx, T, dt);
  if (dt == kBf16) return norm_grad_launch<Bf16Elem>(a, al, dw, stream);
  if (dt == kF16) return norm_grad_launch<F16Elem>(a, al, dw, stream);
  return norm_grad_launch<F32Elem>(a, al, dw, stream);
}

}  // namespace moe
