// Rows to and from 8 bits (rows8.cuh has the format): checkpoints of activations for the backward pass.
#include "rows8.cuh"

namespace moe {

namespace {

constexpr int kRows8Threads = 256;

struct Rows8Args {
  const void* x;              // packed from
  void* out;                  // unpacked to
  uint8_t *q, *sf;
  const int32_t *counts, *ids;
  long long ldx, ldq, ldsf;   // ldx: of x or out
  int rows, cols, align, div, src_rows;
  int words;                  // codes in whole words
  uint32_t* status;
};

template <class T, bool AL>
__global__ void __launch_bounds__(kRows8Threads) pack_rows8_kernel(const Rows8Args a) {
  using raw = typename T::raw;
  constexpr int N = Pack<T>::N, kLanes = kGroup8 / N, kPer = kRows8Threads / kLanes;
  grid_dependency_wait();
  grid_launch_dependents();
  int seg, cnt;
  expert_segment(a.counts, blockIdx.y, a.align, a.rows, blockIdx.x == 0, seg, cnt, a.status);
  const int groups = groups8(a.cols), lane = threadIdx.x % kLanes;
  const raw* lo = static_cast<const raw*>(a.x);
  const raw* hi = lo + (a.rows - 1) * a.ldx + a.cols;
  const long long units = static_cast<long long>(cnt) * groups, step = static_cast<long long>(gridDim.x) * kPer;
  for (long long u0 = static_cast<long long>(blockIdx.x) * kPer; u0 < units; u0 += step) {
    const long long u = u0 + threadIdx.x / kLanes, row = seg + u / groups;
    const int g = static_cast<int>(u % groups), c = g * kGroup8 + lane * N;
    const bool live = u < units && c < a.cols;
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
    if (live) {
      Pack<T> p;
      if constexpr (AL) {
        p = load_pack<T>(lo + row * a.ldx + c);
      } else {
        ShiftedPack<T> s;
        s.load(lo + row * a.ldx + c, lo, hi);
        p = s.get();
      }
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (AL || c + i < a.cols) v[i] = p.f(i);
    }
    uint32_t w[N / 4];
    const uint32_t scale = encode8<N>(v, w);
    if (live) {
      store_codes8<N>(a.q + row * a.ldq + c, w, a.cols - c, a.words);
      if (lane == 0) a.sf[row * a.ldsf + g] = static_cast<uint8_t>(scale);
    }
  }
}

// Row r of the output is row r of the codes, or row ids[r] / div of them.
template <class T, bool AL>
__global__ void __launch_bounds__(kRows8Threads) unpack_rows8_kernel(const Rows8Args a) {
  using raw = typename T::raw;
  constexpr int N = Pack<T>::N;
  grid_dependency_wait();
  grid_launch_dependents();
  int seg, cnt;
  expert_segment(a.counts, blockIdx.y, a.align, a.rows, blockIdx.x == 0, seg, cnt, a.status);
  const int packs = (a.cols + N - 1) / N;
  const long long units = static_cast<long long>(cnt) * packs, step = static_cast<long long>(gridDim.x) * kRows8Threads;
  for (long long u = static_cast<long long>(blockIdx.x) * kRows8Threads + threadIdx.x; u < units; u += step) {
    const long long row = seg + u / packs;
    const int c = static_cast<int>(u % packs) * N;
    long long src = row;
    if (a.ids) {
      const int id = __ldg(a.ids + row);
      src = id >= 0 ? id / a.div : -1;
      if (src >= a.src_rows) src = -1;
      if (src < 0 && c == 0) record_error(a.status, kDevErrIndex);
    }
    uint32_t w[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i) w[i] = 0;
    float s = 1.f;
    if (src >= 0) {
      load_codes8<N>(a.q + src * a.ldq + c, w, a.cols - c, a.words);
      s = scale8(a.sf[src * a.ldsf + c / kGroup8]);
    }
    Pack<T> p;
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      float v[4];
      values8(w[i], s, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) p.v[4 * i + j] = from_value8<T>(v[j]);
    }
    raw* o = static_cast<raw*>(a.out) + row * a.ldx + c;
    if constexpr (AL) {
      store_pack<T>(o, p);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (c + i < a.cols) o[i] = p.v[i];
    }
  }
}

Rows8Args rows8_args(RowsView x, const Rows8View& m, const int32_t* counts, int rows, int cols, int align, uint32_t* status) {
  Rows8Args a{};
  a.ldx = x.ld;
  a.q = m.q;
  a.sf = m.sf;
  a.ldq = m.ldq;
  a.ldsf = m.lds;
  a.counts = counts;
  a.rows = rows;
  a.cols = cols;
  a.align = align;
  a.div = 1;
  a.src_rows = rows;
  a.status = status;
  return a;
}

// CTAs per segment: `units` in all at `per` a CTA, sixteen CTAs per SM at most.
dim3 rows8_grid(long long units, int per, int E) {
  long long n = (units + per - 1) / per;
  const long long most = (16LL * num_sms() + E - 1) / E;
  if (n > most) n = most;
  return dim3(static_cast<unsigned>(n < 1 ? 1 : n), static_cast<unsigned>(E));
}

template <class T>
cudaError_t pack_launch(const Rows8Args& a, bool al, int E, cudaStream_t stream) {
  constexpr int per = kRows8Threads / (kGroup8 / Pack<T>::N);
  return launch_pdl(al ? pack_rows8_kernel<T, true> : pack_rows8_kernel<T, false>,
                    rows8_grid(static_cast<long long>(a.rows) * groups8(a.cols), per, E), dim3(kRows8Threads), 0, stream, a);
}
template <class T>
cudaError_t unpack_launch(const Rows8Args& a, bool al, int E, cudaStream_t stream) {
  return launch_pdl(al ? unpack_rows8_kernel<T, true> : unpack_rows8_kernel<T, false>,
                    rows8_grid(static_cast<long long>(a.rows) * ((a.cols + Pack<T>::N - 1) / Pack<T>::N), kRows8Threads, E),
                    dim3(kRows8Threads), 0, stream, a);
}

}  // namespace

cudaError_t launch_pack_rows8(int dt, RowsView x, const int32_t* counts, int rows, int cols, int E, int align, Rows8View out,
                              uint32_t* status, cudaStream_t stream) {
  Rows8Args a = rows8_args(x, out, counts, rows, cols, align, status);
  const int n = static_cast<int>(16 / dtype_bytes(dt)), segs = counts ? E : 1;
  a.x = x.ptr;
  a.words = codes_aligned(out, rows, n);
  const bool al = cols % n == 0 && rows_aligned(x, rows, dt);
  if (dt == kBf16) return pack_launch<Bf16Elem>(a, al, segs, stream);
  if (dt == kF16) return pack_launch<F16Elem>(a, al, segs, stream);
  return pack_launch<F32Elem>(a, al, segs, stream);
}

cudaError_t launch_unpack_rows8(int dt, Rows8View x, const int32_t* ids, int div, int src_rows, const int32_t* counts,
                                int rows, int cols, int E, int align, RowsView out, uint32_t* status, cudaStream_t stream) {
  Rows8Args a = rows8_args(out, x, counts, rows, cols, align, status);
  const int n = static_cast<int>(16 / dtype_bytes(dt)), segs = counts ? E : 1;
  a.out = out.ptr;
  a.ids = ids;
  a.div = div;
  a.src_rows = ids ? src_rows : rows;
  a.words = codes_aligned(x, a.src_rows, n);
  const bool al = cols % n == 0 && rows_aligned(out, rows, dt);
  if (dt == kBf16) return unpack_launch<Bf16Elem>(a, al, segs, stream);
  if (dt == kF16) return unpack_launch<F16Elem>(a, al, segs, stream);
  return unpack_launch<F32Elem>(a, al, segs, stream);
}

}  // namespace moe
