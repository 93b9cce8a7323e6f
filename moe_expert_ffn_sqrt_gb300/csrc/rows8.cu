// Rows to and from 8 bits (rows8.cuh has the format): checkpoints of activations for the backward pass.
//
// Packing reads 16 bits and writes 8 of each value once: 16384 x 7168 bf16, 353 MB, 59 us (88% of a plain copy's rate), bound
// by HBM with 16-byte loads of 64 warps per SM on their way.  A thread keeps its columns and walks rows, so that a step costs
// three additions of addresses: places found by division 72 us, several groups' loads ahead 87 (two) to 120 us (four), the
// next row's load ahead 60.  Rows that start anywhere: 3000 x 2521 11.1 us of 3.4, unpacked 10.3.  Unpacking 16384 x 7168 63 us
// (82%), for the weight gradient 4096 x 7168 16 us of 13.
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

// A thread has the same columns of every rows-th row (a group of 128 columns to 16 lanes, fp32 32): `lanes` threads a row,
// of which a CTA has several where `lanes` is less than its threads; blockIdx.z: which `lanes` packs of the row.
template <class T, bool AL>
__global__ void __launch_bounds__(kRows8Threads) pack_rows8_kernel(const Rows8Args a, int lanes) {
  using raw = typename T::raw;
  constexpr int N = Pack<T>::N;
  grid_dependency_wait();
  grid_launch_dependents();
  int seg, cnt;
  expert_segment(a.counts, blockIdx.y, a.align, a.rows, blockIdx.x == 0 && blockIdx.z == 0, seg, cnt, a.status);
  const int sub = threadIdx.x % lanes, c = (blockIdx.z * lanes + sub) * N, per = kRows8Threads / lanes;
  const bool cols = c < a.cols;
  const int step = gridDim.x * per;
  const raw* lo = static_cast<const raw*>(a.x);
  const raw* hi = lo + (a.rows - 1) * a.ldx + a.cols;
  long long row = static_cast<long long>(blockIdx.x) * per;          // the CTA's first; every warp goes on as long as it does
  const long long mine = seg + row + threadIdx.x / lanes;
  const raw* x = lo + mine * a.ldx + c;
  uint8_t* q = a.q + mine * a.ldq;
  const bool first = threadIdx.x % 32 == 0 || sub == 0, last = threadIdx.x % 32 == 31 || sub == lanes - 1;
  uint8_t* sf = a.sf + mine * a.ldsf + c / kGroup8;
  int left = cnt - static_cast<int>(row < cnt ? row : cnt) - static_cast<int>(threadIdx.x) / lanes;     // rows from this one on
  for (; row < cnt; row += step, left -= step) {
    const bool live = cols && left > 0;
    Words<T> p;
    if (live) {
      if constexpr (AL) {
        p = Words<T>(*reinterpret_cast<const uint4*>(x));
      } else {
        ShiftedPack<T> s;
        s.load(x, lo, hi);
        p = Words<T>(s.get());
      }
    }
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = AL || c + i < a.cols ? p.f(i) : 0.f;
    uint32_t w[N / 4];
    const uint32_t scale = encode8<N>(v, w);
    if constexpr (AL) {
      if (live) store_codes8<N>(q + c, w, N, true);
    } else {
      store_row_codes8<N>(q, c, left > 0 ? a.cols : 0, w, a.words, first, last);
    }
    if (live && c % kGroup8 == 0) *sf = static_cast<uint8_t>(scale);
    x += step * a.ldx;
    q += step * a.ldq;
    sf += step * a.ldsf;
  }
}

// Row r of the output is row r of the codes, or row ids[r] / div of them.  Threads as in the pack kernel; two rows' codes are
// on their way together.
template <class T, bool AL>
__global__ void __launch_bounds__(kRows8Threads) unpack_rows8_kernel(const Rows8Args a, int lanes) {
  using raw = typename T::raw;
  constexpr int N = Pack<T>::N, kAhead = 2;
  grid_dependency_wait();
  grid_launch_dependents();
  int seg, cnt;
  expert_segment(a.counts, blockIdx.y, a.align, a.rows, blockIdx.x == 0 && blockIdx.z == 0, seg, cnt, a.status);
  const int sub = threadIdx.x % lanes, c = (blockIdx.z * lanes + sub) * N, per = kRows8Threads / lanes;
  const int step = gridDim.x * per;
  const bool first = threadIdx.x % 32 == 0 || sub == 0, last = threadIdx.x % 32 == 31 || sub == lanes - 1;
  const uint8_t *q = a.q + c, *sf = a.sf + c / kGroup8;
  long long row = static_cast<long long>(blockIdx.x) * per;          // the CTA's first; every warp goes on as long as it does
  const int mine = threadIdx.x / lanes;
  raw* out = static_cast<raw*>(a.out) + (seg + row + mine) * a.ldx;
  for (; row < cnt; row += kAhead * step) {
    uint32_t w[kAhead][N / 4], s[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      long long src = seg + row + mine + k * step;
#pragma unroll
      for (int i = 0; i < N / 4; ++i) w[k][i] = 0;
      s[k] = 127;
      if (c >= a.cols || row + mine + k * step >= cnt) continue;
      if (a.ids) {
        const int id = __ldg(a.ids + src);
        src = id >= 0 ? static_cast<unsigned>(id) / static_cast<unsigned>(a.div) : -1;
        if (src >= a.src_rows) src = -1;
        if (src < 0) {
          if (c == 0) record_error(a.status, kDevErrIndex);
          continue;
        }
      }
      load_codes8<N>(q + src * a.ldq, w[k], a.cols - c, a.words);
      s[k] = sf[src * a.ldsf];
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      float v[N];
      decode8<T, N>(w[k], s[k], v);
      Words<T> p;
#pragma unroll
      for (int i = 0; i < N; i += 2) p.set2(i, v[i], v[i + 1]);
      const bool there = row + mine + k * step < cnt;
      if constexpr (AL) {
        if (there && c < a.cols) *reinterpret_cast<uint4*>(out + c) = make_uint4(p.w[0], p.w[1], p.w[2], p.w[3]);
      } else {
        store_shifted<T>(out, c, there ? a.cols : 0, p, first, last);
      }
      out += step * a.ldx;
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

// Threads per row: the most (of 256, 128, ..) that leave at most an eighth of a row's last round idle; least: a group's.
template <class T, class K>
cudaError_t rows8_launch(K kernel, const Rows8Args& a, int E, cudaStream_t stream) {
  const int packs = (a.cols + Pack<T>::N - 1) / Pack<T>::N, least = kGroup8 / Pack<T>::N;
  int lanes = kRows8Threads;
  while (lanes > least && (packs + lanes - 1) / lanes * lanes - packs > packs / 8) lanes /= 2;
  const int z = (packs + lanes - 1) / lanes, per = kRows8Threads / lanes;
  const long long live = a.counts ? a.rows - static_cast<long long>(E) * (a.align - 1) : a.rows;
  return launch_pdl(kernel, dim3(row_blocks(live, E, per, z), static_cast<unsigned>(E), static_cast<unsigned>(z)),
                    dim3(kRows8Threads), 0, stream, a, lanes);
}
template <class T>
cudaError_t pack_launch(const Rows8Args& a, bool al, int E, cudaStream_t stream) {
  return rows8_launch<T>(al ? pack_rows8_kernel<T, true> : pack_rows8_kernel<T, false>, a, E, stream);
}
template <class T>
cudaError_t unpack_launch(const Rows8Args& a, bool al, int E, cudaStream_t stream) {
  return rows8_launch<T>(al ? unpack_rows8_kernel<T, true> : unpack_rows8_kernel<T, false>, a, E, stream);
}

}  // namespace

cudaError_t launch_pack_rows8(int dt, RowsView x, const int32_t* counts, int rows, int cols, int E, int align, Rows8View out,
                              uint32_t* status, cudaStream_t stream) {
  Rows8Args a = rows8_args(x, out, counts, rows, cols, align, status);
  const int n = static_cast<int>(16 / dtype_bytes(dt)), segs = counts ? E : 1;
  a.x = x.ptr;
  a.words = codes_aligned(out, rows, n);
  const bool al = cols % n == 0 && rows_aligned(x, rows, dt) && a.words;
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
