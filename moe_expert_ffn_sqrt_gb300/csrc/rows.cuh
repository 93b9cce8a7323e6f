// Row data of the training operators: element types and 16-byte accesses, aligned or not.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>
#include <type_traits>

#include "kernels.h"

namespace moe {

struct Bf16Elem {
  using raw = uint16_t;
  static __device__ __forceinline__ float to_f(raw v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
  static __device__ __forceinline__ raw from_f(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }
};
struct F16Elem {
  using raw = uint16_t;
  static __device__ __forceinline__ float to_f(raw v) { return __half2float(__ushort_as_half(v)); }
  static __device__ __forceinline__ raw from_f(float f) { return __half_as_ushort(__float2half_rn(f)); }
};
struct F32Elem {
  using raw = float;
  static __device__ __forceinline__ float to_f(raw v) { return v; }
  static __device__ __forceinline__ raw from_f(float f) { return f; }
};

// The elements of 16 bytes.
template <class T>
struct Pack {
  static constexpr int N = 16 / sizeof(typename T::raw);
  typename T::raw v[N];
  __device__ __forceinline__ float f(int i) const { return T::to_f(v[i]); }
  __device__ __forceinline__ void set(int i, float x) { v[i] = T::from_f(x); }
};

// From and to a 16-byte boundary.
template <class T>
__device__ __forceinline__ Pack<T> load_pack(const typename T::raw* p) {
  Pack<T> r;
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  memcpy(&r, &u, 16);
  return r;
}
template <class T>
__device__ __forceinline__ void store_pack(typename T::raw* p, const Pack<T>& r) {
  uint4 u;
  memcpy(&u, &r, 16);
  *reinterpret_cast<uint4*>(p) = u;
}

// A pack from any element on, out of the two aligned 16-byte words that hold it; what they hold of other rows is
// read and left.  [lo, hi): the matrix' first element and the end of its last row.  Where a word would reach
// past them, element by element (zeros outside).
template <class T>
struct ShiftedPack {
  uint4 a, b;
  uint32_t off;                                     // bytes from a's start
  __device__ __forceinline__ void load(const typename T::raw* p, const typename T::raw* lo, const typename T::raw* hi) {
    using U = uintptr_t;
    const U u = reinterpret_cast<U>(p);
    const uint4* q = reinterpret_cast<const uint4*>(u & ~U(15));
    off = static_cast<uint32_t>(u & 15);
    if (reinterpret_cast<U>(q) >= reinterpret_cast<U>(lo) && reinterpret_cast<U>(q + 2) <= reinterpret_cast<U>(hi)) {
      a = q[0];
      b = q[1];
    } else {
      Pack<T> t;
#pragma unroll
      for (int i = 0; i < Pack<T>::N; ++i) {
        t.v[i] = typename T::raw(0);
        if (p + i >= lo && p + i < hi) t.v[i] = p[i];
      }
      memcpy(&a, &t, 16);
      b = make_uint4(0, 0, 0, 0);
      off = 0;
    }
  }
  __device__ __forceinline__ Pack<T> get() const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t h[6], s[5];
#pragma unroll
    for (int i = 0; i < 6; ++i) h[i] = (off & 8) ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) s[i] = (off & 4) ? h[i + 1] : h[i];
    if (sizeof(typename T::raw) < 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = __funnelshift_r(s[i], s[i + 1], (off & 3) * 8);
    }
    Pack<T> r;
    memcpy(&r, s, 16);
    return r;
  }
};

// Elements [from, to) of a pack (all of them at a 16-byte boundary).
template <class T>
__device__ __forceinline__ void store_part(typename T::raw* p, const Pack<T>& r, int from, int to) {
  if (from == 0 && to == Pack<T>::N) {
    store_pack<T>(p, r);
    return;
  }
#pragma unroll
  for (int i = 0; i < Pack<T>::N; ++i)
    if (i >= from && i < to) p[i] = r.v[i];
}

// A pack as words: two 16-bit values are taken out of and put into a word at a time.  (As an array of 16-bit values the
// compiler gives each a register of its own.)
template <class T>
struct Words {
  static constexpr int N = Pack<T>::N;
  uint32_t w[4];
  __device__ __forceinline__ Words() : w{0, 0, 0, 0} {}
  __device__ __forceinline__ Words(const uint4& u) : w{u.x, u.y, u.z, u.w} {}
  __device__ __forceinline__ Words(const Pack<T>& p) { memcpy(w, &p, 16); }
  __device__ __forceinline__ operator Pack<T>() const {
    Pack<T> p;
    memcpy(&p, w, 16);
    return p;
  }
  __device__ __forceinline__ float f(int j) const {
    if constexpr (N == 4) return __uint_as_float(w[j]);
    else if constexpr (std::is_same<T, Bf16Elem>::value)
      return __uint_as_float(j & 1 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
    else {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[j / 2]));
      return j & 1 ? v.y : v.x;
    }
  }
  // values j and j + 1, j even
  __device__ __forceinline__ void set2(int j, float a, float b) {
    if constexpr (N == 4) {
      w[j] = __float_as_uint(a);
      w[j + 1] = __float_as_uint(b);
    } else if constexpr (std::is_same<T, Bf16Elem>::value) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
      w[j / 2] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __floats2half2_rn(a, b);
      w[j / 2] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  // Each value plus o's, rounded to T.  (Two 16-bit values at a time, with one rounding; a sum in fp32 first would round to
  // the same: it is exact unless the smaller value is below 2^-13 of the larger, which then stays what it is.)
  __device__ __forceinline__ void add(const Words& o) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (N == 4) {
        w[i] = __float_as_uint(__uint_as_float(w[i]) + __uint_as_float(o.w[i]));
      } else if constexpr (std::is_same<T, Bf16Elem>::value) {
        const __nv_bfloat162 h = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), *reinterpret_cast<const __nv_bfloat162*>(&o.w[i]));
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __half2 h = __hadd2(*reinterpret_cast<const __half2*>(&w[i]), *reinterpret_cast<const __half2*>(&o.w[i]));
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
  }
  // After this the compiler has the words alone: without it, it holds the values over a reduction, in twice the registers.
  __device__ __forceinline__ void keep() {
#pragma unroll
    for (int i = 0; i < 4; ++i) asm volatile("" : "+r"(w[i]));
  }
};

// Stores a row's packs where the row starts anywhere: `row` its first element, c the thread's first column (its pack may lie
// past the row's end H).  Called by all lanes of a warp, whose packs follow one another; first, last: whether the lane's pack
// is the first or last of those that do.  A lane stores the aligned 16 bytes that end in its pack, with the end of the lane's
// before it; only the packs at the ends go element by element.  (All element by element: 1450 rows of 2521 fp16 columns,
// normed, 24 us; so 12.)
template <class T>
__device__ __forceinline__ void store_shifted(typename T::raw* row, int c, int H, const Words<T>& own, bool first, bool last) {
  constexpr int N = Words<T>::N, kSize = 16 / N;
  const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15) / kSize;      // columns of the first word before c
  ShiftedPack<T> s;
  s.a = make_uint4(__shfl_up_sync(0xffffffffu, own.w[0], 1), __shfl_up_sync(0xffffffffu, own.w[1], 1),
                   __shfl_up_sync(0xffffffffu, own.w[2], 1), __shfl_up_sync(0xffffffffu, own.w[3], 1));
  s.b = make_uint4(own.w[0], own.w[1], own.w[2], own.w[3]);
  s.off = 16 - mis * kSize;
  Pack<T> out = s.get();
  if (mis == 0) out = own;
  const int c0 = c - mis;
  if ((!first || mis == 0) && c0 + N <= H) {
    store_pack<T>(row + c0, out);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (c0 + i < H && (!first || i >= mis)) row[c0 + i] = out.v[i];
  }
  if (last && mis) {
    const Pack<T> p = own;
#pragma unroll
    for (int i = 1; i < N; ++i)
      if (i >= N - mis && c + i < H) row[c + i] = p.v[i];
  }
}

// Expert e's rows in buffers of `rows` rows: cnt rows from row seg on (counts null: all of them).  Called by the whole
// CTA; where `report`, a segment that would leave the buffers is recorded; it is cut in any case.
__device__ __forceinline__ void expert_segment(const int32_t* counts, int e, int align, int rows, bool report, int& seg,
                                               int& cnt, uint32_t* status) {
  __shared__ unsigned long long s_seg;
  seg = 0;
  cnt = rows;
  if (!counts) return;
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
  const int c = __ldg(counts + e);
  cnt = min(max(c, 0), rows - seg);
  if (report && threadIdx.x == 0 && (c < 0 || c > cnt)) record_error(status, kDevErrIndex);
}

}  // namespace moe
