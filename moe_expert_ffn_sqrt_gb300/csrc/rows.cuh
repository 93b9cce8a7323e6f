// Row data of the training operators: element types and 16-byte accesses, aligned or not.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>

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

}  // namespace moe
