// Row data of the training operators: element types and 16-byte (or single-element) accesses.
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

// N consecutive elements: 16 bytes with one access (N = 16 / sizeof), or one element (rows whose
// base, pitch or width is not a multiple of 16 bytes).
template <class T, int N>
struct Pack {
  typename T::raw v[N];
  __device__ __forceinline__ float f(int i) const { return T::to_f(v[i]); }
  __device__ __forceinline__ void set(int i, float x) { v[i] = T::from_f(x); }
};

template <class T, int N>
__device__ __forceinline__ Pack<T, N> load_pack(const typename T::raw* p) {
  Pack<T, N> r;
  if constexpr (N == 1) {
    r.v[0] = *p;
  } else {
    static_assert(sizeof(r) == 16, "one 16-byte access");
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    memcpy(&r, &u, 16);
  }
  return r;
}

template <class T, int N>
__device__ __forceinline__ void store_pack(typename T::raw* p, const Pack<T, N>& r) {
  if constexpr (N == 1) {
    *p = r.v[0];
  } else {
    uint4 u;
    memcpy(&u, &r, 16);
    *reinterpret_cast<uint4*>(p) = u;
  }
}

}  // namespace moe
