// Rows held in 8 bits: E4M3 codes with one UE8M0 scale per 128 columns, by the rule of moe_route's x_q and x_sf
// (page "DeepSeek V4 MegaMoE Kernel 深度解析", 二 阶段 3: amax -> UE8M0 -> E4M3).
//
// Per group of 128 columns (the last one may be shorter) the scale is the smallest 2^e, e in [-127, 127], with
// amax <= 448 * 2^e over the group's finite values (e = 0 where amax = 0); a value's code is v / 2^e rounded to the
// nearest of E4M3 (ties to even, off by at most 2^-4 of the value, 2^-10 * 2^e below 2^-6 * 2^e).  An infinity or NaN
// gets the NaN code: a conversion that saturated would pass an overflow on as a number.
#pragma once
#include <cuda_fp8.h>

#include "rows.cuh"

namespace moe {

constexpr int kGroup8 = 128;
__host__ __device__ __forceinline__ int groups8(int cols) { return (cols + kGroup8 - 1) / kGroup8; }

// max over the lanes that hold a group: N columns per lane
template <int N>
__device__ __forceinline__ float group_max(float m) {
#pragma unroll
  for (int d = kGroup8 / N / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  return m;
}

// Codes (N / 4 words) and scale byte of a group's values, N (4 or 8) in each of its 128 / N lanes; called by whole warps.
// The maximum skips NaN by itself, and a NaN's conversion is the NaN code: only an infinity, which shows in the maximum,
// takes another look.  For amax = (1 + m / 2^23) 2^(x - 127) the exponent is x - 135, one more where m > 0x600000 (448 is
// 1.75 * 2^8); it is at most 120, so that 2^-e is a normal number.
template <int N>
__device__ __forceinline__ uint32_t encode8(const float (&value)[N], uint32_t (&w)[N / 4]) {
  float v[N], m = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = value[i];
    m = fmaxf(m, fabsf(v[i]));
  }
  m = group_max<N>(m);
  if (__any_sync(0xffffffffu, m == INFINITY)) {
    m = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (fabsf(v[i]) == INFINITY) v[i] = __int_as_float(0x7fc00000);
      m = fmaxf(m, fabsf(v[i]));
    }
    m = group_max<N>(m);
  }
  const uint32_t b = __float_as_uint(m);
  uint32_t s = (b + 0x1FFFFFu) >> 23;                    // e + 135
  s = s > 8 ? s - 8 : 0;                                 // e + 127
  if (b == 0) s = 127;
  const float inv = __uint_as_float((254 - s) << 23);
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i] * inv, v[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2] * inv, v[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  return s;
}

// The first `n` of N codes to q (whole words where `words`: q on an N-byte boundary).
template <int N>
__device__ __forceinline__ void store_codes8(uint8_t* q, const uint32_t (&w)[N / 4], int n, bool words) {
  if (words && n >= N) {
    if constexpr (N == 8)
      *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(q) = w[0];
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i < n) q[i] = static_cast<uint8_t>(w[i / 4] >> (8 * (i % 4)));
}

// A row's codes, N to a lane from column c on (c may lie past the row's end), called as store_shifted: where rows start on no
// N-byte boundary (not `words`), a lane stores the aligned N bytes that end in its codes.
template <int N>
__device__ __forceinline__ void store_row_codes8(uint8_t* row, int c, int cols, const uint32_t (&w)[N / 4], bool words,
                                                 bool first, bool last) {
  if (words) {
    if (c < cols) store_codes8<N>(row + c, w, cols - c, true);
    return;
  }
  const int m = static_cast<int>(reinterpret_cast<uintptr_t>(row) & (N - 1));
  uint32_t out[N / 4];
  if constexpr (N == 8) {
    const unsigned long long own = static_cast<unsigned long long>(w[1]) << 32 | w[0], prev = __shfl_up_sync(0xffffffffu, own, 1);
    const unsigned long long o = m ? own << (8 * m) | prev >> (64 - 8 * m) : own;
    out[0] = static_cast<uint32_t>(o);
    out[1] = static_cast<uint32_t>(o >> 32);
  } else {
    const uint32_t prev = __shfl_up_sync(0xffffffffu, w[0], 1);
    out[0] = m ? w[0] << (8 * m) | prev >> (32 - 8 * m) : w[0];
  }
  const int c0 = c - m;
  if ((!first || m == 0) && c0 + N <= cols) {
    store_codes8<N>(row + c0, out, N, true);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (c0 + i < cols && (!first || i >= m)) row[c0 + i] = static_cast<uint8_t>(out[i / 4] >> (8 * (i % 4)));
  }
  if (last && m) {
#pragma unroll
    for (int i = 1; i < N; ++i)
      if (i >= N - m && c + i < cols) row[c + i] = static_cast<uint8_t>(w[i / 4] >> (8 * (i % 4)));
  }
}

// Values (as T holds them, in fp32) of N codes with scale byte s.  Two codes to fp16 at a time is exact, so is the product
// with 2^(s - 127) within fp32's range, and T holds a value of its own type's rows exactly but where a code rounded up to
// the next power of two past T's largest, which then stands for it (65536 of fp16, 2^128 of bf16 and fp32); only scales
// from kLimit on can reach that.  (s = 255, which no call here writes, is UE8M0's NaN.)
template <class T, int N>
__device__ __forceinline__ void decode8(const uint32_t (&w)[N / 4], uint32_t s, float (&v)[N]) {
  constexpr bool kHalf = std::is_same<T, F16Elem>::value;
  constexpr uint32_t kLimit = kHalf ? 135 : 247;           // 448 * 2^8 > 65504, 448 * 2^120 > 2^128
  const float scale = __uint_as_float((s << 23) | (s ? 0u : 0x00400000u));
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i / 2] >> (16 * (i % 2))), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    v[2 * i] = f.x * scale;
    v[2 * i + 1] = f.y * scale;
  }
  if (s >= kLimit) {
    const float most = kHalf ? 65504.f : std::is_same<T, Bf16Elem>::value ? 3.3895314e38f : 3.402823466e38f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (fabsf(v[i]) > most) v[i] = copysignf(most, v[i]);
      if (s == 255) v[i] = __int_as_float(0x7fc00000);
    }
  }
}

// The same of 8 codes, taken out one by one (the codes and the scale stay in three registers).
template <class T>
struct Codes8 {
  uint32_t w[2];
  float scale;
  __device__ __forceinline__ void set_scale(uint32_t s) {
    scale = s == 255 ? __int_as_float(0x7fc00000) : __uint_as_float((s << 23) | (s ? 0u : 0x00400000u));
  }
  __device__ __forceinline__ float f(int i) const {
    constexpr float most = std::is_same<T, F16Elem>::value ? 65504.f : 3.3895314e38f;
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i / 4] >> (16 * (i / 2 % 2))), __NV_E4M3);
    const float2 p = __half22float2(__half2(h));
    float v = (i % 2 ? p.y : p.x) * scale;
    v = fabsf(v) > most ? copysignf(most, v) : v;
    // (rows of other types may hold values that fp16 rounds)
    return std::is_same<T, F16Elem>::value ? F16Elem::to_f(F16Elem::from_f(v)) : v;
  }
};

// N codes from q on (whole words where `words`); zeros past the first n.
template <int N>
__device__ __forceinline__ void load_codes8(const uint8_t* q, uint32_t (&w)[N / 4], int n, bool words) {
  if (words && n >= N) {
    if constexpr (N == 8) {
      const uint2 u = *reinterpret_cast<const uint2*>(q);
      w[0] = u.x;
      w[1] = u.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(q);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < N / 4; ++i) w[i] = 0;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i < n) w[i / 4] |= static_cast<uint32_t>(q[i]) << (8 * (i % 4));
}

// Every row of a matrix on a 16-byte boundary (not given: true).
inline bool rows_aligned(const RowsView& m, int rows, int dt) {
  return !m.ptr || (reinterpret_cast<uintptr_t>(m.ptr) % 16 == 0 && (rows <= 1 || m.ld * dtype_bytes(dt) % 16 == 0));
}
// Every row's codes on an n-byte boundary.
inline bool codes_aligned(const Rows8View& m, int rows, int n) {
  return reinterpret_cast<uintptr_t>(m.q) % n == 0 && (rows <= 1 || m.ldq % n == 0);
}

}  // namespace moe
