// Gradient of the routing weights with respect to the gate logits (the scoring of moe_route:
// page "DeepSeek V4 MegaMoE Kernel 深度解析", 经典 MoE 的计算过程 / 第一步：路由).
//
// With s = softmax(l) or sqrt(softplus(l)), w_k = s_k of the K selected experts (divided by their sum
// when renormalised) and dw = dL/dw:
//   g_k = s_k dL/ds_k = w_k (dw_k - sum_j w_j dw_j)   renormalised,   w_k dw_k   otherwise
//   softmax:         dl_i = [i selected] g_i - p_i sum_j g_j     (renormalised: sum_j g_j = 0)
//   sqrt(softplus):  dl_k = g_k sigmoid(l_k) / (2 softplus(l_k)), zero elsewhere
// so only the unnormalised softmax needs the whole row of logits.  The forward's own weights stand in
// for the scores, so nothing divides by a sum that may underflow.  The selection itself (and with it
// e_score_correction_bias) has no gradient.
// One warp per token; the [T, E] write (and the logits' read, where needed) bounds it.
#include "kernels.h"
#include "rows.cuh"

namespace moe {

namespace {

constexpr int kGradWarps = 8;

// sigmoid(l) / softplus(l); tends to 1 for l -> -inf, where both underflow together.
__device__ __forceinline__ float sigmoid_over_softplus(float l) {
  if (l < -20.f) return 1.f;                       // 1 - e^l / 2 + ..., e^-20 / 2 < 2^-24
  const float e = expf(-fabsf(l));
  const float sig = l >= 0.f ? 1.f / (1.f + e) : e / (1.f + e);
  return sig / (fmaxf(l, 0.f) + log1pf(e));
}

template <class T>
__global__ void __launch_bounds__(kGradWarps * 32) route_grad_kernel(const float* __restrict__ logits,
                                                                     const int32_t* __restrict__ ids,
                                                                     const float* __restrict__ w,
                                                                     const float* __restrict__ dw, int T_, int E, int K,
                                                                     int softmax, int renorm,
                                                                     typename T::raw* __restrict__ out,
                                                                     uint32_t* status) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int t = blockIdx.x * kGradWarps + warp;
  if (t >= T_) return;
  const float* lrow = logits + static_cast<size_t>(t) * E;
  typename T::raw* orow = out + static_cast<size_t>(t) * E;
  int id = -1;
  float wk = 0.f, dk = 0.f;
  if (lane < K) {
    id = __ldg(ids + static_cast<size_t>(t) * K + lane);
    wk = __ldg(w + static_cast<size_t>(t) * K + lane);
    dk = __ldg(dw + static_cast<size_t>(t) * K + lane);
    if (id < 0 || id >= E) {
      record_error(status, kDevErrIndex);
      id = -1;
      wk = dk = 0.f;
    }
  }
  float g = wk * dk;
  if (renorm) {
    float c = g;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) c += __shfl_xor_sync(0xffffffffu, c, off);
    g = id >= 0 ? wk * (dk - c) : 0.f;
  }
  float total = 0.f, lmax = -INFINITY, sum = 0.f;
  const bool dense = softmax && !renorm;
  if (dense) {
    total = g;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
    for (int e = lane; e < E; e += 32) lmax = fmaxf(lmax, __ldg(lrow + e));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) lmax = fmaxf(lmax, __shfl_xor_sync(0xffffffffu, lmax, off));
    for (int e = lane; e < E; e += 32) sum += expf(__ldg(lrow + e) - lmax);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  }
  for (int e = lane; e < E; e += 32)
    orow[e] = T::from_f(dense ? -(expf(__ldg(lrow + e) - lmax) / sum) * total : 0.f);
  // an expert named twice gets both terms, from its first slot
  float mine = 0.f;
  bool first = id >= 0;
  for (int k = 0; k < K; ++k) {
    const int ik = __shfl_sync(0xffffffffu, id, k);
    const float gk = __shfl_sync(0xffffffffu, g, k);
    if (ik == id) {
      mine += gk;
      if (k < lane) first = false;
    }
  }
  __syncwarp();
  if (first) {
    const float l = __ldg(lrow + id);
    float v = mine;
    if (!softmax)
      v = 0.5f * mine * sigmoid_over_softplus(l);
    else if (dense)
      v = mine - (expf(l - lmax) / sum) * total;
    orow[id] = T::from_f(v);
  }
}

}  // namespace

cudaError_t launch_route_grad(int dt, const float* logits, const int32_t* ids, const float* w, const float* dw, int T,
                              int E, int K, int softmax, int renorm, void* out, uint32_t* status, cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  const int grid = (T + kGradWarps - 1) / kGradWarps;
  if (dt == kBf16)
    route_grad_kernel<Bf16Elem><<<grid, kGradWarps * 32, 0, stream>>>(logits, ids, w, dw, T, E, K, softmax, renorm,
                                                                      static_cast<uint16_t*>(out), status);
  else if (dt == kF16)
    route_grad_kernel<F16Elem><<<grid, kGradWarps * 32, 0, stream>>>(logits, ids, w, dw, T, E, K, softmax, renorm,
                                                                     static_cast<uint16_t*>(out), status);
  else
    route_grad_kernel<F32Elem><<<grid, kGradWarps * 32, 0, stream>>>(logits, ids, w, dw, T, E, K, softmax, renorm,
                                                                     static_cast<float*>(out), status);
  return cudaGetLastError();
}

}  // namespace moe
