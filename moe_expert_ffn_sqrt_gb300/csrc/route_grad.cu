// Gradient of the routing weights with respect to the gate logits (the scoring of moe_route:
// page "DeepSeek V4 MegaMoE Kernel 深度解析", 经典 MoE 的计算过程 / 第一步：路由).
//
// With s = softmax(l), sqrt(softplus(l)) or sigmoid(l), w_k = c s_k of the K selected experts (divided by their sum
// when renormalised; c = 1 for moe_route's weights) and dw = dL/dw:
//   g_k = s_k dL/ds_k = w_k sum_j w_j / c (dw_k - dw_j)   renormalised,   w_k dw_k   otherwise
// (the same as w_k (dw_k - sum_j w_j dw_j / c), since the weights add up to c, but without its cancellation where one
// weight is nearly c)
//   softmax:         dl_i = [i selected] g_i - p_i sum_j g_j     (renormalised: sum_j g_j = 0)
//                         = (1 - p_i) g_i - p_i sum_{j != i} g_j  of a selected i: near p_i = 1 the first form subtracts two
//                           nearly equal numbers, and 1 - p_i is there the other exponentials' share of the sum
//   sqrt(softplus):  dl_k = g_k sigmoid(l_k) / (2 softplus(l_k)), zero elsewhere
//   sigmoid:         dl_k = g_k (1 - s_k) = g_k sigmoid(-l_k), zero elsewhere
// so only the unnormalised softmax needs the whole row of logits.  The forward's own weights stand in
// for the scores, so nothing divides by a sum that may underflow.  The selection itself (and with it
// e_score_correction_bias) has no gradient.
// One warp per token, 16-byte accesses where E is a multiple of four.  16384 tokens, K = 6, fp32, from HBM: 64, 256 and
// 512 experts 7.0, 10.1 and 14.7 us (9.6, 35 and 68 MB), renormalised 4.7, 6.2 and 8.2: the bytes at 7 TB/s behind about
// 5 us (4) of one token's loads, reductions and stores after one another; sqrt(softplus), normalised, 256 experts 5.5, sigmoid
// to bf16 4.6 of 1.2 for the bytes (calls in a row); a few tokens 1.7 us, the launch.
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

// Value i of a lane is expert V * lane + 32 * V * (i / V) + i % V: V = 4 where rows are whole groups of four
// (16-byte accesses), else 1.  PER: values per lane.
// L: type of the logits.  FN: moe_score_fn; one kernel for all three took 6.3 us instead of 5.5 for 16384 x 256 sqrt(softplus),
// renormalised.  whole: softmax as it is; told apart from !renorm by the caller, not here: where the compiler knows that one
// is the other's opposite, it makes two paths of the kernel, and 5.0 us (softmax, renormalised) become 5.5.
template <class T, class L, int PER, int V, int FN>
__global__ void __launch_bounds__(kGradWarps * 32) route_grad_kernel(const typename L::raw* __restrict__ logits, long long ldl,
                                                                     const int32_t* __restrict__ ids,
                                                                     const float* __restrict__ w,
                                                                     const float* __restrict__ dw, int T_, int E, int K,
                                                                     int renorm, int whole, float over_scale,
                                                                     typename T::raw* __restrict__ out, long long ldo,
                                                                     uint32_t* status) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int t = blockIdx.x * kGradWarps + warp;
  grid_dependency_wait();
  grid_launch_dependents();
  if (t >= T_) return;
  constexpr bool softmax = FN == 0;
  const typename L::raw* lrow = logits + t * ldl;
  typename T::raw* orow = out + t * ldo;
  const bool dense = FN == 0 && whole;
  float p[PER];
#pragma unroll
  for (int i = 0; i < PER; i += V) {
    const int e = V * lane + 32 * i;
    if constexpr (V == 4) {
      typename L::raw q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) p[i + j] = -INFINITY;
      if (dense && e < E) {
        if constexpr (sizeof(q) == 16) {
          const uint4 u = __ldg(reinterpret_cast<const uint4*>(lrow + e));
          memcpy(q, &u, 16);
        } else {
          const uint2 u = __ldg(reinterpret_cast<const uint2*>(lrow + e));
          memcpy(q, &u, 8);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) p[i + j] = L::to_f(q[j]);
      }
    } else {
      p[i] = dense && e < E ? L::to_f(__ldg(lrow + e)) : -INFINITY;
    }
  }
  int id = -1;
  float wk = 0.f, dk = 0.f, lk = 0.f;
  if (lane < K) {
    id = __ldg(ids + static_cast<size_t>(t) * K + lane);
    wk = __ldg(w + static_cast<size_t>(t) * K + lane);
    dk = __ldg(dw + static_cast<size_t>(t) * K + lane);
    if (id < 0 || id >= E) {
      record_error(status, kDevErrIndex);
      id = -1;
      wk = dk = 0.f;
    } else if (dense || !softmax) {
      lk = L::to_f(__ldg(lrow + id));
    }
  }
  float g = wk * dk;
  if (renorm) {
    float c = 0.f;
    for (int j = 0; j < K; ++j) c = fmaf(__shfl_sync(0xffffffffu, wk, j), dk - __shfl_sync(0xffffffffu, dk, j), c);
    g = id >= 0 ? wk * (c * over_scale) : 0.f;
  }
  // p becomes the row's -p_e sum_j g_j (dense) or zeros
  float total = 0.f, sum = 0.f, pk = 0.f, not_k = 1.f;      // pk, not_k: of the lane's selected expert, p and 1 - p
  if (dense) {
    float lmax = -INFINITY;
    total = g;
#pragma unroll
    for (int i = 0; i < PER; ++i) lmax = fmaxf(lmax, p[i]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      total += __shfl_xor_sync(0xffffffffu, total, off);
      lmax = fmaxf(lmax, __shfl_xor_sync(0xffffffffu, lmax, off));
    }
    const bool nothing = lmax == -INFINITY;               // a row of masked experts alone: no probability at all
    if (nothing) lmax = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      p[i] = expf(p[i] - lmax);
      sum += V * lane + 32 * (i / V * V) + i % V < E ? p[i] : 0.f;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (nothing) sum = 1.f;
    if (id >= 0) pk = expf(lk - lmax) / sum;
    not_k = 1.f - pk;
    if (__any_sync(0xffffffffu, pk > 0.5f)) {
      // one selected expert has more than all others: its exponential is the only one that is 1
      // (a second pass over the row for such tokens alone: with 256 experts 10.1 us, 10.6 where every token is one; leaving
      // one largest term out of every row's sum from the start 10.6 always)
      float rest = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) rest += p[i] < 1.f ? p[i] : 0.f;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, off);
      if (pk > 0.5f) not_k = rest / sum;
    }
  }
#pragma unroll
  for (int i = 0; i < PER; i += V) {
    const int e = V * lane + 32 * i;
    if (e >= E) continue;
#pragma unroll
    for (int j = 0; j < V; ++j) p[i + j] = dense ? -(p[i + j] / sum) * total : 0.f;
    if constexpr (V == 4) {
      typename T::raw o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = T::from_f(p[i + j]);
      if constexpr (sizeof(o) == 16) {
        uint4 u;
        memcpy(&u, o, 16);
        *reinterpret_cast<uint4*>(orow + e) = u;
      } else {
        uint2 u;
        memcpy(&u, o, 8);
        *reinterpret_cast<uint2*>(orow + e) = u;
      }
    } else {
      orow[e] = T::from_f(p[i]);
    }
  }
  // an expert named twice gets both terms, from its first slot
  float mine = 0.f, others = 0.f;
  bool first = id >= 0;
  for (int k = 0; k < K; ++k) {
    const int ik = __shfl_sync(0xffffffffu, id, k);
    const float gk = __shfl_sync(0xffffffffu, g, k);
    if (ik == id) {
      mine += gk;
      if (k < lane) first = false;
    } else {
      others += gk;
    }
  }
  __syncwarp();                                     // the row is written before its selected entries
  if (first) {
    float v = mine;
    if (FN == 1)
      v = 0.5f * mine * sigmoid_over_softplus(lk);
    else if (FN == 2)
      v = mine / (1.f + expf(lk));
    else if (dense)
      v = not_k * mine - pk * others;
    orow[id] = T::from_f(v);
  }
}

struct GradArgs {
  const void* logits;
  long long ldl;
  const int32_t* ids;
  const float *w, *dw;
  int T, E, K, fn, renorm;
  float over_scale;
  void* out;
  long long ldo;
  uint32_t* status;
};

template <class T, class L, int PER, int V>
cudaError_t route_grad_launch(const GradArgs& a, cudaStream_t stream) {
  const auto go = [&](auto kernel) {
    return launch_pdl(kernel, dim3((a.T - 1) / kGradWarps + 1), dim3(kGradWarps * 32), 0, stream,
                      static_cast<const typename L::raw*>(a.logits), a.ldl, a.ids, a.w, a.dw, a.T, a.E, a.K, a.renorm,
                      a.fn == 0 && !a.renorm, a.over_scale, static_cast<typename T::raw*>(a.out), a.ldo, a.status);
  };
  if (a.fn == 0) return go(route_grad_kernel<T, L, PER, V, 0>);
  if (a.fn == 1) return go(route_grad_kernel<T, L, PER, V, 1>);
  return go(route_grad_kernel<T, L, PER, V, 2>);
}

// Four logits (and gradients) at a time where every row starts on a boundary of four.
template <class T, class L>
cudaError_t route_grad_by_size(const GradArgs& a, cudaStream_t q) {
  const int per = (a.E + 31) / 32;
  const auto fours = [&](const void* p, long long ld, size_t size) {
    return reinterpret_cast<uintptr_t>(p) % (4 * size) == 0 && (a.T <= 1 || ld % 4 == 0);
  };
  if (a.E % 4 == 0 && fours(a.logits, a.ldl, sizeof(typename L::raw)) && fours(a.out, a.ldo, sizeof(typename T::raw))) {
    if (per <= 4) return route_grad_launch<T, L, 4, 4>(a, q);
    if (per <= 8) return route_grad_launch<T, L, 8, 4>(a, q);
    if (per <= 16) return route_grad_launch<T, L, 16, 4>(a, q);
    return route_grad_launch<T, L, 32, 4>(a, q);
  }
  if (per <= 4) return route_grad_launch<T, L, 4, 1>(a, q);
  if (per <= 16) return route_grad_launch<T, L, 16, 1>(a, q);
  return route_grad_launch<T, L, 32, 1>(a, q);
}

}  // namespace

cudaError_t launch_route_grad(int ldt, RowsView logits, const int32_t* ids, const float* w, const float* dw, int T, int E,
                              int K, int fn, int renorm, float scale, int dt, RowsView out, uint32_t* status,
                              cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  const GradArgs a{logits.ptr, logits.ld, ids, w, dw, T, E, K, fn, renorm, 1.f / scale, out.ptr, out.ld, status};
  if (ldt == kF32) {
    if (dt == kBf16) return route_grad_by_size<Bf16Elem, F32Elem>(a, stream);
    if (dt == kF16) return route_grad_by_size<F16Elem, F32Elem>(a, stream);
    return route_grad_by_size<F32Elem, F32Elem>(a, stream);
  }
  if (dt == kBf16) return route_grad_by_size<Bf16Elem, Bf16Elem>(a, stream);
  return route_grad_by_size<F16Elem, F16Elem>(a, stream);
}

}  // namespace moe
