// Routing from logits: scores, a bias for balance, groups of experts, top-K and weights.
//
//   s_e   = softmax(l)_e, sqrt(softplus(l_e)) or sigmoid(l_e);   key_e = s_e + b_e
//   group = sum of its one or two largest keys; the topk_groups best groups stay (ties: the lower group)
//   ids   = the K largest keys of their experts, descending (ties: the lower expert)
//   w_k   = scale * s_k (/ sum_j s_j)
// NaN keys count as -infinity, so the ids are valid and different whatever the logits hold.
//
// One warp per token.  Its lanes are split over the groups, L = 2^i <= 32 / groups to each, and a lane holds experts
// sub + L i of its group.
//
// The choice does not depend on how a score is evaluated: a key in fp32 is off by a known bound, and a token where two
// keys (or groups) that decide are closer than that is done again in 64 bits.  Two experts of equal logit and bias are
// an exact tie and need no second look; without a bias keys go by the logits themselves, which all scores rise with.
#include "rows.cuh"

namespace moe {

namespace {

constexpr int kSelectWarps = 8;
constexpr unsigned kAll = 0xffffffffu;

struct SelectArgs {
  const void* logits;
  long long ld;
  const float* bias;
  int T, E, K;
  int G, KG, best, fn, renorm;
  int per_group, L;           // experts per group, lanes per group
  float scale;
  int32_t* ids;
  float* w;
};

// In the order of floats as unsigned numbers, none of them 0 (which marks no expert).
__device__ __forceinline__ uint32_t ordered(float k) {
  if (!(k == k)) k = -INFINITY;
  const uint32_t u = __float_as_uint(k + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t o) { return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o); }

// Scores; softmax of a row: lmax its largest logit, sum its exponentials' (a row of -infinities has scores of 0).
struct Scores {
  int fn;
  float lmax, sum;
  __device__ __forceinline__ float operator()(float l) const {
    if (fn == 0) return l == -INFINITY ? 0.f : expf(l - lmax) / sum;
    if (fn == 1) return sqrtf(fmaxf(l, 0.f) + log1pf(expf(-fabsf(l))));
    return 1.f / (1.f + expf(-l));
  }
};
struct Scores64 {
  int fn;
  double lmax, sum;
  __device__ __forceinline__ double operator()(double l) const {
    if (fn == 0) return l == -INFINITY ? 0. : exp(l - lmax) / sum;
    if (fn == 1) return sqrt(fmax(l, 0.) + log1p(exp(-fabs(l))));
    return 1. / (1. + exp(-l));
  }
};

// A token's experts in 64 bits: lane k gets the k-th (the others what was there).
template <class T, int PER>
__device__ __noinline__ int select_exact(const SelectArgs& a, const typename T::raw* row, int id) {
  const int lane = threadIdx.x % 32, g = lane / a.L, sub = lane % a.L;
  Scores64 score{a.fn, -INFINITY, 0.};
  double key[PER];
  if (a.fn == 0) {
    float m = -INFINITY;
    for (int e = lane; e < a.E; e += 32) m = fmaxf(m, T::to_f(row[e]));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, d));
    score.lmax = m;
    for (int e = lane; e < a.E; e += 32) score.sum += exp(static_cast<double>(T::to_f(row[e])) - score.lmax);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) score.sum += __shfl_xor_sync(kAll, score.sum, d);
  }
  double k1 = -INFINITY, k2 = -INFINITY;
  int n = 0;
  for (int i = 0; i < PER; ++i) {
    const int r = sub + a.L * i;
    key[i] = -INFINITY;
    if (g < a.G && r < a.per_group) {
      const int e = g * a.per_group + r;
      const double s = score(T::to_f(row[e]));
      double k = a.bias ? s + a.bias[e] : s;
      if (!(k == k)) k = -INFINITY;
      key[i] = a.bias ? k : static_cast<double>(from_ordered(ordered(T::to_f(row[e]))));
      if (k > k1) {
        k2 = k1;
        k1 = k;
      } else if (k > k2) {
        k2 = k;
      }
      n = i + 1;
    }
  }
  bool open = g < a.G;
  if (a.KG < a.G) {
    for (int d = 1; d < a.L; d <<= 1) {
      const double o1 = __shfl_xor_sync(kAll, k1, d), o2 = __shfl_xor_sync(kAll, k2, d);
      const double lo = fmin(k1, o1), hi2 = fmax(k2, o2);
      k1 = fmax(k1, o1);
      k2 = fmax(lo, hi2);
    }
    double mine = a.best == 2 && a.per_group > 1 ? k1 + k2 : k1;
    if (!(mine == mine)) mine = -INFINITY;
    int rank = 0;
    for (int h = 0; h < a.G; ++h) {
      const double o = __shfl_sync(kAll, mine, h * a.L);
      rank += o > mine || (o == mine && h < g);
    }
    open = open && rank < a.KG;
  }
  unsigned long long taken = 0;
  for (int k = 0; k < a.K; ++k) {
    double bk = 0.;
    int be = 0x7fffffff, bi = -1;
    for (int i = 0; open && i < n; ++i)
      if (!(taken >> i & 1) && (bi < 0 || key[i] > bk)) {
        bk = key[i];
        bi = i;
      }
    if (bi >= 0) be = g * a.per_group + sub + a.L * bi;
    const int mine = be;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const double ok = __shfl_xor_sync(kAll, bk, d);
      const int oe = __shfl_xor_sync(kAll, be, d);
      if (oe != 0x7fffffff && (be == 0x7fffffff || ok > bk || (ok == bk && oe < be))) {
        bk = ok;
        be = oe;
      }
    }
    if (bi >= 0 && mine == be) taken |= 1ull << bi;
    if (lane == k) id = be;
  }
  return id;
}

template <class T, int PER>
__global__ void __launch_bounds__(kSelectWarps * 32) select_kernel(const SelectArgs a) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const long long t = static_cast<long long>(blockIdx.x) * kSelectWarps + warp;
  grid_dependency_wait();
  grid_launch_dependents();
  if (t >= a.T) return;
  const typename T::raw* row = static_cast<const typename T::raw*>(a.logits) + t * a.ld;
  const int g = lane / a.L, sub = lane % a.L;
  float v[PER];
  float lmax = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int r = sub + a.L * i;
    v[i] = g < a.G && r < a.per_group ? T::to_f(row[g * a.per_group + r]) : -INFINITY;
    lmax = fmaxf(lmax, v[i]);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) lmax = fmaxf(lmax, __shfl_xor_sync(kAll, lmax, d));
  Scores score{a.fn, lmax, 0.f};
  if (a.fn == 0) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (g < a.G && sub + a.L * i < a.per_group) score.sum += expf(v[i] - lmax);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) score.sum += __shfl_xor_sync(kAll, score.sum, d);
  }
  // How far the difference of two scores may be off: fp32 exponentials, logarithms, roots and divisions are within
  // two steps of 2^-24 each, eight in all; softmax's sum of PER + 5 additions more, while the difference d of two logits,
  // off by 2^-24 d, is outweighed by e^-d.  Of the largest score, since none is larger.
  const float near = score(lmax) * ((a.fn == 0 ? PER + 8 : 8) * 0x1p-23f);
  uint32_t key[PER];
  float k1 = -INFINITY, k2 = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int r = sub + a.L * i;
    key[i] = 0;
    if (g < a.G && r < a.per_group) {
      float k = v[i];
      if (a.bias || a.KG < a.G) {
        float s = score(v[i]) + (a.bias ? __ldg(a.bias + g * a.per_group + r) : 0.f);
        if (!(s == s)) s = -INFINITY;
        k2 = fmaxf(k2, fminf(k1, s));
        k1 = fmaxf(k1, s);
        if (a.bias) k = s;
      }
      key[i] = ordered(k);
    }
  }
  bool unsure = false, open = true;
  if (a.KG < a.G) {
    for (int d = 1; d < a.L; d <<= 1) {
      const float o1 = __shfl_xor_sync(kAll, k1, d), o2 = __shfl_xor_sync(kAll, k2, d);
      k2 = fmaxf(fminf(k1, o1), fmaxf(k2, o2));
      k1 = fmaxf(k1, o1);
    }
    const bool two = a.best == 2 && a.per_group > 1;
    float mine = two ? k1 + k2 : k1;
    if (!(mine == mine)) mine = -INFINITY;
    float size = fminf(fabsf(k1), 3e38f) * 0x1p-23f;
    if (two) size += fminf(fabsf(k2), 3e38f) * 0x1p-23f;
    size += near;
    int surely = 0, maybe = 0;        // groups that are better
    for (int h = 0; h < a.G; ++h) {
      const float o = __shfl_sync(kAll, mine, h * a.L), os = __shfl_sync(kAll, size, h * a.L);
      if (h == g) continue;
      const bool better = o > mine || (o == mine && h < g), close = fabsf(o - mine) <= size + os;
      surely += better && !close;
      maybe += better || close;
    }
    open = maybe < a.KG;
    unsure = g < a.G && !open && surely < a.KG;
    unsure = __any_sync(kAll, unsure);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (!open) key[i] = 0;
  }
  // lane k keeps the k-th largest key; every lane ends with the first that is left out (key 0 where there is none)
  int id = 0, won = 0;
  uint32_t mk = 0, best = 0;
  for (int k = 0; k <= a.K; ++k) {
    uint32_t b = 0;
    int bi = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (key[i] > b) {
        b = key[i];
        bi = i;
      }
    best = __reduce_max_sync(kAll, b);
    const int e = b == best && best ? g * a.per_group + sub + a.L * bi : 0x7fffffff;
    won = static_cast<int>(__reduce_min_sync(kAll, static_cast<uint32_t>(e)));
    if (lane == k) {
      id = won;
      mk = best;
    }
    if (e == won && best) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (i == bi) key[i] = 0;
    }
  }
  if (a.bias) {
    uint32_t nk = __shfl_down_sync(kAll, mk, 1);
    int nid = __shfl_down_sync(kAll, id, 1);
    if (lane == a.K - 1) {
      nk = best;
      nid = won;
    }
    if (lane < a.K && nk != 0) {
      const float f = from_ordered(mk), nf = from_ordered(nk);
      const float tol = near + (fminf(fabsf(f), 3e38f) + fminf(fabsf(nf), 3e38f)) * 0x1p-23f;
      if (f - nf <= tol) unsure = unsure || T::to_f(row[id]) != T::to_f(row[nid]) || __ldg(a.bias + id) != __ldg(a.bias + nid);
    }
    unsure = __any_sync(kAll, unsure);
  }
  if (unsure) id = select_exact<T, PER>(a, row, id);
  float s = lane < a.K ? score(T::to_f(row[id])) : 0.f;
  if (a.renorm) {
    float sum = s;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
    s = sum == 0.f ? 0.f : s / sum;
  }
  if (lane < a.K) {
    a.ids[t * a.K + lane] = id;
    a.w[t * a.K + lane] = s * a.scale;
  }
}

template <class T, int PER>
cudaError_t select_launch(const SelectArgs& a, cudaStream_t stream) {
  return launch_pdl(select_kernel<T, PER>, dim3((a.T + kSelectWarps - 1) / kSelectWarps), dim3(kSelectWarps * 32), 0, stream, a);
}

template <class T>
cudaError_t select_by_size(const SelectArgs& a, cudaStream_t stream) {
  const int per = (a.per_group + a.L - 1) / a.L;
  if (per <= 2) return select_launch<T, 2>(a, stream);
  if (per <= 4) return select_launch<T, 4>(a, stream);
  if (per <= 8) return select_launch<T, 8>(a, stream);
  if (per <= 16) return select_launch<T, 16>(a, stream);
  if (per <= 32) return select_launch<T, 32>(a, stream);
  return select_launch<T, 64>(a, stream);
}

}  // namespace

cudaError_t launch_select(int ldt, RowsView logits, const float* bias, int T, int E, int K, const SelectRule& rule,
                          int32_t* ids, float* w, cudaStream_t stream) {
  SelectArgs a{};
  a.logits = logits.ptr;
  a.ld = logits.ld;
  a.bias = bias;
  a.T = T;
  a.E = E;
  a.K = K;
  a.KG = rule.topk_groups;
  a.G = rule.topk_groups < rule.groups ? rule.groups : 1;     // all groups used: one group of all experts
  if (a.G == 1) a.KG = 1;
  a.best = rule.best;
  a.fn = rule.fn;
  a.renorm = rule.renorm;
  a.scale = rule.scale;
  a.per_group = E / a.G;
  a.L = 32;
  while (a.L * a.G > 32) a.L /= 2;
  a.ids = ids;
  a.w = w;
  if (ldt == kBf16) return select_by_size<Bf16Elem>(a, stream);
  if (ldt == kF16) return select_by_size<F16Elem>(a, stream);
  return select_by_size<F32Elem>(a, stream);
}

}  // namespace moe
