// Routing from logits: scores, a bias for balance, groups of experts, top-K and weights.
//
//   s_e   = softmax(l)_e, sqrt(softplus(l_e)) or sigmoid(l_e);   key_e = s_e + b_e
//   group = sum of its one or two largest keys; the topk_groups best groups stay (ties: the lower group)
//   ids   = the K largest keys of their experts, descending (ties: the lower expert)
//   w_k   = scale * s_k (/ sum_j s_j)
// NaN keys count as -infinity, so the ids are valid and different whatever the logits hold.
//
// One warp per token.  Its lanes are split over the groups, L = 2^i <= 32 / groups to each; a lane holds experts
// V (sub + L i) .. + V - 1 of its group, V = 4 where rows and groups are whole fours (one load each).
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
  int per_group, L, log_l;    // experts per group, lanes per group
  float scale;
  int32_t* ids;
  float* w;
};

// In the order of floats as unsigned numbers, none of them 0 (which marks no expert).
__device__ __forceinline__ uint32_t ordered(float k) {
  const int u = __float_as_int(fmaxf(k, -INFINITY) + 0.f);            // (NaN to -infinity, -0 to 0)
  return static_cast<uint32_t>(u) ^ (static_cast<uint32_t>(u >> 31) | 0x80000000u);
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
// The same, for keys: fast exponentials and divisions for softmax (over: 1 / sum) and sigmoid.
struct FastScores {
  int fn;
  float lmax, over;
  __device__ __forceinline__ float operator()(float l) const {
    if (fn == 0) return l == -INFINITY ? 0.f : __expf(l - lmax) * over;
    if (fn == 1) return sqrtf(fmaxf(l, 0.f) + log1pf(expf(-fabsf(l))));
    return __fdividef(1.f, 1.f + __expf(-l));
  }
  // How far the difference of two scores may be off at most.  __expf(x) is within 2 + 1.2 |x| steps of 2^-23, the division
  // within two.  Sigmoid: 1 / (1 + e^-l) is off by s (4.5 + 1.2 max(-l, 0)) 2^-23, which rises with l.  Softmax: the
  // difference of two logits d adds |d| / 2 steps, all outweighed by e^-d: two steps of the largest score, and the sum's PER
  // + 5 additions.  Square root, logarithm: accurate ones, eight steps.  (Scores below 2^-126 come out as 0.)
  template <int PER>
  __device__ __forceinline__ float apart() const {
    const float steps = fn == 0 ? PER + 16.f : fn == 1 ? 16.f : 16.f + 4.f * fmaxf(-lmax, 0.f);
    return (*this)(lmax) * (steps * 0x1p-23f) + 0x1p-120f;
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

// V values from p on (zeros where there are none).
template <class T, int V>
__device__ __forceinline__ void load_values(const typename T::raw* p, bool there, float (&v)[V]) {
  if constexpr (V == 4) {
    typename T::raw r[4];
    if constexpr (sizeof(r) == 16) {
      const uint4 u = there ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
      memcpy(r, &u, 16);
    } else {
      const uint2 u = there ? __ldg(reinterpret_cast<const uint2*>(p)) : make_uint2(0, 0);
      memcpy(r, &u, 8);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = T::to_f(r[j]);
  } else {
    v[0] = there ? T::to_f(__ldg(p)) : 0.f;
  }
}

// A lane's largest two keys (0: none) and where they are.
struct Top2 {
  uint32_t k1, k2;
  int i1, i2;
  __device__ __forceinline__ void add(uint32_t k, int i) {
    const bool first = k > k1, second = k > k2;
    k2 = first ? k1 : second ? k : k2;
    i2 = first ? i1 : second ? i : i2;
    k1 = first ? k : k1;
    i1 = first ? i : i1;
  }
};

template <class T, int PER, int V>
__global__ void __launch_bounds__(kSelectWarps * 32) select_kernel(const SelectArgs a) {
  const int lane = threadIdx.x % 32, g = lane >> a.log_l, sub = lane & (a.L - 1);
  grid_dependency_wait();
  grid_launch_dependents();
  const bool used = g < a.G;
  const int e0 = used ? g * a.per_group : 0;
  // the lane's i-th expert is e0 + at(i)
  const auto at = [&](int i) { return V * (sub + a.L * (i / V)) + i % V; };
  float bias[PER];
#pragma unroll
  for (int i = 0; i < PER; i += V) {
    const bool there = a.bias && used && at(i) < a.per_group;
#pragma unroll
    for (int j = 0; j < V; ++j) bias[i + j] = there ? __ldg(a.bias + e0 + at(i) + j) : 0.f;
  }
  for (long long t = static_cast<long long>(blockIdx.x) * kSelectWarps + threadIdx.x / 32; t < a.T; t += gridDim.x * kSelectWarps) {
    const typename T::raw* row = static_cast<const typename T::raw*>(a.logits) + t * a.ld;
    float v[PER];
#pragma unroll
    for (int i = 0; i < PER; i += V) {
      float f[V];
      load_values<T, V>(row + e0 + at(i), used && at(i) < a.per_group, f);
#pragma unroll
      for (int j = 0; j < V; ++j) v[i + j] = f[j];
    }
    uint32_t key[PER], top = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      key[i] = used && at(i) < a.per_group ? ordered(v[i]) : 0;
      top = max(top, key[i]);
    }
    const float lmax = from_ordered(__reduce_max_sync(kAll, top));
    float sum = 1.f;
    if (a.fn == 0) {
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (key[i] && v[i] != -INFINITY) sum += __expf(v[i] - lmax);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
    }
    const FastScores fast{a.fn, lmax, 1.f / sum};
    const float near = fast.template apart<PER>();
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (key[i]) key[i] = ordered(fast(v[i]) + bias[i]);
    }
    Top2 head{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < PER; ++i) head.add(key[i], i);
    bool unsure = false;
    int left = 0;                     // the lane's experts that may still be taken
#pragma unroll
    for (int i = 0; i < PER; ++i) left += key[i] != 0;
    if (a.KG < a.G) {
      uint32_t k1 = head.k1, k2 = head.k2;
      for (int d = 1; d < a.L; d <<= 1) {
        const uint32_t o1 = __shfl_xor_sync(kAll, k1, d), o2 = __shfl_xor_sync(kAll, k2, d);
        k2 = max(min(k1, o1), max(k2, o2));
        k1 = max(k1, o1);
      }
      // what the group is worth, and how far that may be off: two scores and additions
      float worth = -INFINITY, size = 0.f;
      if (used) {
        const float f1 = from_ordered(k1), f2 = from_ordered(k2);
        worth = a.bias ? f1 : fast(f1);
        size = fabsf(worth);
        if (a.best == 2 && k2) {
          const float w2 = a.bias ? f2 : fast(f2);
          worth += w2;
          size += fabsf(w2);
        }
        size = size <= 3e38f ? size : 0.f;       // (an infinite worth is exact)
      }
      uint32_t mine = used && sub == 0 ? ordered(worth) : 0;
      const float tol = 2.f * near + __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(size))) * 0x1p-21f;
      unsigned open = 0;
      float last = 0.f;
      for (int k = 0; k < a.KG; ++k) {
        const uint32_t best = __reduce_max_sync(kAll, mine);
        const int who = __ffs(__ballot_sync(kAll, mine == best)) - 1;      // the lowest group of equals
        open |= 1u << who;
        if (lane == who) mine = 0;
        last = from_ordered(best);
      }
      unsure = last - from_ordered(__reduce_max_sync(kAll, mine)) <= tol;
      if (!(open >> (g << a.log_l) & 1)) {
        head = Top2{0, 0, 0, 0};
        left = 0;
      }
    }
    // lane k keeps the k-th largest key; every lane ends with the first that is left out (key 0 where there is none)
    int id = 0, won = 0;
    uint32_t mk = 0, best = 0;
    unsigned long long taken = 0;
    for (int k = 0; k <= a.K; ++k) {
      best = __reduce_max_sync(kAll, head.k1);
      const int e = head.k1 == best ? e0 + at(head.i1) : 0x7fffffff;
      won = static_cast<int>(__reduce_min_sync(kAll, static_cast<uint32_t>(e)));
      if (lane == k) {
        id = won;
        mk = best;
      }
      if (e == won && best) {
        taken |= 1ull << head.i1;
        --left;
        head.k1 = head.k2;
        head.i1 = head.i2;
        head.k2 = 0;
        if (head.k1 == 0 && left > 0) {
#pragma unroll
          for (int i = 0; i < PER; ++i)
            if (!(taken >> i & 1)) head.add(key[i], i);
        }
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
        if (f - nf <= tol)
          unsure = unsure || T::to_f(row[id]) != T::to_f(row[nid]) || __ldg(a.bias + id) != __ldg(a.bias + nid);
      }
    }
    if (__any_sync(kAll, unsure)) id = select_exact<T, PER>(a, row, id);
    const Scores score{a.fn, lmax, sum};
    float s = lane < a.K ? score(T::to_f(row[id])) : 0.f;
    if (a.renorm) {
      float all = s;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) all += __shfl_xor_sync(kAll, all, d);
      s = all == 0.f ? 0.f : s / all;
    }
    if (lane < a.K) {
      a.ids[t * a.K + lane] = id;
      a.w[t * a.K + lane] = s * a.scale;
    }
  }
}

template <class T, int PER, int V>
cudaError_t select_launch(const SelectArgs& a, cudaStream_t stream) {
  const long long ctas = (static_cast<long long>(a.T) + kSelectWarps - 1) / kSelectWarps, most = 8LL * num_sms();
  return launch_pdl(select_kernel<T, PER, V>, dim3(static_cast<unsigned>(ctas < most ? ctas : most)), dim3(kSelectWarps * 32), 0,
                    stream, a);
}

template <class T>
cudaError_t select_by_size(const SelectArgs& a, cudaStream_t stream) {
  const size_t four = 4 * sizeof(typename T::raw);
  if (a.per_group % 4 == 0 && reinterpret_cast<uintptr_t>(a.logits) % four == 0 && (a.T <= 1 || a.ld % 4 == 0)) {
    const int per = (a.per_group + 4 * a.L - 1) / (4 * a.L) * 4;
    if (per <= 4) return select_launch<T, 4, 4>(a, stream);
    if (per <= 8) return select_launch<T, 8, 4>(a, stream);
    if (per <= 16) return select_launch<T, 16, 4>(a, stream);
    if (per <= 32) return select_launch<T, 32, 4>(a, stream);
    return select_launch<T, 64, 4>(a, stream);
  }
  const int per = (a.per_group + a.L - 1) / a.L;
  if (per <= 8) return select_launch<T, 8, 1>(a, stream);
  if (per <= 32) return select_launch<T, 32, 1>(a, stream);
  return select_launch<T, 64, 1>(a, stream);
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
  a.log_l = 5;
  while ((a.G << a.log_l) > 32) --a.log_l;
  a.L = 1 << a.log_l;
  a.ids = ids;
  a.w = w;
  if (ldt == kBf16) return select_by_size<Bf16Elem>(a, stream);
  if (ldt == kF16) return select_by_size<F16Elem>(a, stream);
  return select_by_size<F32Elem>(a, stream);
}

}  // namespace moe
