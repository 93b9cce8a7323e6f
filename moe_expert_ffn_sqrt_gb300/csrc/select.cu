// Routing from logits: scores, a bias for balance, groups of experts, top-K and weights.
//
//   s_e   = softmax(l)_e, sqrt(softplus(l_e)) or sigmoid(l_e);   key_e = s_e + b_e
//   group = sum of its one or two largest keys; the topk_groups best groups stay (ties: the lower group)
//   ids   = the K largest keys of their experts, descending (ties: the lower expert)
//   w_k   = scale * s_k (/ sum_j s_j)
// NaN keys count as -infinity, so the ids are valid and different whatever the logits hold.
//
// One warp per token.  Its lanes are split over the groups, L = 2^i <= 32 / groups to each; a lane holds experts
// V (sub + L i) .. + V - 1 of its group, V = 4 where rows and groups are whole fours (one load each).  The K + 1 largest of
// the lanes' largest two keys give a bound that the K + 1 largest keys reach; the few keys that do (in shared memory, one to
// a lane) are ranked by comparing all of them.  Where more than 32 do (many equal keys), K + 1 rounds of a maximum over the
// warp instead.
//
// The choice does not depend on how a score is evaluated: a key in fp32 is off by a known bound, and where two keys (or
// groups) that decide are closer than that, the keys that are near are evaluated in 64 bits, one to a lane.  Two experts of
// equal logit and bias are an exact tie and need no second look, unless they are the last one in and the first one out and a
// third, other key is near them.  Without a bias keys go by the logits themselves, which all scores rise with.
//
// 16384 tokens of 256 experts in 8 groups, 4 of them used, K = 6: sigmoid and bias 19.1 us, of 2.6 for the bytes; sqrt(softplus)
// 27.5 (an accurate exponential, logarithm and root for every expert), softmax 29.0 (the row's sum); without a bias, where keys
// are the logits, 16.0, 18.0 and 22.9.  One group, K = 8: 16.5, 24.7 and 26.8, without a bias 12.9, 14.3 and 15.6.  The
// instructions bound it, 861 a token (sigmoid), with the schedulers busy for 60% (64 registers, 32 warps per SM; 80 registers
// 20.9 us, five CTAs of 8 warps 21.4).  The second looks take 0.2 us of it.  K rounds of a maximum instead of the ranking took
// 43 us.  8 tokens: 3.5 us, one warp's chain.  Where all experts' keys are alike (say a row of padding, a zero bias and
// groups) the groups' order takes a 64-bit evaluation of every expert, some 10 us for the warps that have such tokens.
#include "rows.cuh"

namespace moe {

namespace {

constexpr int kSelectWarps = 4, kSelectCtas = 8;       // of a CTA; CTAs per SM that are there at a time
constexpr unsigned kAll = 0xffffffffu;
constexpr int kNone = 0x7fffffff;

struct SelectArgs {
  const uint8_t* logits;      // rows of type dt, row_bytes apart
  long long row_bytes;
  int dt;
  const float* bias;
  int T, E, K;
  int G, KG, best, renorm;
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
// 0 for what is not finite
__device__ __forceinline__ float size_of(float f) {
  const float a = fabsf(f);
  return a <= 3.402823466e38f ? a : 0.f;
}

// sqrt(softplus(l)).  Far below zero it is e^(l/2) (1 - e^l / 4 + ..), e^-20 / 4 < 2^-30: a normal number down to l = -174,
// where e^l is subnormal from -87 on and 0 from -104 on.
__device__ __forceinline__ float root_softplus(float l) {
  const bool far = l < -20.f;
  const float e = expf(far ? 0.5f * l : -fabsf(l));
  return far ? e : sqrtf(fmaxf(l, 0.f) + log1pf(e));
}

// Scores (FN: moe_score_fn); softmax of a row: lmax its largest logit, sum its exponentials' (a masked expert, a logit of
// -infinity, has 0, in a row of nothing else too).
template <int FN>
struct Scores {
  float lmax, sum;
  __device__ __forceinline__ float operator()(float l) const {
    if (FN == 0) {
      // (d is rounded by up to |d| 2^-24, which would be the exponential's relative error: it gets the rest back)
      const float d = l - lmax, back = d - l, rest = (l - (d - back)) - (lmax + back), e = expf(d);
      return l == -INFINITY ? 0.f : (e > 0.f ? fmaf(e, rest, e) : e) / sum;       // (d may be -infinity: no rest)
    }
    if (FN == 1) return root_softplus(l);
    return 1.f / (1.f + expf(-l));
  }
};
// The same, for keys: fast exponentials and divisions for softmax (over: 1 / sum) and sigmoid.
template <int FN>
struct FastScores {
  float lmax, over;
  __device__ __forceinline__ float operator()(float l) const {
    if (FN == 0) return l == -INFINITY ? 0.f : __expf(l - lmax) * over;
    if (FN == 1) return root_softplus(l);
    float e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(l * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
    return s;
  }
  // How far the difference of two scores may be off at most.  Exponentials of x are within 2 + 1.5 |x| steps of 2^-23,
  // reciprocals and products within one or two.  Sigmoid: 1 / (1 + e^-l) is off by s (5 + 1.5 max(-l, 0)) 2^-23, at most
  // eight steps (s is below e^l).  Softmax: the difference of two logits d adds |d| / 2 steps, all outweighed by e^-d: two
  // steps of the largest score, and the sum's PER + 5 additions.  Square root, logarithm: accurate ones, eight steps of the
  // largest score.  (Scores below 2^-126 come out as 0.)
  template <int PER>
  __device__ __forceinline__ float apart() const {
    if (FN == 2) return 0x1p-19f;
    return (*this)(lmax) * ((FN == 0 ? PER + 16.f : 16.f) * 0x1p-23f) + 0x1p-120f;
  }
};
template <int FN>
struct Scores64 {
  double lmax, sum;
  __device__ __forceinline__ double operator()(double l) const {
    if (FN == 0) return l == -INFINITY ? 0. : exp(l - lmax) / sum;
    if (FN == 1) return sqrt(fmax(l, 0.) + log1p(exp(-fabs(l))));
    return 1. / (1. + exp(-l));
  }
};

__device__ __forceinline__ float logit(const SelectArgs& a, const uint8_t* row, int e) {
  if (a.dt == kF32) return __ldg(reinterpret_cast<const float*>(row) + e);
  const uint16_t u = __ldg(reinterpret_cast<const uint16_t*>(row) + e);
  return a.dt == kBf16 ? Bf16Elem::to_f(u) : F16Elem::to_f(u);
}
// V logits from expert e on (zeros where there are none).
template <int V>
__device__ __forceinline__ void logits(const SelectArgs& a, const uint8_t* row, int e, bool there, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = there ? logit(a, row, e) : 0.f;
  } else if (a.dt == kF32) {
    const float4 f = there ? __ldg(reinterpret_cast<const float4*>(row) + e / 4) : make_float4(0.f, 0.f, 0.f, 0.f);
    v[0] = f.x;
    v[1] = f.y;
    v[2] = f.z;
    v[3] = f.w;
  } else {
    const uint2 u = there ? __ldg(reinterpret_cast<const uint2*>(row) + e / 4) : make_uint2(0, 0);
    const uint16_t r[4] = {static_cast<uint16_t>(u.x), static_cast<uint16_t>(u.x >> 16), static_cast<uint16_t>(u.y),
                           static_cast<uint16_t>(u.y >> 16)};
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = a.dt == kBf16 ? Bf16Elem::to_f(r[j]) : F16Elem::to_f(r[j]);
  }
}

// Scores of the row in 64 bits (softmax: its largest logit and sum).
template <int FN>
__device__ __forceinline__ Scores64<FN> scores64(const SelectArgs& a, const uint8_t* row, float lmax) {
  Scores64<FN> s{lmax, 0.};
  if (FN == 0) {
    for (int e = threadIdx.x % 32; e < a.E; e += 32) {
      const float l = logit(a, row, e);
      if (l != -INFINITY) s.sum += exp(static_cast<double>(l) - s.lmax);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s.sum += __shfl_xor_sync(kAll, s.sum, d);
  }
  return s;
}
__device__ __forceinline__ double clean(double k) { return k == k ? k : -INFINITY; }

// A token's experts all in 64 bits, K rounds: lane k gets the k-th (the others what was there).  For rows where many keys
// are near one another.
template <int FN, int PER>
__device__ __noinline__ int select_all64(const SelectArgs& a, const uint8_t* row, float lmax, int id) {
  const int lane = threadIdx.x % 32, g = lane >> a.log_l, sub = lane & (a.L - 1);
  const Scores64<FN> score = scores64<FN>(a, row, lmax);
  double key[PER];
  double k1 = -INFINITY, k2 = -INFINITY;
  int n = 0;
  for (int i = 0; i < PER; ++i) {
    const int r = sub + a.L * i;
    key[i] = -INFINITY;
    if (g < a.G && r < a.per_group) {
      const int e = g * a.per_group + r;
      const double l = logit(a, row, e), s = score(l), k = clean(a.bias ? s + a.bias[e] : s);
      key[i] = a.bias ? k : clean(l);
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
    const double mine = clean(a.best == 2 && a.per_group > 1 ? k1 + k2 : k1);
    int rank = 0;
    for (int h = 0; h < a.G; ++h) {
      const double o = __shfl_sync(kAll, mine, h << a.log_l);
      rank += o > mine || (o == mine && h < g);
    }
    open = open && rank < a.KG;
  }
  unsigned long long taken = 0;
  for (int k = 0; k < a.K; ++k) {
    double bk = 0.;
    int be = kNone, bi = -1;
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
      if (oe != kNone && (be == kNone || ok > bk || (ok == bk && oe < be))) {
        bk = ok;
        be = oe;
      }
    }
    if (bi >= 0 && mine == be) taken |= 1ull << bi;
    if (lane == k) id = be;
  }
  return id;
}

// A token's weights from 64-bit scores (lane k has its k-th expert): for tokens with a score below kTiny.  fp32 has few bits
// for those, or none, and they count where all of a token's are as small, or the scale is large.
constexpr float kTiny = 0x1p-100f;
template <int FN>
__device__ __noinline__ void weights64(const SelectArgs& a, long long t, float lmax, int id) {
  const int lane = threadIdx.x % 32;
  const uint8_t* row = a.logits + t * a.row_bytes;
  const float l = lane < a.K ? logit(a, row, id) : -INFINITY;
  if (!__any_sync(kAll, l != -INFINITY)) return;          // masked experts all: zeros
  const Scores64<FN> score = scores64<FN>(a, row, lmax);
  double s = lane < a.K ? score(l) : 0.;
  if (a.renorm) {
    double all = s;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) all += __shfl_xor_sync(kAll, all, d);
    s = all == 0. ? 0. : s / all;
  }
  if (lane < a.K) a.w[t * a.K + lane] = static_cast<float>(s * a.scale);
}

template <int FN, int PER, int V>
__global__ void __launch_bounds__(kSelectWarps * 32, PER <= 8 ? kSelectCtas : 1) select_kernel(const SelectArgs a) {
  __shared__ uint2 s_near[kSelectWarps][34];           // experts that are near (id, key), then the chosen ones in order
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane >> a.log_l, sub = lane & (a.L - 1);
  uint2* list = s_near[warp];
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
  for (long long t = static_cast<long long>(blockIdx.x) * kSelectWarps + warp; t < a.T; t += gridDim.x * kSelectWarps) {
    const uint8_t* row = a.logits + t * a.row_bytes;
    float v[PER];
    uint32_t key[PER], top = 0;
#pragma unroll
    for (int i = 0; i < PER; i += V) {
      const bool there = used && at(i) < a.per_group;
      float f[V];
      logits<V>(a, row, e0 + at(i), there, f);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        v[i + j] = f[j];
        key[i + j] = there;
        if (FN != 2 || !a.bias) {
          if (there) key[i + j] = ordered(f[j]);
          top = max(top, key[i + j]);
        }
      }
    }
    float lmax = 0.f, sum = 1.f;
    if (FN != 2) lmax = from_ordered(__reduce_max_sync(kAll, top));
    if (FN == 0) {
      sum = 0.f;
      if (a.renorm) {                   // (weights are divided by their own sum: the row's cancels, and is good enough for keys)
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (key[i] && v[i] != -INFINITY) sum += __expf(v[i] - lmax);
      } else {
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (key[i] && v[i] != -INFINITY) sum += expf(v[i] - lmax);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
    }
    const FastScores<FN> fast{lmax, 1.f / sum};
    const float near = fmaxf(fast.template apart<PER>(), 0.f);         // (NaN: there are no scores but masked experts' zeros)
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (key[i]) key[i] = ordered(fast(v[i]) + bias[i]);
    }
    uint32_t k1 = 0, k2 = 0;            // the lane's largest two keys
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      k2 = max(k2, min(k1, key[i]));
      k1 = max(k1, key[i]);
    }
    // The lanes' experts with `is` into list, 32 of them at most; returns how many there are.
    const auto collect = [&](auto is) {
      int n = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) n += is(i);
      int p = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kAll, p, d);
        if (lane >= d) p += o;
      }
      const int c = __shfl_sync(kAll, p, 31);
      p -= n;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        {
          const bool in = is(i);
          if (in && p < 32) list[p] = make_uint2(e0 + at(i), key[i]);
          p += in;
        }
      __syncwarp();
      return c;
    };
    const auto key64 = [&](const Scores64<FN>& score, int e) {
      const double s = score(logit(a, row, e));
      return clean(a.bias ? s + __ldg(a.bias + e) : s);
    };
    bool all64 = false;                 // too many keys are near one another
    if (a.KG < a.G) {
      uint32_t g1 = k1, g2 = k2;
      for (int d = 1; d < a.L; d <<= 1) {
        const uint32_t o1 = __shfl_xor_sync(kAll, g1, d), o2 = __shfl_xor_sync(kAll, g2, d);
        g2 = max(min(g1, o1), max(g2, o2));
        g1 = max(g1, o1);
      }
      // what the group is worth, and how far that may be off: two scores and additions
      const bool two = a.best == 2 && g2;
      float worth = -INFINITY, size = 0.f, f2 = 0.f;
      if (used) {
        f2 = from_ordered(two ? g2 : g1);
        worth = a.bias ? from_ordered(g1) : fast(from_ordered(g1));
        size = size_of(worth);
        if (two) {
          const float w2 = a.bias ? f2 : fast(f2);
          worth += w2;
          size += size_of(w2);
        }
      }
      uint32_t mine = used && sub == 0 ? ordered(worth) : 0;
      // (without a bias a NaN logit is -infinity in the keys here, whose score is 0: where one may count, all groups take the
      // second look; where all scores are NaN but masked experts' zeros, from all of their experts)
      const bool none = FN == 0 && !a.bias && sum != sum;
      bool nan = none;
      if (!a.bias && !none && __any_sync(kAll, f2 == -INFINITY)) {
#pragma unroll
        for (int i = 0; i < PER; ++i) nan = nan || v[i] != v[i];
        nan = __any_sync(kAll, nan);
      }
      const float tol = nan ? INFINITY : 2.f * near + __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(size))) * 0x1p-21f;
      unsigned open = 0;                // by the lanes with sub = 0
      uint32_t kth = 0;
      for (int k = 0; k < a.KG; ++k) {
        const uint32_t best = __reduce_max_sync(kAll, mine);
        const int who = __ffs(__ballot_sync(kAll, mine == best)) - 1;      // the lowest group of equals
        open |= 1u << who;
        if (lane == who) mine = 0;
        kth = best;
      }
      const float last = from_ordered(kth), next = from_ordered(__reduce_max_sync(kAll, mine));
      // (an infinite tol: some group's sum is past fp32's range, and last - next may be inf - inf)
      if (tol == INFINITY || last - next <= tol) {
        // groups that are surely in, and those that may be: the latter in 64 bits, from their experts that may be among
        // the best two
        const bool in = used && worth - next > tol, maybe = used && !in && !(last - worth > tol);
        const uint32_t bound = !maybe ? 0xffffffffu : a.bias ? ordered(f2 - tol) : none ? 1u : two ? g2 : g1;
        const int c = collect([&](int i) { return maybe && key[i] >= bound; });
        all64 = c > 32;
        if (!all64) {
          const Scores64<FN> score = scores64<FN>(a, row, lmax);
          const int e = lane < c ? list[lane].x : 0;
          const double k = lane < c ? key64(score, e) : 0.;
          const int of = lane < c ? e / a.per_group : -1;
          double b1 = -INFINITY, b2 = -INFINITY;
          for (int r = 0; r < c; ++r) {
            const double o = __shfl_sync(kAll, k, r);
            if (__shfl_sync(kAll, of, r) != g) continue;
            if (o > b1) {
              b2 = b1;
              b1 = o;
            } else if (o > b2) {
              b2 = o;
            }
          }
          const double exact = clean(two ? b1 + b2 : b1);
          const unsigned may = __ballot_sync(kAll, maybe && sub == 0);
          open = __ballot_sync(kAll, in && sub == 0);
          const int places = a.KG - __popc(open);
          int rank = 0;
          for (unsigned m = may; m; m &= m - 1) {
            const int h = __ffs(m) - 1;
            const double o = __shfl_sync(kAll, exact, h);
            rank += o > exact || (o == exact && h < (lane & ~(a.L - 1)));
          }
          open |= __ballot_sync(kAll, maybe && sub == 0 && rank < places);
        }
        __syncwarp();
      }
      if (!(open >> (g << a.log_l) & 1)) {
        k1 = k2 = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) key[i] = 0;
      }
    }
    int id = 0;
    if (!all64) {
      // the K + 1 largest of the lanes' largest two keys (fewer: every key) are a bound for the K + 1 largest keys
      uint32_t bound = 0;
      for (int k = 0; k <= a.K; ++k) {
        bound = __reduce_max_sync(kAll, k1);
        const int who = __ffs(__ballot_sync(kAll, k1 == bound)) - 1;
        if (lane == who) {
          k1 = k2;
          k2 = 0;
        }
      }
      bound = max(bound, 1u);
      int c = collect([&](int i) { return key[i] >= bound; });
      if (c <= 32) {
        // the order of (key, lower id first) as one number
        const uint2 m = lane < c ? list[lane] : make_uint2(0, 0);
        const unsigned long long mine = static_cast<unsigned long long>(m.y) << 32 | ~m.x;
        int rank = 0;
#pragma unroll 4
        for (int r = 0; r < c; ++r) {
          const uint2 o = list[r];
          rank += (static_cast<unsigned long long>(o.y) << 32 | ~o.x) > mine;
        }
        __syncwarp();
        if (lane < c && rank <= a.K) list[rank] = m;
        if (lane == 0 && c <= a.K) list[a.K].y = 0;
      } else {
        __syncwarp();
        for (int k = 0; k <= a.K; ++k) {
          uint32_t b = 0;
          int bi = 0;
#pragma unroll
          for (int i = 0; i < PER; ++i)
            if (key[i] > b) {
              b = key[i];
              bi = i;
            }
          const uint32_t best = __reduce_max_sync(kAll, b);
          const int e = b == best && best ? e0 + at(bi) : kNone;
          const int won = static_cast<int>(__reduce_min_sync(kAll, static_cast<uint32_t>(e)));
          if (lane == 0) list[k] = make_uint2(won, best);
          if (e == won && best) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
              if (i == bi) key[i] = 0;
          }
        }
      }
      __syncwarp();
      const uint2 own = lane < a.K ? list[lane] : make_uint2(0, 1);
      id = own.x;
      if (a.bias) {
        bool unsure = false, tie = false;
        const uint2 after = lane < a.K ? list[lane + 1] : make_uint2(0, 0);
        const float f = from_ordered(own.y);
        if (after.y != 0) {
          const int ne = after.x;
          const float nf = from_ordered(after.y);
          if (f - nf <= near + (size_of(f) + size_of(nf)) * 0x1p-23f) {
            unsure = logit(a, row, id) != logit(a, row, ne) || __ldg(a.bias + id) != __ldg(a.bias + ne);
            tie = !unsure && lane == a.K - 1;
          }
        }
        if (__any_sync(kAll, unsure || tie)) {
          const float kth = __shfl_sync(kAll, f, a.K - 1);
          const uint32_t low = ordered(kth - (near + size_of(kth) * 0x1p-21f));
          if (!__any_sync(kAll, unsure)) {
            // the last one in and the first one out are equals: a key behind the two may be near them, and larger
            const uint32_t high = __shfl_sync(kAll, own.y, a.K - 1);
            const int last = __shfl_sync(kAll, id, a.K - 1);
            const float l = logit(a, row, last), b = __ldg(a.bias + last);
            unsigned long long alike = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) alike |= static_cast<unsigned long long>(key[i] >= low && key[i] <= high) << i;
            for (; alike && !unsure; alike &= alike - 1) {
              const int e = e0 + at(__ffsll(alike) - 1);
              unsure = logit(a, row, e) != l || __ldg(a.bias + e) != b;
            }
          }
          if (__any_sync(kAll, unsure)) {
            // every key that may be among the K largest, in 64 bits
            __syncwarp();
            all64 = c > 32;             // (the rounds have used the keys up)
            if (!all64) c = collect([&](int i) { return key[i] >= low; });
            all64 = all64 || c > 32;
            if (!all64) {
              const Scores64<FN> score = scores64<FN>(a, row, lmax);
              const int e = lane < c ? list[lane].x : kNone;
              const double k = lane < c ? key64(score, e) : -INFINITY;
              int rank = 0;
              for (int r = 0; r < c; ++r) {
                const double o = __shfl_sync(kAll, k, r);
                const int oe = __shfl_sync(kAll, e, r);
                rank += o > k || (o == k && oe < e);
              }
              __syncwarp();
              if (lane < c && rank < a.K) list[rank].x = e;
              __syncwarp();
              if (lane < a.K) id = list[lane].x;
            }
          }
        }
      }
    }
    if (all64) id = select_all64<FN, PER>(a, row, lmax, id);
    __syncwarp();
    const Scores<FN> score{lmax, sum};
    float s = lane < a.K ? score(logit(a, row, id)) : 1.f;
    const bool tiny = __any_sync(kAll, s < kTiny);
    if (a.renorm) {
      float all = lane < a.K ? s : 0.f;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) all += __shfl_xor_sync(kAll, all, d);
      s = all == 0.f ? 0.f : s / all;
    }
    if (lane < a.K) {
      a.ids[t * a.K + lane] = id;
      a.w[t * a.K + lane] = s * a.scale;
    }
    if (tiny) weights64<FN>(a, t, lmax, id);
  }
}

template <int FN, int PER, int V>
cudaError_t select_launch(const SelectArgs& a, cudaStream_t stream) {
  // (as many tokens to every warp that is there at a time: 16384 tokens 21.8 us when this took 19.4; a warp a token 22)
  const int ctas = (a.T - 1) / kSelectWarps + 1, most = 2 * kSelectCtas * num_sms();
  return launch_pdl(select_kernel<FN, PER, V>, dim3(ctas < most ? ctas : most), dim3(kSelectWarps * 32), 0, stream, a);
}

template <int FN>
cudaError_t select_by_size(const SelectArgs& a, cudaStream_t stream) {
  const size_t four = 4 * dtype_bytes(a.dt);
  if (a.per_group % 4 == 0 && reinterpret_cast<uintptr_t>(a.logits) % four == 0 && (a.T <= 1 || a.row_bytes % four == 0)) {
    const int per = (a.per_group + 4 * a.L - 1) / (4 * a.L) * 4;
    if (per <= 8) return select_launch<FN, 8, 4>(a, stream);
    if (per <= 16) return select_launch<FN, 16, 4>(a, stream);
    if (per <= 32) return select_launch<FN, 32, 4>(a, stream);
    return select_launch<FN, 64, 4>(a, stream);
  }
  const int per = (a.per_group + a.L - 1) / a.L;
  if (per <= 8) return select_launch<FN, 8, 1>(a, stream);
  if (per <= 16) return select_launch<FN, 16, 1>(a, stream);
  if (per <= 32) return select_launch<FN, 32, 1>(a, stream);
  return select_launch<FN, 64, 1>(a, stream);
}

}  // namespace

cudaError_t launch_select(int ldt, RowsView logits, const float* bias, int T, int E, int K, const SelectRule& rule,
                          int32_t* ids, float* w, cudaStream_t stream) {
  SelectArgs a{};
  a.logits = static_cast<const uint8_t*>(logits.ptr);
  a.row_bytes = logits.ld * static_cast<long long>(dtype_bytes(ldt));
  a.dt = ldt;
  a.bias = bias;
  a.T = T;
  a.E = E;
  a.K = K;
  a.KG = rule.topk_groups;
  a.G = rule.topk_groups < rule.groups ? rule.groups : 1;     // all groups used: one group of all experts
  if (a.G == 1) a.KG = 1;
  a.best = rule.best;
  a.renorm = rule.renorm;
  a.scale = rule.scale;
  a.per_group = E / a.G;
  a.log_l = 5;
  while ((a.G << a.log_l) > 32) --a.log_l;
  a.L = 1 << a.log_l;
  a.ids = ids;
  a.w = w;
  if (rule.fn == 0) return select_by_size<0>(a, stream);
  if (rule.fn == 1) return select_by_size<1>(a, stream);
  return select_by_size<2>(a, stream);
}

}  // namespace moe
