// Root-mean-square norm of rows, with the residual's addition before it and 8-bit output rows, and its gradients.
//
//   s = x + residual (rounded to the rows' type, as it is stored: forward and backward then see the same stream)
//   r = (mean(s^2) + eps)^(-1/2);   y_i = s_i r w_i
//   g_i = dy_i w_i:   dx_i = r g_i - s_i r^3 mean(s g) + dsum_i;   dw_i = sum over rows of dy_i s_i r
// Both are taken in fp32; each output is rounded once, the 8-bit rows (rows8.cuh) from the fp32 y.  One pass over a
// row gives both of the backward's sums (s^2 and s g), so nothing but s is kept from the forward.
//
// HBM bounds them where rows are many: each value is read and written once.  16384 x 7168 bf16 with residual, 16-bit and
// 8-bit outputs, 1.06 GB in 159 us (98% of a plain copy's rate); without residual 114 us (76%: about 170 instructions a
// pack); gradients of 8192 x 7168 with dsum 75.2 us (92%), 4 us of it the launch that adds the CTAs' parts of dw up.  8192 x
// 4096 fp32 with residual 81 us (98%), 16384 x 2048 bf16 42 (94%), its gradients 44 (90%).  Rows that start on no 16-byte
// boundary are bound by the shifts' instructions: 9000 x 6001 bf16, residual and all outputs, 168 us of 72 (no residual, y
// alone 76 of 32), 20000 x 300 31 of 8, 1450 x 2521 fp16 17 of 5.  A row of 7168 alone takes 2.9 us: launch, one load, the
// reduction's two steps, the stores.
//
// Rows past the ring are further from their bytes.  Gradients of 1025 to 2048 packs, one CTA of 1024 threads per SM with
// nothing of the next row on its way and, in 16 bits, spilled registers: 8192 x 8704 bf16 with dsum 163 us of 84, 2000 x 12000
// 62 of 28, 8192 x 7168 fp32 155 of 138.  Beyond 2048 packs x and dy are read four times (sums, dw, sums again, dx), w an
// element at a time, which keeps L1 busy for 94% of the time: 2000 x 17000 bf16 165 us of 40, 2000 x 17001 250, 2000 x 30000
// 285 of 71, 3000 x 9000 fp32 166 of 64.  Forward, twice: 2000 x 17000 bf16 with residual to 16 bits 68 us of 40, off
// boundaries 83.
//
// (Reading each row twice, from L1 and L2 the second time: 205 us and, the gradients, 266; a row in registers with the next
// one's loads ahead, two CTAs of 448 threads: 243, 151.)
#include "rows8.cuh"

namespace moe {

namespace {

constexpr int kNormThreads = 256;

struct NormArgs {
  const void *x, *res;
  void *sum, *y;
  const float* w;
  uint8_t *q, *sf;
  long long ldx, ldr, lds, ldy, ldq, ldsf;
  float eps, over_h;          // over_h: 1 / H
  int T, H;
  int q_words;                // codes in whole words
};

// Sum over the block of K values per thread, in a fixed order; every thread gets it.
template <int K>
__device__ __forceinline__ void block_sum(float (&v)[K], float (*sh)[K]) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], d);
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) sh[warp][k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = lane < warps ? sh[lane][k] : 0.f;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], d);
}

// A matrix of rows of H columns.  AL: every row on a 16-byte boundary and H in whole packs.
template <class T>
struct Mat {
  using raw = typename T::raw;
  raw *lo, *hi;               // its first element and the end of its last row
  long long ld;
  __device__ __forceinline__ Mat(const void* p, long long l, int rows, int H)
      : lo(static_cast<raw*>(const_cast<void*>(p))), hi(lo + (rows - 1) * l + H), ld(l) {}
  // columns [c, c + N) of a row; zeros past its end
  template <bool AL>
  __device__ __forceinline__ Words<T> get(long long row, int c, int H) const {
    const raw* p = lo + row * ld + c;
    if constexpr (AL) {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      Words<T> v;
      v.w[0] = u.x;
      v.w[1] = u.y;
      v.w[2] = u.z;
      v.w[3] = u.w;
      return v;
    } else {
      ShiftedPack<T> s;
      s.load(p, lo, hi);
      Pack<T> v = s.get();
#pragma unroll
      for (int i = 0; i < Pack<T>::N; ++i)
        if (c + i >= H) v.v[i] = T::from_f(0.f);
      return v;
    }
  }
};

// Row pointers of the outputs (null: not wanted).
template <class T>
struct RowOut {
  typename T::raw *sum, *y;
  uint8_t *q, *sf;
  __device__ __forceinline__ RowOut(const NormArgs& a, long long t)
      : sum(static_cast<typename T::raw*>(a.sum)), y(static_cast<typename T::raw*>(a.y)), q(a.q), sf(a.sf) {
    on(a, t);
  }
  __device__ __forceinline__ void on(const NormArgs& a, long long rows) {
    if (sum) sum += rows * a.lds;
    if (y) y += rows * a.ldy;
    if (q) {
      q += rows * a.ldq;
      sf += rows * a.ldsf;
    }
  }
};
template <class T, bool AL>
__device__ __forceinline__ void put_words(typename T::raw* p, int left, const Words<T>& words) {
  if constexpr (AL) {
    *reinterpret_cast<uint4*>(p) = make_uint4(words.w[0], words.w[1], words.w[2], words.w[3]);
  } else {
    const Pack<T> v = words;
#pragma unroll
    for (int i = 0; i < Pack<T>::N; ++i)
      if (i < left) p[i] = v.v[i];
  }
}

// The same by all lanes of a warp, whose packs follow one another (c may lie past the row's end).
template <class T, bool AL>
__device__ __forceinline__ void put_row(typename T::raw* row, int c, int H, const Words<T>& words) {
  if constexpr (AL) {
    if (c < H) put_words<T, true>(row + c, H - c, words);
  } else {
    const int lane = threadIdx.x % 32;
    store_shifted<T>(row, c, H, words, lane == 0, lane == 31);
  }
}

// The outputs of N values of y from column c of a row on (called by all lanes of a warp).
template <class T, bool AL>
__device__ __forceinline__ void norm_out(const NormArgs& a, const RowOut<T>& row, int c, const float (&v)[Pack<T>::N]) {
  constexpr int N = Pack<T>::N;
  if (row.y) {
    Words<T> o;
#pragma unroll
    for (int j = 0; j < N; j += 2) o.set2(j, v[j], v[j + 1]);
    put_row<T, AL>(row.y, c, a.H, o);
  }
  if (row.q) {
    uint32_t q[N / 4];
    const uint32_t scale = encode8<N>(v, q);
    const int lane = threadIdx.x % 32;
    store_row_codes8<N>(row.q, c, a.H, q, a.q_words, lane == 0, lane == 31);
    if (c < a.H && c % kGroup8 == 0) row.sf[c / kGroup8] = static_cast<uint8_t>(scale);
  }
}

// A row's packs over the threads that share it: pack i of thread `tid` is tid + i * threads.  A warp per row (WARP) or
// the CTA; the CTA's sums meet in two buffers in turn, so that one barrier a row is enough.
template <bool WARP, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float (*sh)[32][K], int& turn) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], d);
  if constexpr (!WARP) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) sh[turn][warp][k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = lane < warps ? sh[turn][lane][k] : 0.f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], d);
    turn ^= 1;
  }
}

// The thread's part of w (zeros past the row's end).
template <class T, bool AL, int PER>
__device__ __forceinline__ void weights(float (&w)[PER][Pack<T>::N], const float* g, int tid, int threads, int H) {
  constexpr int N = Pack<T>::N;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = (tid + i * threads) * N;
    if constexpr (AL) {
#pragma unroll
      for (int j = 0; j < N; j += 4) {
        const float4 f = c < H ? __ldg(reinterpret_cast<const float4*>(g + c + j)) : make_float4(0.f, 0.f, 0.f, 0.f);
        w[i][j] = f.x;
        w[i][j + 1] = f.y;
        w[i][j + 2] = f.z;
        w[i][j + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) w[i][j] = c + j < H ? __ldg(g + c + j) : 0.f;
    }
  }
}

// Rows in registers, PER packs a thread, NT threads at most, MIN CTAs per SM.  AHEAD: the next row's loads are on their way
// while this one is worked on, and w stays in registers.
template <class T, bool AL, int PER, bool WARP, int NT, int MIN, bool AHEAD>
__global__ void __launch_bounds__(NT, MIN) norm_kernel(const NormArgs a) {
  constexpr int N = Pack<T>::N;
  __shared__ float sh[2][32][1];
  const int H = a.H, threads = WARP ? 32 : blockDim.x, tid = WARP ? threadIdx.x % 32 : threadIdx.x;
  const int rows = WARP ? blockDim.x / 32 : 1;            // rows of a CTA at a time
  const long long step = static_cast<long long>(gridDim.x) * rows;
  long long t = static_cast<long long>(blockIdx.x) * rows + (WARP ? threadIdx.x / 32 : 0);
  grid_dependency_wait();
  grid_launch_dependents();
  const Mat<T> x(a.x, a.ldx, a.T, H), r(a.res, a.ldr, a.T, H);
  RowOut<T> out(a, t);
  Words<T> px[PER], pr[PER];
  auto fetch = [&](long long row) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (tid + i * threads) * N;
      px[i] = pr[i] = Words<T>{};
      if (c < H && row < a.T) {
        px[i] = x.template get<AL>(row, c, H);
        if (a.res) pr[i] = r.template get<AL>(row, c, H);
      }
    }
  };
  if (AHEAD) fetch(t);
  float w[PER][N];
  weights<T, AL, PER>(w, a.w, tid, threads, H);
  int turn = 0;
  for (; t < a.T; t += step, out.on(a, step)) {
    if (!AHEAD) fetch(t);
    Words<T> p[PER];
    float ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (tid + i * threads) * N;
      p[i] = px[i];
      if (a.res) p[i].add(pr[i]);
      p[i].keep();
      if (out.sum) put_row<T, AL>(out.sum, c, H, p[i]);
#pragma unroll
      for (int j = 0; j < N; ++j) ss[0] = fmaf(p[i].f(j), p[i].f(j), ss[0]);
    }
    if (AHEAD) fetch(t + step);
    row_sum<WARP, 1>(ss, sh, turn);
    if (!AHEAD) weights<T, AL, PER>(w, a.w, tid, threads, H);
#pragma unroll
    for (int i = 0; i < PER; ++i) p[i].keep();
    const float rs = rsqrtf(ss[0] * a.over_h + a.eps);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (tid + i * threads) * N;
      float v[N];
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = p[i].f(j) * rs * w[i][j];
      norm_out<T, AL>(a, out, c, v);
    }
  }
}

// Rows too wide for registers: one CTA per row, which is read twice.
template <class T, bool AL>
__global__ void __launch_bounds__(kNormThreads) norm_wide_kernel(const NormArgs a) {
  constexpr int N = Pack<T>::N;
  __shared__ float sh[32][1];
  grid_dependency_wait();
  grid_launch_dependents();
  const long long t = blockIdx.x;
  const int H = a.H;
  const Mat<T> x(a.x, a.ldx, a.T, H), r(a.res, a.ldr, a.T, H), s(a.sum, a.lds, a.T, H);
  const RowOut<T> out(a, t);
  float ss[1] = {0.f};
  for (int c = threadIdx.x * N; c < H; c += kNormThreads * N) {
    Words<T> p = x.template get<AL>(t, c, H);
    if (a.res) p.add(r.template get<AL>(t, c, H));
    if (a.sum) put_words<T, AL>(out.sum + c, H - c, p);
#pragma unroll
    for (int i = 0; i < N; ++i) ss[0] = fmaf(p.f(i), p.f(i), ss[0]);
  }
  block_sum<1>(ss, sh);
  const float rs = rsqrtf(ss[0] * a.over_h + a.eps);
  const int whole = groups8(H) * kGroup8;      // (a group's lanes meet in group_max)
  for (int c0 = 0; c0 < whole; c0 += kNormThreads * N) {
    const int c = c0 + threadIdx.x * N;
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
    if (c < H) {
      Words<T> p;
      if (a.sum) {
        p = s.template get<AL>(t, c, H);
      } else {
        p = x.template get<AL>(t, c, H);
        if (a.res) p.add(r.template get<AL>(t, c, H));
      }
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (AL || c + i < H) v[i] = p.f(i) * rs * __ldg(a.w + c + i);
    }
    norm_out<T, AL>(a, out, c, v);
  }
}

// ------------------------------------------------------------------------------------------
// Many rows: they arrive in a ring of S shared-memory stages by bulk copies, and G groups of threads
// take them in turn (row k of the CTA's is in stage k % S and group k % G's), each into registers, so that a group's
// reductions run under the copies and the others' work.  One CTA per SM.
// S is a multiple of G: then a stage is always the same group's, which has seen its last row arrive before it waits for the
// next one.  (A group that waited for a row whose stage's last row, another group's, had not arrived yet would take the
// barrier's older phase for the one it wants: copies of different rows may arrive in any order.)
// Rows that start anywhere (not AL) come with the ends of the 16-byte words that they begin and end in, and are shifted as
// they are taken out; the few elements of a word that reaches out of the matrix are copied one by one.

// Groups of several warps, at most (15 barriers there are; 8: 4000 x 1001 bf16 17.4 us instead of 15.9, 14: 2000 x 700 fp32
// 5.9 instead of 5.6).  Groups of one warp (ONE) need none, and there are as many as have their stages: with 8 of them
// 20000 x 300 bf16 56 us and its gradients 38 instead of 31.5 and 30.7.  (A warp per row without the ring 102 and 48.)
constexpr int kRingStages = 32, kRingGroups = 9;
// Threads of all groups, at most.
constexpr int ring_threads(bool al) { return al ? 960 : 608; }
constexpr int kRingGradThreads = 608;
constexpr int kRingWarps = 30, kRingGradWarps = 16;             // of a group, at most
constexpr int kRingBytes = 223 * 1024;                          // stages and w
constexpr int kRingSmem = kRingBytes + 128;
// Stages, if that makes enough of them: two a group in the backward, one (but two in all) in the forward.  What arrives much
// ahead of the other SMs' rows costs the memory its locality: 16384 x 7168 with residual, two groups, 2 stages 160 us, 4 of
// them 183; the backward of 8192 x 7168 (one group) 1 stage 95 us, 2 stages 75, 4 79.
constexpr int kRingAhead = 60 * 1024;
// Packs a thread; the forward takes four where a row has more than kRingWide and its instructions are the bound (fp32 without
// residual, rows that start anywhere), since a row's reduction costs the same for twice the packs: 8192 x 4096 fp32 to 8 bits
// alone 44.8 us instead of 68 and to fp32 44.6 of 47.7 (with residual 95 of 88), 9000 x 6001 bf16 167 instead of 208.  In 16
// bits on boundaries they do not fit the 64 registers: 16384 x 7168 to 8 bits alone 100 us of 110, but to bf16 84 of 75 and
// with residual 191 of 159.  From 320 to 440 packs either is as fast (2801 odd bf16 columns 33.9 with four, 32.5; 3501 fp16
// 40.3, 40.9).  Three where they make one warp of a group of two (65 to 96 packs): 2000 x 521 bf16 4.7 us instead of 6.1, 20000
// x 765 22.4 instead of 35.0, 2000 x 261 fp32 4.0 of 5.2, 20000 x 383 18.2 of 25.9.
constexpr int kRingPer = 2, kRingWide = 512;

struct Ring {
  int G, threads, S;          // groups, threads of a group, stages
  int per;                    // packs of a thread
};

struct RingState {
  uint64_t full[kRingStages], empty[kRingStages], w_full;
};

template <class E>
__device__ __forceinline__ void copy_element(uint32_t to, uintptr_t from) {
  if constexpr (sizeof(E) == 2)
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(to), "h"(*reinterpret_cast<const uint16_t*>(from)) : "memory");
  else
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(to), "f"(*reinterpret_cast<const float*>(from)) : "memory");
}

// Bytes of a row's place in a stage (not AL: wherever in its first word it starts, and a word that a shift reads on).
template <bool AL>
__host__ __device__ __forceinline__ uint32_t ring_slot(uint32_t row_bytes) {
  return AL ? row_bytes : (row_bytes + 15) / 16 * 16 + 32;
}
// Shared memory of w.
__host__ __device__ __forceinline__ uint32_t ring_w_bytes(int H) { return static_cast<uint32_t>(H + 7) / 8 * 32; }

// Whether the phase with the given parity is over (asked only, where mbar_wait may put the thread to sleep).
__device__ __forceinline__ bool mbar_over(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
               : "=r"(ok)
               : "r"(bar), "r"(parity)
               : "memory");
  return ok != 0;
}

// Copies one row of the MOST matrices `in` (null: not there) of rows of `bytes` bytes, ld bytes apart, of elements of type E
// to a stage, to arrive on bar.
template <bool AL, class E, int MOST>
__device__ __forceinline__ void ring_row(long long t, uint32_t stage, uint32_t bar, const void* const (&in)[MOST],
                                         const long long (&ld)[MOST], int n, int T, uint32_t bytes, uint32_t slot) {
  using U = uintptr_t;
  uint32_t to = stage;
  if constexpr (AL) {
    mbar_arrive_expect_tx(bar, n * bytes);
#pragma unroll
    for (int i = 0; i < MOST; ++i)
      if (in[i]) {
        bulk_load(to, static_cast<const uint8_t*>(in[i]) + t * ld[i], bytes, bar);
        to += slot;
      }
  } else {
    U from[MOST];
    uint32_t skip[MOST], size[MOST], all = 0;
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
      size[i] = 0;
      if (!in[i]) continue;
      const U lo = reinterpret_cast<U>(in[i]), row = lo + static_cast<U>(t * ld[i]), end = row + bytes;
      const U hi = lo + static_cast<U>((T - 1) * ld[i]) + bytes;
      U a = row & ~U(15), b = (end + 15) & ~U(15);
      skip[i] = 0;
      if (a < lo) {                   // (the matrix' first row)
        a += 16;
        skip[i] = 16;
        for (U e = row; e < a; e += sizeof(E)) copy_element<E>(to + static_cast<uint32_t>(e & 15), e);
      }
      if (b > hi) {                   // (its last one)
        b -= 16;
        for (U e = b; e < end; e += sizeof(E)) copy_element<E>(to + skip[i] + static_cast<uint32_t>(e - a), e);
      }
      from[i] = a;
      size[i] = static_cast<uint32_t>(b - a);
      all += size[i];
      to += slot;
    }
    if (t == 0 || t == T - 1) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");    // (elements copied one by one)
    mbar_arrive_expect_tx(bar, all);
    to = stage;
#pragma unroll
    for (int i = 0; i < MOST; ++i)
      if (in[i]) {
        if (size[i]) bulk_load(to + skip[i], reinterpret_cast<const void*>(from[i]), size[i], bar);
        to += slot;
      }
  }
}

// The loading warp: lane s refills stage s whenever it is empty (one lane for all of them: gradients of 20000 x
// 300 bf16 81 us instead of 38, of 9887 x 544 fp16 26 instead of 16, 8192 x 4096 fp32 to 8 bits alone 66 instead of 68).  It stays until its copies are there or have had as long as a wait has (they would land in the shared memory of
// whoever comes after the CTA); status: where a wait that runs out is recorded (null: nowhere).
template <bool AL, class E, int MOST>
__device__ __forceinline__ void ring_load(const Ring& R, RingState& st, uint32_t smem, const void* const (&in)[MOST],
                                          const long long (&ld)[MOST], int T, uint32_t bytes, const float* w, int H,
                                          uint32_t* status) {
  const int lane = threadIdx.x % 32;
  if (lane == 0) {
    const uint32_t wbytes = static_cast<uint32_t>(H) / 4 * 16;
    for (int i = H / 4 * 4; i < (H + 7) / 8 * 8; ++i)      // the last values, and zeros to the end of a pack
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(smem + 4 * i), "f"(i < H ? __ldg(w + i) : 0.f) : "memory");
    if (wbytes) {
      mbar_arrive_expect_tx(smem_u32(&st.w_full), wbytes);
      bulk_load(smem, w, wbytes, smem_u32(&st.w_full));
    } else {
      mbar_arrive(smem_u32(&st.w_full));
    }
  }
  int n = 0;
#pragma unroll
  for (int i = 0; i < MOST; ++i) n += in[i] != nullptr;
  const uint32_t slot = ring_slot<AL>(bytes), stage = smem + ring_w_bytes(H) + lane * n * slot;
  const int mine = lane < R.S ? lane : 0;
  const uint32_t full = smem_u32(&st.full[mine]), empty = smem_u32(&st.empty[mine]);
  long long t = lane < R.S ? blockIdx.x + static_cast<long long>(lane) * gridDim.x : T;
  uint32_t ph = 0;
  long long since = clock64();
  while (__any_sync(0xffffffffu, t < T)) {
    const bool go = t < T && mbar_over(empty, ph ^ 1);
    if (go) {
      ring_row<AL, E, MOST>(t, stage, full, in, ld, n, T, bytes, slot);
      t += static_cast<long long>(R.S) * gridDim.x;
      ph ^= 1;
    }
    // (a wait that runs out ends the copies; the groups' own waits for them then run out too)
    if (__any_sync(0xffffffffu, go)) {
      since = clock64();
    } else if (__any_sync(0xffffffffu, clock64() - since > kWaitBudgetCycles)) {
      record_error(status, kDevErrTimeout);
      break;
    } else {
      __nanosleep(100);
    }
  }
  if (lane == 0) mbar_wait(smem_u32(&st.w_full), 0, status);
  if (lane < R.S) mbar_wait(full, ph ^ 1, status);
}

__device__ __forceinline__ void ring_init(const Ring& R, RingState& st) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < R.S; ++s) {
      mbar_init(smem_u32(&st.full[s]), 1);
      mbar_init(smem_u32(&st.empty[s]), R.threads / 32);
    }
    mbar_init(smem_u32(&st.w_full), 1);
    fence_barrier_init();
  }
}

// A group's place in the ring: its k-th row's stage and the parity to wait for.
struct RingPlace {
  int s;
  uint32_t ph;
  __device__ __forceinline__ RingPlace(int k, int S) : s(k % S), ph((k / S) & 1) {}
  __device__ __forceinline__ void on(int n, int S) {
    s += n;
    while (s >= S) {
      s -= S;
      ph ^= 1;
    }
  }
};

template <class T>
__device__ __forceinline__ Words<T> shared_words(uint32_t addr) {
  Words<T> v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3])
               : "r"(addr)
               : "memory");
  return v;
}
// Columns [c, c + N) of a row of H from its first element's place on (not AL: any place; zeros past the end).
template <class T, bool AL>
__device__ __forceinline__ Words<T> shared_row(uint32_t row, int c, int H) {
  constexpr int N = Words<T>::N;
  if constexpr (AL) {
    return shared_words<T>(row + c * (16 / N));
  } else {
    const uint32_t p = row + c * (16 / N);
    const Words<T> a = shared_words<T>(p & ~15u), b = shared_words<T>((p & ~15u) + 16);
    ShiftedPack<T> s;
    s.a = make_uint4(a.w[0], a.w[1], a.w[2], a.w[3]);
    s.b = make_uint4(b.w[0], b.w[1], b.w[2], b.w[3]);
    s.off = p & 15;
    Pack<T> v = s.get();
    if (c + N > H) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (c + i >= H) v.v[i] = T::from_f(0.f);
    }
    return v;
  }
}
// Where in its first word row t of a matrix starts.
template <bool AL>
__device__ __forceinline__ uint32_t ring_off(const void* p, long long row_bytes, long long t) {
  return AL ? 0 : static_cast<uint32_t>((reinterpret_cast<uintptr_t>(p) + static_cast<uintptr_t>(t * row_bytes)) & 15);
}
__device__ __forceinline__ float4 shared_float4(uint32_t addr) {
  float4 f;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w) : "r"(addr));
  return f;
}

// Sum over a group of up to W warps of K values per thread, in a fixed order (sh: zeros where there is no warp); false: some thread's
// `ok` was.
template <int K, int W, bool ONE>
__device__ __forceinline__ bool group_sum(float (&v)[K], float (*sh)[W], int group, int threads, int warp, int lane, bool ok) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], d);
  if constexpr (ONE) return __all_sync(0xffffffffu, ok);
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) sh[k][warp] = v[k];
  ok = named_barrier_and(1 + group, threads, ok);
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = sh[k][lane % W];
#pragma unroll
  for (int d = W / 2; d > 0; d >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], d);
  return ok;
}

template <class T, bool AL, bool ONE, int PER>
__global__ void __launch_bounds__(ring_threads(AL) + 32, 1) norm_ring_kernel(const NormArgs a, const Ring R) {
  constexpr int N = Pack<T>::N;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ RingState st;
  __shared__ __align__(16) float sh[kRingGroups][2][1][32];
  const int H = a.H, threads = ONE ? 32 : R.threads, lane = threadIdx.x % 32, group = threadIdx.x / threads;
  const int tid = threadIdx.x - group * threads;
  const uint32_t smem = (smem_u32(smem_raw) + 127) & ~127u, bytes = H * (16 / N), slot = ring_slot<AL>(bytes);
  ring_init(R, st);
  for (int i = threadIdx.x; i < kRingGroups * 2 * 32; i += blockDim.x) (&sh[0][0][0][0])[i] = 0.f;
  grid_dependency_wait();
  grid_launch_dependents();
  __syncthreads();
  if (group == R.G) {
    const void* in[2] = {a.x, a.res};
    const long long ld[2] = {a.ldx * (16 / N), a.ldr * (16 / N)};
    ring_load<AL, typename T::raw>(R, st, smem, in, ld, a.T, bytes, a.w, H, nullptr);
    return;
  }
  const uint32_t stage0 = smem + ring_w_bytes(H), stage = (a.res ? 2 : 1) * slot;
  bool ok = mbar_wait(smem_u32(&st.w_full), 0, nullptr);
  RingPlace at(group, R.S);
  int turn = 0;
  const int first = blockIdx.x + group * gridDim.x, step = R.G * gridDim.x;
  RowOut<T> out(a, first);
  for (long long t = first; t < a.T; t += step, out.on(a, step), at.on(R.G, R.S), turn ^= 1) {
    ok = mbar_wait(smem_u32(&st.full[at.s]), at.ph, nullptr) && ok;
    const uint32_t from = stage0 + at.s * stage;
    Words<T> p[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (tid + i * threads) * N;
      p[i] = Words<T>{};
      if (c < H) {
        p[i] = shared_row<T, AL>(from + ring_off<AL>(a.x, a.ldx * (16 / N), t), c, H);
        if (a.res) p[i].add(shared_row<T, AL>(from + slot + ring_off<AL>(a.res, a.ldr * (16 / N), t), c, H));
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&st.empty[at.s]));
    float ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (tid + i * threads) * N;
      if (out.sum) put_row<T, AL>(out.sum, c, H, p[i]);
#pragma unroll
      for (int j = 0; j < N; ++j) ss[0] = fmaf(p[i].f(j), p[i].f(j), ss[0]);
      p[i].keep();
    }
    ok = group_sum<1, 32, ONE>(ss, sh[ONE ? 0 : group][turn], group, threads, tid / 32, lane, ok);
    if (!ok) {                          // there is no workspace for a status: the group's rows become NaN
      for (; t < a.T; t += step, out.on(a, step))
        for (int c = tid; c < H; c += threads) {
          if (out.sum) out.sum[c] = T::from_f(NAN);
          if (out.y) out.y[c] = T::from_f(NAN);
          if (out.q) {
            out.q[c] = 0x7f;
            if (c % kGroup8 == 0) out.sf[c / kGroup8] = 255;
          }
        }
      return;
    }
    const float rs = rsqrtf(ss[0] * a.over_h + a.eps);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (tid + i * threads) * N;
      float v[N];
#pragma unroll
      for (int j = 0; j < N; j += 4) {
        const float4 w = c < H ? shared_float4(smem + (c + j) * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
        v[j] = p[i].f(j) * rs * w.x;
        v[j + 1] = p[i].f(j + 1) * rs * w.y;
        v[j + 2] = p[i].f(j + 2) * rs * w.z;
        v[j + 3] = p[i].f(j + 3) * rs * w.w;
      }
      norm_out<T, AL>(a, out, c, v);
    }
  }
}

struct NormGradArgs {
  const void *dy, *x, *dsum;
  void* dx;
  const float* w;
  float *rs, *part;           // [T], [S, H]
  long long lddy, ldx, lddsum, lddx;
  float eps, over_h;
  int T, H;
  uint32_t* status;
};

// Rows in registers, as norm_kernel; a thread adds its columns' part of dw up over its rows (w: a CTA's sums to `part`).
template <class T, bool AL, int PER, bool WARP, int NT, int MIN, bool AHEAD>
__global__ void __launch_bounds__(NT, MIN) norm_grad_kernel(const NormGradArgs a) {
  constexpr int N = Pack<T>::N;
  __shared__ float sh[2][32][2];
  __shared__ float meet[WARP ? NT / 32 : 1][WARP ? 32 * PER * N + 4 : 1];
  const int H = a.H, threads = WARP ? 32 : blockDim.x, tid = WARP ? threadIdx.x % 32 : threadIdx.x;
  const int rows = WARP ? blockDim.x / 32 : 1;
  const long long step = static_cast<long long>(gridDim.x) * rows;
  long long t = static_cast<long long>(blockIdx.x) * rows + (WARP ? threadIdx.x / 32 : 0);
  grid_dependency_wait();
  grid_launch_dependents();
  const Mat<T> dy(a.dy, a.lddy, a.T, H), x(a.x, a.ldx, a.T, H), ds(a.dsum, a.lddsum, a.T, H);
  typename T::raw* dx = static_cast<typename T::raw*>(a.dx) + t * a.lddx;
  Words<T> px[PER], pd[PER], pu[PER];
  auto fetch = [&](long long row) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (tid + i * threads) * N;
      px[i] = pd[i] = pu[i] = Words<T>{};
      if (c < H && row < a.T) {
        px[i] = x.template get<AL>(row, c, H);
        pd[i] = dy.template get<AL>(row, c, H);
        if (a.dsum) pu[i] = ds.template get<AL>(row, c, H);
      }
    }
  };
  if (AHEAD) fetch(t);
  float w[PER][N], acc[PER][N];
  weights<T, AL, PER>(w, a.w, tid, threads, H);
#pragma unroll
  for (int i = 0; i < PER; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) acc[i][j] = 0.f;
  int turn = 0;
  for (; t < a.T; t += step, dx += step * a.lddx) {
    if (!AHEAD) {
      fetch(t);
      weights<T, AL, PER>(w, a.w, tid, threads, H);
    }
    Words<T> p[PER], d[PER], u[PER];
    float m[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      p[i] = px[i];
      d[i] = pd[i];
      u[i] = pu[i];
#pragma unroll
      for (int j = 0; j < N; ++j) {
        m[0] = fmaf(p[i].f(j), p[i].f(j), m[0]);
        m[1] = fmaf(p[i].f(j), d[i].f(j) * w[i][j], m[1]);
      }
    }
    if (AHEAD) fetch(t + step);
    row_sum<WARP, 2>(m, sh, turn);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      p[i].keep();
      d[i].keep();
      u[i].keep();
    }
    const float rs = rsqrtf(m[0] * a.over_h + a.eps), k = m[1] * a.over_h * rs * rs;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (tid + i * threads) * N;
      Words<T> o;
      float v[N];
#pragma unroll
      for (int j = 0; j < N; ++j) {
        acc[i][j] = fmaf(d[i].f(j), p[i].f(j) * rs, acc[i][j]);
        v[j] = (d[i].f(j) * w[i][j] - p[i].f(j) * k) * rs;
        if (a.dsum) v[j] += u[i].f(j);
      }
#pragma unroll
      for (int j = 0; j < N; j += 2) o.set2(j, v[j], v[j + 1]);
      if (a.dx) put_row<T, AL>(dx, c, H, o);
    }
  }
  if (!a.part) return;
  float* out = a.part + static_cast<size_t>(blockIdx.x) * H;
  if constexpr (WARP) {
    float* mine = meet[threadIdx.x / 32];
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) mine[(tid + i * 32) * N + j] = acc[i][j];
    __syncthreads();
    for (int c = threadIdx.x; c < H; c += blockDim.x) {
      float v = 0.f;
      for (int k = 0; k < rows; ++k) v += meet[k][c];
      out[c] = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (tid + i * threads) * N;
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (c + j < H) out[c + j] = acc[i][j];
    }
  }
}

// (the rows' sums and their use as in norm_ring_kernel)
template <class T, bool AL, bool ONE>
__global__ void __launch_bounds__(kRingGradThreads + 32, 1) norm_grad_ring_kernel(const NormGradArgs a, const Ring R) {
  constexpr int N = Pack<T>::N, PER = kRingPer;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ RingState st;
  __shared__ __align__(16) float sh[kRingGroups][2][2][kRingGradWarps];
  const int H = a.H, threads = ONE ? 32 : R.threads, lane = threadIdx.x % 32, group = threadIdx.x / threads;
  const int tid = threadIdx.x - group * threads;
  const uint32_t smem = (smem_u32(smem_raw) + 127) & ~127u, bytes = H * (16 / N), slot = ring_slot<AL>(bytes);
  ring_init(R, st);
  for (int i = threadIdx.x; i < kRingGroups * 2 * 2 * kRingGradWarps; i += blockDim.x) (&sh[0][0][0][0])[i] = 0.f;
  grid_dependency_wait();
  grid_launch_dependents();
  __syncthreads();
  if (group == R.G) {
    const void* in[3] = {a.x, a.dy, a.dsum};
    const long long ld[3] = {a.ldx * (16 / N), a.lddy * (16 / N), a.lddsum * (16 / N)};
    ring_load<AL, typename T::raw>(R, st, smem, in, ld, a.T, bytes, a.w, H, a.status);
    return;
  }
  const uint32_t stage0 = smem + ring_w_bytes(H), stage = (a.dsum ? 3 : 2) * slot;
  bool ok = mbar_wait(smem_u32(&st.w_full), 0, a.status);
  float acc[PER][N];
#pragma unroll
  for (int i = 0; i < PER; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) acc[i][j] = 0.f;
  RingPlace at(group, R.S);
  int turn = 0;
  const int first = blockIdx.x + group * gridDim.x, step = R.G * gridDim.x;
  typename T::raw* dx = static_cast<typename T::raw*>(a.dx) + first * a.lddx;
  for (long long t = first; t < a.T; t += step, dx += step * a.lddx, at.on(R.G, R.S), turn ^= 1) {
    ok = mbar_wait(smem_u32(&st.full[at.s]), at.ph, a.status) && ok;
    const uint32_t from = stage0 + at.s * stage;
    Words<T> p[PER], d[PER], u[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (tid + i * threads) * N;
      p[i] = d[i] = u[i] = Words<T>{};
      if (c < H) {
        p[i] = shared_row<T, AL>(from + ring_off<AL>(a.x, a.ldx * (16 / N), t), c, H);
        d[i] = shared_row<T, AL>(from + slot + ring_off<AL>(a.dy, a.lddy * (16 / N), t), c, H);
        if (a.dsum) u[i] = shared_row<T, AL>(from + 2 * slot + ring_off<AL>(a.dsum, a.lddsum * (16 / N), t), c, H);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&st.empty[at.s]));
    float m[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (tid + i * threads) * N;
#pragma unroll
      for (int j = 0; j < N; j += 4) {
        const float4 w = c < H ? shared_float4(smem + (c + j) * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float wj[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          m[0] = fmaf(p[i].f(j + k), p[i].f(j + k), m[0]);
          m[1] = fmaf(p[i].f(j + k), d[i].f(j + k) * wj[k], m[1]);
        }
      }
      p[i].keep();
      d[i].keep();
      u[i].keep();
    }
    ok = group_sum<2, kRingGradWarps, ONE>(m, sh[ONE ? 0 : group][turn], group, threads, tid / 32, lane, ok);
    if (!ok) break;
    const float rs = rsqrtf(m[0] * a.over_h + a.eps), k = m[1] * a.over_h * rs * rs;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (tid + i * threads) * N;
      Words<T> o;
#pragma unroll
      for (int j = 0; j < N; j += 4) {
        const float4 w = c < H ? shared_float4(smem + (c + j) * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float wj[4] = {w.x, w.y, w.z, w.w};
        float v[4];
#pragma unroll
        for (int l = 0; l < 4; ++l) {
          const float f = p[i].f(j + l), g = d[i].f(j + l);
          acc[i][j + l] = fmaf(g, f * rs, acc[i][j + l]);
          v[l] = (g * wj[l] - f * k) * rs;
          if (a.dsum) v[l] += u[i].f(j + l);
        }
        o.set2(j, v[0], v[1]);
        o.set2(j + 2, v[2], v[3]);
      }
      if (a.dx) put_row<T, AL>(dx, c, H, o);
    }
  }
  if (!a.part) return;
  // the groups' sums meet where the stages were: every group has taken its last row out of them
  const int all = R.G * threads;
  named_barrier(15, all);
  float* meet = reinterpret_cast<float*>(smem_raw + (stage0 - smem_u32(smem_raw)));
  const int pitch = (H + 7) / 8 * 8;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = (tid + i * threads) * N;
    if (c < H)
#pragma unroll
      for (int j = 0; j < N; j += 4)
        *reinterpret_cast<float4*>(meet + group * pitch + c + j) = make_float4(acc[i][j], acc[i][j + 1], acc[i][j + 2], acc[i][j + 3]);
  }
  named_barrier(15, all);
  for (int c = threadIdx.x; c < H; c += all) {
    float v = meet[c];
    for (int k = 1; k < R.G; ++k) v += meet[k * pitch + c];
    a.part[static_cast<size_t>(blockIdx.x) * H + c] = v;
  }
}

template <class T, bool AL>
__global__ void __launch_bounds__(kNormThreads) norm_grad_wide_kernel(const NormGradArgs a) {
  constexpr int N = Pack<T>::N;
  __shared__ float sh[32][2];
  grid_dependency_wait();
  grid_launch_dependents();
  const long long t = blockIdx.x;
  const int H = a.H;
  const Mat<T> dy(a.dy, a.lddy, a.T, H), x(a.x, a.ldx, a.T, H), ds(a.dsum, a.lddsum, a.T, H);
  float m[2] = {0.f, 0.f};
  for (int c = threadIdx.x * N; c < H; c += kNormThreads * N) {
    const Words<T> p = x.template get<AL>(t, c, H), d = dy.template get<AL>(t, c, H);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (AL || c + i < H) {
        m[0] = fmaf(p.f(i), p.f(i), m[0]);
        m[1] = fmaf(p.f(i), d.f(i) * __ldg(a.w + c + i), m[1]);
      }
  }
  block_sum<2>(m, sh);
  const float rs = rsqrtf(m[0] * a.over_h + a.eps), k = m[1] * a.over_h * rs * rs;
  if (threadIdx.x == 0) a.rs[t] = rs;
  if (!a.dx) return;
  for (int c = threadIdx.x * N; c < H; c += kNormThreads * N) {
    const Words<T> p = x.template get<AL>(t, c, H), d = dy.template get<AL>(t, c, H);
    Words<T> o, u;
    if (a.dsum) u = ds.template get<AL>(t, c, H);
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0.f;
      if (AL || c + i < H) v[i] = (d.f(i) * __ldg(a.w + c + i) - p.f(i) * k) * rs;
      if (a.dsum) v[i] += u.f(i);
    }
#pragma unroll
    for (int i = 0; i < N; i += 2) o.set2(i, v[i], v[i + 1]);
    put_words<T, AL>(static_cast<typename T::raw*>(a.dx) + t * a.lddx + c, H - c, o);
  }
}

// Partial sums of dw over rows blockIdx.y, + gridDim.y, ...; thread = column.
template <class T>
__global__ void __launch_bounds__(256) norm_dw_wide_kernel(const NormGradArgs a) {
  using raw = typename T::raw;
  grid_dependency_wait();
  grid_launch_dependents();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.H) return;
  float s = 0.f;
  for (long long t = blockIdx.y; t < a.T; t += gridDim.y)
    s = fmaf(T::to_f(static_cast<const raw*>(a.dy)[t * a.lddy + c]),
             T::to_f(static_cast<const raw*>(a.x)[t * a.ldx + c]) * a.rs[t], s);
  a.part[static_cast<size_t>(blockIdx.y) * a.H + c] = s;
}

// dw from its S partial sums: a CTA has 32 columns, each of its 32 warps every 32nd slice.
__global__ void __launch_bounds__(1024) norm_dw_sum_kernel(const float* __restrict__ part, int S, int H, float* __restrict__ dw) {
  __shared__ float sh[32][33];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < H) {
#pragma unroll 5
    for (int k = warp; k < S; k += 32) s += part[static_cast<size_t>(k) * H + c];
  }
  sh[warp][lane] = s;
  __syncthreads();
  s = sh[lane][warp];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  if (lane == 0 && blockIdx.x * 32 + warp < H) dw[blockIdx.x * 32 + warp] = s;
}

// How rows of `packs` packs run: a warp each with one or a few packs a lane; many rows through the ring; few rows in CTAs of
// up to 1024 threads with one pack a thread, each row over as many threads as it can fill, or with two; or by the kernels for
// wide rows.
enum NormPlanKind { kWarpOne, kWarpMore, kCtaFew, kCtaMost, kWide, kRing, kRingOne };
struct NormPlan {
  NormPlanKind kind;
  int threads, grid;
  Ring ring;
};
// What forward and backward differ in: packs that a warp takes, warps of short rows' CTAs per SM (by 16), the ring's threads,
// warps of a group and a group's stages, and values that are few.
struct NormLimits {
  int warp_packs, resident, ring_per, ring_threads, ring_warps, ring_stages, few;
};
// inputs: matrices of a row that are read; al: all rows on 16-byte boundaries and in whole packs.
NormPlan norm_plan(int T, int H, int dt, const NormLimits& m, int inputs, bool al) {
  const long long row_bytes = static_cast<long long>(H) * dtype_bytes(dt);
  const int packs = static_cast<int>((row_bytes + 15) / 16), sms = num_sms();
  NormPlan p{kWide, kNormThreads, T, Ring{1, 0, 0, kRingPer}};
  if (packs <= 32 || (al && packs <= m.warp_packs && T >= 2 * sms)) {
    p.kind = packs <= 32 ? kWarpOne : kWarpMore;
    const int warps = T >= 16 * sms ? 8 : T >= 8 * sms ? 4 : T >= 4 * sms ? 2 : 1;       // (few rows: over all SMs)
    p.threads = 32 * warps;
    const int ctas = (T - 1) / warps + 1, all = sms * 16 * m.resident / warps;
    p.grid = ctas < all ? ctas : all;
    return p;
  }
  // few rows: all at a time, a pack a thread (500 x 2048 bf16 3.0 us, through the ring 3.6).  Backward as long as the partial
  // sums of dw, one row of them for each row, are few: 160 x 1024 bf16 4.3 us of 5.5, but 304 x 1024 6.1 of 5.5, 240 x 1536 6.5
  // of 5.6 and 456 x 2048 9.3 of 5.9; off boundaries, where the ring takes longer, 160 x 2001 6.5 of 7.4, but 160 x 2500 8.6 of
  // 7.6; fp32, with twice the threads, 304 x 1001 5.9 of 6.6 and 304 x 1024 4.9 of 5.0, but 456 x 1024 5.5 of 5.3
  const int one = (packs + 31) / 32 * 32, at_once = one <= 1024 ? 1024 / one : 1;
  const bool few = T <= sms || (T <= sms * (at_once < 4 ? at_once : 4) && static_cast<long long>(T) * H <= m.few);
  if (packs <= m.ring_per * 32 * m.ring_warps && !few) {
    p.ring.per = m.ring_per;
    p.ring.threads = ((packs + m.ring_per - 1) / m.ring_per + 31) / 32 * 32;
    const int slot = static_cast<int>(al ? ring_slot<true>(row_bytes) : ring_slot<false>(row_bytes));
    const int stage = inputs * slot, fit = (kRingBytes - static_cast<int>(ring_w_bytes(H))) / stage;
    int G = m.ring_threads / p.ring.threads;
    const bool one = !al && p.ring.threads == 32;
    const int most = one ? kRingStages / m.ring_stages : kRingGroups;
    if (G > most) G = most;
    if (G > fit) G = fit;
    if (G > 0 && fit > 1) {
      int S = kRingAhead / stage;
      if (S < m.ring_stages * G) S = m.ring_stages * G;
      if (S < 2) S = 2;
      if (S > fit) S = fit;
      if (S > kRingStages) S = kRingStages;
      p.kind = one ? kRingOne : kRing;
      p.ring.G = G;
      p.ring.S = S / G * G;
      p.threads = G * p.ring.threads + 32;
      p.grid = sms;
      return p;
    }
  }
  const int per = packs <= 1024 ? 1 : 2;
  if (packs > 2048) return p;
  p.kind = per == 1 ? kCtaFew : kCtaMost;
  p.threads = ((packs + per - 1) / per + 31) / 32 * 32;
  p.grid = few || T < sms ? T : sms;
  return p;
}
NormPlan norm_forward_plan(int T, int H, int dt, int inputs, bool al) {
  const int packs = static_cast<int>((static_cast<long long>(H) * dtype_bytes(dt) + 15) / 16);
  const int per = packs > kRingWide && (!al || (inputs == 1 && dt == kF32)) ? 4 : !al && packs > 64 && packs <= 96 ? 3 : kRingPer;
  const int threads = ring_threads(al), warps = threads / 32;
  return norm_plan(T, H, dt, NormLimits{128, 2, per, threads, warps < kRingWarps ? warps : kRingWarps, 1, 1 << 30}, inputs, al);
}
NormPlan norm_grad_plan(int T, int H, int dt, int inputs, bool al) {
  return norm_plan(T, H, dt, NormLimits{64, 1, kRingPer, kRingGradThreads, kRingGradWarps, 2, dt != kF32 && al ? 250000 : 350000},
                   inputs, al);
}

template <class K, class A>
cudaError_t ring_launch(K kernel, const A& a, const NormPlan& p, std::atomic<unsigned long long>& done, cudaStream_t stream) {
  const cudaError_t err = allow_smem(reinterpret_cast<const void*>(kernel), kRingSmem, done);
  if (err != cudaSuccess) return err;
  return launch_pdl(kernel, dim3(p.grid), dim3(p.threads), kRingSmem, stream, a, p.ring);
}

template <class T, bool AL, bool ONE, int PER>
cudaError_t norm_ring_launch(const NormArgs& a, const NormPlan& p, cudaStream_t stream) {
  static std::atomic<unsigned long long> done{0};
  return ring_launch(norm_ring_kernel<T, AL, ONE, PER>, a, p, done, stream);
}
template <class T, bool AL>
cudaError_t norm_ring_launch(const NormArgs& a, const NormPlan& p, cudaStream_t stream) {
  if constexpr (!AL) {
    if (p.kind == kRingOne)
      return p.ring.per == 2 ? norm_ring_launch<T, AL, true, 2>(a, p, stream) : norm_ring_launch<T, AL, true, 3>(a, p, stream);
  }
  if constexpr (!AL || Pack<T>::N == 4) {
    if (p.ring.per == 4) return norm_ring_launch<T, AL, false, 4>(a, p, stream);
  }
  return norm_ring_launch<T, AL, false, 2>(a, p, stream);
}

template <class T, bool AL>
cudaError_t norm_launch(const NormArgs& a, const NormPlan& p, cudaStream_t stream) {
  static std::atomic<unsigned long long> done{0};
  const auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(p.grid), dim3(p.threads), 0, stream, a); };
  switch (p.kind) {
    case kRing:
    case kRingOne: return norm_ring_launch<T, AL>(a, p, stream);
    case kWarpOne: return go(norm_kernel<T, AL, 1, true, 256, AL ? 4 : 2, true>);
    case kWarpMore:
      if constexpr (AL) return go(norm_kernel<T, AL, 4, true, 256, 2, true>);
      return cudaErrorInvalidValue;
    case kCtaFew: return go(norm_kernel<T, AL, 1, false, 1024, 1, false>);
    case kCtaMost: return go(norm_kernel<T, AL, 2, false, 1024, 1, false>);
    default: return go(norm_wide_kernel<T, AL>);
  }
}

int norm_slices(int T) { return T < 64 ? (T < 1 ? 1 : T) : 64; }      // of the wide rows' kernels

template <class T, bool AL>
cudaError_t norm_grad_launch(NormGradArgs a, const NormPlan& p, float* dw, cudaStream_t stream) {
  cudaError_t err;
  int slices = p.grid;
  static std::atomic<unsigned long long> done{0};
  if (p.kind == kRing || p.kind == kRingOne) {
    if (!dw) a.part = nullptr;
    if (p.kind == kRing) {
      err = ring_launch(norm_grad_ring_kernel<T, AL, false>, a, p, done, stream);
    } else {
      err = cudaErrorInvalidValue;
      if constexpr (!AL) {
        static std::atomic<unsigned long long> done_one{0};
        err = ring_launch(norm_grad_ring_kernel<T, AL, true>, a, p, done_one, stream);
      }
    }
  } else if (p.kind == kWide) {
    // the gradient of w first: dx may take the place of what it reads
    slices = norm_slices(a.T);
    void* dx = a.dx;
    if (dw) {
      a.dx = nullptr;
      err = launch_pdl(norm_grad_wide_kernel<T, AL>, dim3(a.T), dim3(kNormThreads), 0, stream, a);
      if (err != cudaSuccess) return err;
      err = launch_pdl(norm_dw_wide_kernel<T>, dim3((a.H + 255) / 256, slices), dim3(256), 0, stream, a);
      if (err != cudaSuccess) return err;
    }
    a.dx = dx;
    err = dx ? launch_pdl(norm_grad_wide_kernel<T, AL>, dim3(a.T), dim3(kNormThreads), 0, stream, a) : cudaSuccess;
  } else {
    if (!dw) a.part = nullptr;
    else if (slices == 1) a.part = dw;
    const auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(p.grid), dim3(p.threads), 0, stream, a); };
    switch (p.kind) {
      case kWarpOne: err = go(norm_grad_kernel<T, AL, 1, true, 256, 2, true>); break;
      case kWarpMore:
        err = cudaErrorInvalidValue;
        if constexpr (AL) err = go(norm_grad_kernel<T, AL, 2, true, 256, 2, true>);
        break;
      case kCtaFew: err = go(norm_grad_kernel<T, AL, 1, false, 1024, 1, false>); break;
      default: err = go(norm_grad_kernel<T, AL, 2, false, 1024, 1, false>); break;
    }
    if (slices == 1) return err;
  }
  if (err != cudaSuccess || !dw) return err;
  return launch_pdl(norm_dw_sum_kernel, dim3((a.H + 31) / 32), dim3(1024), 0, stream, static_cast<const float*>(a.part), slices,
                    a.H, dw);
}

}  // namespace

cudaError_t launch_norm(int dt, RowsView x, RowsView res, const float* w, float eps, int T, int H, RowsView sum, RowsView y,
                        Rows8View y8, cudaStream_t stream) {
  NormArgs a{};
  a.x = x.ptr;
  a.res = res.ptr;
  a.sum = sum.ptr;
  a.y = y.ptr;
  a.w = w;
  a.q = y8.q;
  a.sf = y8.sf;
  a.ldx = x.ld;
  a.ldr = res.ld;
  a.lds = sum.ld;
  a.ldy = y.ld;
  a.ldq = y8.ldq;
  a.ldsf = y8.lds;
  a.eps = eps;
  a.over_h = 1.f / static_cast<float>(H);
  a.T = T;
  a.H = H;
  const int n = static_cast<int>(16 / dtype_bytes(dt));
  a.q_words = codes_aligned(y8, T, n);
  const bool al = H % n == 0 && rows_aligned(x, T, dt) && rows_aligned(res, T, dt) && rows_aligned(sum, T, dt) &&
                  rows_aligned(y, T, dt);
  const NormPlan p = norm_forward_plan(T, H, dt, 1 + (res.ptr != nullptr), al);
  if (dt == kBf16) return al ? norm_launch<Bf16Elem, true>(a, p, stream) : norm_launch<Bf16Elem, false>(a, p, stream);
  if (dt == kF16) return al ? norm_launch<F16Elem, true>(a, p, stream) : norm_launch<F16Elem, false>(a, p, stream);
  return al ? norm_launch<F32Elem, true>(a, p, stream) : norm_launch<F32Elem, false>(a, p, stream);
}

// The wide rows' reciprocal roots [T], then the partial sums of dw.  The plans differ by type and alignment: room for any.
size_t norm_scratch_bytes(int T, int H) {
  size_t slices = 1;
  for (int dt = kBf16; dt <= kF32; ++dt) {
    for (int k = 0; k < 4; ++k) {
      const NormPlan p = norm_grad_plan(T, H, dt, 2 + k / 2, k % 2);
      const size_t n = static_cast<size_t>(p.kind == kWide ? norm_slices(T) : p.grid);
      if (n > slices) slices = n;
    }
  }
  return (static_cast<size_t>(T) * 4 + 255) / 256 * 256 + slices * H * 4;
}

cudaError_t launch_norm_grad(int dt, RowsView dy, RowsView x, const float* w, float eps, RowsView dsum, int T, int H,
                             RowsView dx, float* dw, void* scratch, uint32_t* status, cudaStream_t stream) {
  NormGradArgs a{};
  a.status = status;
  a.dy = dy.ptr;
  a.x = x.ptr;
  a.dsum = dsum.ptr;
  a.dx = dx.ptr;
  a.w = w;
  a.rs = static_cast<float*>(scratch);
  a.part = reinterpret_cast<float*>(static_cast<char*>(scratch) + (static_cast<size_t>(T) * 4 + 255) / 256 * 256);
  a.lddy = dy.ld;
  a.ldx = x.ld;
  a.lddsum = dsum.ld;
  a.lddx = dx.ld;
  a.eps = eps;
  a.over_h = 1.f / static_cast<float>(H);
  a.T = T;
  a.H = H;
  const int n = static_cast<int>(16 / dtype_bytes(dt));
  const bool al = H % n == 0 && rows_aligned(dy, T, dt) && rows_aligned(x, T, dt) && rows_aligned(dsum, T, dt) &&
                  rows_aligned(dx, T, dt);
  const NormPlan p = norm_grad_plan(T, H, dt, 2 + (dsum.ptr != nullptr), al);
  if (dt == kBf16) return al ? norm_grad_launch<Bf16Elem, true>(a, p, dw, stream) : norm_grad_launch<Bf16Elem, false>(a, p, dw, stream);
  if (dt == kF16) return al ? norm_grad_launch<F16Elem, true>(a, p, dw, stream) : norm_grad_launch<F16Elem, false>(a, p, dw, stream);
  return al ? norm_grad_launch<F32Elem, true>(a, p, dw, stream) : norm_grad_launch<F32Elem, false>(a, p, dw, stream);
}

}  // namespace moe
