// C ABI of the training operators (declarations and contracts in include/moe.h): host-side checks,
// workspace layout, and launches on the caller's stream.
#include "../../include/moe.h"
#include "kernels.h"

using namespace moe;

namespace {

constexpr size_t kAlign = 256;
constexpr long long kMaxLd = 1LL << 36;      // elements; the tensor maps take strides below 2^40 bytes
inline size_t up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline uint32_t* status_of(void* ws) { return static_cast<uint32_t*>(ws); }
inline cudaStream_t S(void* s) { return static_cast<cudaStream_t>(s); }
inline moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
inline RowsView view(const moe_rows& m) { return RowsView{m.ptr, static_cast<long long>(m.ld)}; }

bool dtype_ok(moe_dtype dt) { return dt == MOE_BF16 || dt == MOE_F16 || dt == MOE_F32; }

// A matrix with `cols` columns of the type: given, element-aligned, pitch at least its width.
bool rows_ok(const moe_rows& m, int cols, moe_dtype dt) {
  return m.ptr && m.ld >= cols && m.ld <= kMaxLd && aligned(m.ptr, dtype_bytes(dt));
}
bool opt_rows_ok(const moe_rows& m, int cols, moe_dtype dt) { return !m.ptr || rows_ok(m, cols, dt); }
// The same for a 16-bit matrix that the products read or write: every row on a 16-byte boundary.
bool rows16_ok(const moe_rows& m, int cols) { return rows_ok(m, cols, MOE_BF16) && m.ld % 8 == 0 && aligned(m.ptr, 16); }
bool opt_rows16_ok(const moe_rows& m, int cols) { return !m.ptr || rows16_ok(m, cols); }

// T tokens to K sorted rows each, of H columns, in buffers of U rows.
bool sorted_dims_ok(int T, int K, int H, int U) {
  return T >= 0 && K >= 1 && K <= 32 && H >= 1 && U >= 0 && static_cast<long long>(T) * K <= 0x7fffffff;
}

bool pow2_align(int a) { return a >= 1 && a <= 256 && (a & (a - 1)) == 0; }

struct LinearWs {
  size_t maps = 0, dz = 0, part = 0, total = 0;
};

bool linear_dims_ok(int rows, int N, int K, int E, int act) {
  if (rows < 0 || N <= 0 || K <= 0 || E < 0 || E > kLinearMaxExperts) return false;
  if (act < kActNone || act > kActSwiglu) return false;
  if (K % 8 || N % 8 || (act == kActSwiglu && N % 16)) return false;
  // tile and segment arithmetic is 32-bit
  return rows <= (1 << 28) && N <= (1 << 24) && K <= (1 << 24);
}

LinearWs linear_layout(int rows, int N, int E, int act) {
  LinearWs w;
  size_t off = kAlign;                         // [0, 256): status word
  w.maps = off;
  off = up(off + static_cast<size_t>(E) * kLinearMapBytes);
  w.dz = off;
  if (act != kActNone) off = up(off + static_cast<size_t>(rows) * N * 2);
  w.part = off;
  off = up(off + static_cast<size_t>(E > 0 ? E : 1) * linear_bias_slices(rows, N, E, act) * N * 4);
  w.total = off;
  return w;
}

// The shape checks the two linear calls share.
moe_status linear_common(moe_dtype dt, const int32_t* counts, int rows, int N, int K, int E, int align, moe_act act,
                         const void* ws) {
  if (!dtype_ok(dt) || !linear_dims_ok(rows, N, K, E, act)) return MOE_ERR_INVALID_ARG;
  if (dt == MOE_F32) return MOE_ERR_UNSUPPORTED;
  if ((E > 0) != (counts != nullptr) || (E > 0 && !pow2_align(align))) return MOE_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, kAlign)) return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

LinearShape linear_shape(moe_dtype dt, const int32_t* counts, int rows, int N, int K, int E, int align) {
  LinearShape p{};
  p.rows = rows;
  p.N = N;
  p.K = K;
  p.E = E;
  p.align = align;
  p.f16 = dt == MOE_F16;
  p.counts = counts;
  return p;
}

}  // namespace

extern "C" {

moe_status moe_workspace_size_rows(int T, int K, int E, size_t* bytes) {
  if (!bytes || !sorted_dims_ok(T, K, 1, 0) || E < 1 || K > E) return MOE_ERR_INVALID_ARG;
  *bytes = up(kAlign + permute_scratch_bytes(T, K, E));
  return MOE_OK;
}

moe_status moe_dispatch(moe_dtype dt, const int32_t* topk_ids, moe_rows x, int T, int H, int E, int K, int align,
                        moe_rows x_perm, int32_t* sorted_token_ids, int32_t* expert_ids, int32_t* inv_perm,
                        int32_t* m_sum, int32_t* expert_counts, void* ws, size_t ws_bytes, void* stream) {
  if (!dtype_ok(dt) || !sorted_dims_ok(T, K, H, 0) || E < 1 || K > E || !pow2_align(align)) return MOE_ERR_INVALID_ARG;
  if (E > 1024) return MOE_ERR_UNSUPPORTED;
  const size_t U = moe_msum_upper(T, K, E, align);
  if (U > 0x7fffffff) return MOE_ERR_INVALID_ARG;
  if (!m_sum || (U > 0 && (!sorted_token_ids || !expert_ids))) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!topk_ids || !inv_perm || !rows_ok(x, H, dt) || !rows_ok(x_perm, H, dt))) return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < kAlign + permute_scratch_bytes(T, K, E)) return MOE_ERR_WORKSPACE;
  if (dispatch_layout_supported(T, K, E))
    return cuda_status(launch_dispatch_layout(dt, topk_ids, view(x), T, H, E, K, align, static_cast<int>(U), view(x_perm),
                                              sorted_token_ids, expert_ids, inv_perm, m_sum, expert_counts,
                                              status_of(ws), S(stream)));
  int32_t* scratch = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + kAlign);
  const cudaError_t err =
      launch_permute(topk_ids, T, K, E, align, static_cast<int>(U), sorted_token_ids, expert_ids, inv_perm, m_sum,
                     expert_counts, nullptr, nullptr, 0, nullptr, nullptr, status_of(ws), scratch, S(stream));
  if (err != cudaSuccess) return MOE_ERR_CUDA;
  return cuda_status(launch_scatter_rows(dt, view(x), inv_perm, T, K, H, static_cast<int>(U), view(x_perm), status_of(ws),
                                         S(stream)));
}

moe_status moe_dispatch_backward(moe_dtype dt, moe_rows dx_perm, const int32_t* inv_perm, moe_rows residual, int T, int H,
                                 int K, int U, moe_rows dx, void* ws, size_t ws_bytes, void* stream) {
  return moe_combine(dt, dx_perm, inv_perm, nullptr, residual, T, H, K, U, dx, ws, ws_bytes, stream);
}

moe_status moe_combine(moe_dtype dt, moe_rows y_perm, const int32_t* inv_perm, const float* topk_w, moe_rows residual,
                       int T, int H, int K, int U, moe_rows out, void* ws, size_t ws_bytes, void* stream) {
  if (!dtype_ok(dt) || !sorted_dims_ok(T, K, H, U)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!inv_perm || !rows_ok(y_perm, H, dt) || !rows_ok(out, H, dt) || !opt_rows_ok(residual, H, dt)) return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < kAlign) return MOE_ERR_WORKSPACE;
  return cuda_status(launch_sum_rows(dt, view(y_perm), inv_perm, topk_w, view(residual), T, K, H, U, view(out),
                                     status_of(ws), S(stream)));
}

moe_status moe_combine_backward(moe_dtype dt, moe_rows dout, moe_rows y_perm, const int32_t* inv_perm,
                                const float* topk_w, int T, int H, int K, int U, moe_rows dy_perm, float* dtopk_w,
                                void* ws, size_t ws_bytes, void* stream) {
  if (!dtype_ok(dt) || !sorted_dims_ok(T, K, H, U)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!inv_perm || !rows_ok(dout, H, dt) || !rows_ok(dy_perm, H, dt)) return MOE_ERR_INVALID_ARG;
  // y_perm is read for the weights' gradient alone; a plain sum (topk_w NULL) has none
  if ((dtopk_w != nullptr) != (y_perm.ptr != nullptr) || !opt_rows_ok(y_perm, H, dt)) return MOE_ERR_INVALID_ARG;
  if (dtopk_w && !topk_w) return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < kAlign) return MOE_ERR_WORKSPACE;
  return cuda_status(launch_combine_grad(dt, view(dout), view(y_perm), inv_perm, topk_w, T, K, H, U, view(dy_perm),
                                         dtopk_w, status_of(ws), S(stream)));
}

moe_status moe_route_backward(const float* logits, const int32_t* topk_ids, const float* topk_w, const float* dtopk_w,
                              int T, int E, int K, moe_score_fn fn, int renormalize, moe_dtype dt, void* dlogits, void* ws,
                              size_t ws_bytes, void* stream) {
  if (!dtype_ok(dt) || !sorted_dims_ok(T, K, 1, 0) || E < 1 || E > 1024 || K > E) return MOE_ERR_INVALID_ARG;
  if (fn != MOE_SCORE_SOFTMAX && fn != MOE_SCORE_SQRT_SOFTPLUS) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_ids || !topk_w || !dtopk_w || !dlogits) return MOE_ERR_INVALID_ARG;
  if (!aligned(logits, 16) || !aligned(dlogits, 16)) return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < kAlign) return MOE_ERR_WORKSPACE;
  return cuda_status(launch_route_grad(dt, logits, topk_ids, topk_w, dtopk_w, T, E, K, fn == MOE_SCORE_SOFTMAX,
                                       renormalize != 0, dlogits, status_of(ws), S(stream)));
}

moe_status moe_workspace_size_linear(int rows, int N, int K, int E, moe_act act, size_t* bytes) {
  if (!bytes || !linear_dims_ok(rows, N, K, E, act)) return MOE_ERR_INVALID_ARG;
  *bytes = linear_layout(rows, N, E, act).total;
  return MOE_OK;
}

moe_status moe_linear(moe_dtype dt, moe_rows x, const void* w, const float* bias, moe_rows residual, moe_act act,
                      const int32_t* expert_counts, int rows, int N, int K, int E, int align, moe_rows y, moe_rows z,
                      void* ws, size_t ws_bytes, void* stream) {
  const moe_status st = linear_common(dt, expert_counts, rows, N, K, E, align, act, ws);
  if (st != MOE_OK) return st;
  const int cols = act == MOE_ACT_SWIGLU ? N / 2 : N;
  if (rows == 0) return MOE_OK;
  if (!rows16_ok(x, K) || !w || !aligned(w, 16) || !rows16_ok(y, cols)) return MOE_ERR_INVALID_ARG;
  if (!opt_rows16_ok(residual, cols) || !opt_rows16_ok(z, N)) return MOE_ERR_INVALID_ARG;
  if (bias && !aligned(bias, 16)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < kAlign + E * kLinearMapBytes) return MOE_ERR_WORKSPACE;
  return cuda_status(launch_linear(linear_shape(dt, expert_counts, rows, N, K, E, align), view(x),
                                   static_cast<const uint16_t*>(w), bias, view(residual), act, view(y), view(z),
                                   static_cast<char*>(ws) + kAlign, status_of(ws), S(stream)));
}

moe_status moe_linear_backward(moe_dtype dt, moe_rows dy, moe_rows x, const void* w, moe_rows z, moe_act act,
                               const int32_t* expert_counts, int rows, int N, int K, int E, int align,
                               moe_rows dx_residual, moe_rows dx, void* dw, float* dbias, void* ws, size_t ws_bytes,
                               void* stream) {
  const moe_status st = linear_common(dt, expert_counts, rows, N, K, E, align, act, ws);
  if (st != MOE_OK) return st;
  const int cols = act == MOE_ACT_SWIGLU ? N / 2 : N;
  if (!dx.ptr && !dw && !dbias && rows > 0) return MOE_ERR_INVALID_ARG;
  if ((dw && !aligned(dw, 16)) || (dbias && !aligned(dbias, 16))) return MOE_ERR_INVALID_ARG;
  const int En = E > 0 ? E : 1;
  if (rows == 0) {            // no rows: the sums over them are zero
    if (dw && cudaMemsetAsync(dw, 0, static_cast<size_t>(En) * N * K * 2, S(stream)) != cudaSuccess) return MOE_ERR_CUDA;
    if (dbias && cudaMemsetAsync(dbias, 0, static_cast<size_t>(En) * N * 4, S(stream)) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  if (!rows16_ok(dy, cols) || (act != MOE_ACT_NONE ? !rows16_ok(z, N) : z.ptr != nullptr)) return MOE_ERR_INVALID_ARG;
  if (dx.ptr && (!rows16_ok(dx, K) || !w || !aligned(w, 16))) return MOE_ERR_INVALID_ARG;
  if (!opt_rows16_ok(dx_residual, K) || (dx_residual.ptr && !dx.ptr)) return MOE_ERR_INVALID_ARG;
  if (dw && !rows16_ok(x, K)) return MOE_ERR_INVALID_ARG;
  const LinearWs L = linear_layout(rows, N, E, act);
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  const LinearShape p = linear_shape(dt, expert_counts, rows, N, K, E, align);
  char* base = static_cast<char*>(ws);
  RowsView dz = view(dy);
  if (act != MOE_ACT_NONE) dz = RowsView{base + L.dz, N};
  if (act != MOE_ACT_NONE || dbias) {
    if (launch_act_grad(p, view(dy), view(z), act, dz, reinterpret_cast<float*>(base + L.part), dbias, status_of(ws),
                        S(stream)) != cudaSuccess)
      return MOE_ERR_CUDA;
  }
  if (dx.ptr && launch_linear_dx(p, dz, static_cast<const uint16_t*>(w), view(dx_residual), view(dx),
                                 base + L.maps, status_of(ws),
                                 S(stream)) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (dw && launch_linear_dw(p, dz, view(x), static_cast<uint16_t*>(dw), base + L.maps, status_of(ws), S(stream)) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_OK;
}

}  // extern "C"
