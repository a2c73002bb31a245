// q2_fused_api.hip - the C ABI of the fused and grouped linears, the router and
// the combination: argument validation, device check, launch.  Every argument
// check runs before the first HIP call.
#include "q2.h"
#include "q2_fused_host.h"
#include "q2_internal.h"

namespace {

using namespace q2host;

int launch(const q2dev::FusedArgs& a, int fmt, void* ws, hipStream_t stream, const char* what) {
  return hip_status(q2dev::launch_fused(a, fmt, ws, stream), what);
}

int fused_entry(int fmt, const uint16_t* x, const uint8_t* w, const uint16_t* s, const uint16_t* z,
                const uint16_t* A, const uint16_t* B, int64_t r, const q2_epilogue* epi, void* y, int64_t M, int64_t N,
                int64_t K, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  int st = check_sizes(M, N, K);
  if (st || (st = check_linear_k(K))) return st;
  if (r < 0) return fail(Q2_ERR_ARG, "negative rank r=%lld", (long long)r);
  if (r > 65535) return fail(Q2_ERR_ARG, "rank r=%lld too large (at most 65535)", (long long)r);
  const q2_epilogue& e = epi ? *epi : kPlain;
  if ((st = check_epilogue(e, M, N, false))) return st;
  if ((st = check_ptr(x, M > 0 && K > 0, 16, "x")) || (st = check_ptr(w, N > 0 && K > 0, 16, "weights")) ||
      (st = check_ptr(s, N > 0 && K > 0, 2, "scales")) ||
      (fmt == 1 && (st = check_ptr(z, N > 0 && K > 0, 2, "zero points"))))
    return st;
  if (r > 0 && ((st = check_ptr(A, K > 0, 16, "A")) || (st = check_ptr(B, N > 0, 2, "B")))) return st;
  if ((st = check_ptr(y, M > 0 && N > 0, (e.flags & Q2_EPI_OUT_BF16) ? 2 : 4, "y"))) return st;
  if (M == 0 || N == 0) return ok();
  const size_t need = fmt == 0 ? q2_linear_fused_workspace_bytes(M, N, K, r) : 0;
  if ((st = check_workspace(workspace, workspace_bytes, need))) return st;
  const bool out16 = (e.flags & Q2_EPI_OUT_BF16) != 0, res16 = (e.flags & Q2_EPI_RESIDUAL_BF16) != 0;
  const int64_t n_out = (e.flags & Q2_EPI_GATED) ? N / 2 : N;
  if ((st = check_overlap(y, out16, M * n_out, x, M * K * 2, "x", e.residual, res16))) return st;
  if ((st = check_device())) return st;
  const size_t limbs = r > 0 ? q2_lowrank_workspace_bytes(M, r) : 0;
  q2dev::FusedArgs a = {};
  a.x = x; a.x_rows = M; a.w = w; a.s = s; a.z = z;
  a.E = 1; a.M = M; a.N = N; a.K = K;
  if (r > 0) {
    a.lr_a = A;
    a.lr_b = B;
    a.lr_t = static_cast<uint16_t*>(workspace);
    a.r = (int)r;
  }
  set_epilogue(a, e);
  a.y = y;
  return launch(a, fmt, need ? static_cast<uint8_t*>(workspace) + limbs : nullptr, stream, "fused linear launch");
}

int grouped_entry(int fmt, const uint16_t* x, int64_t x_rows, const int32_t* row_index, const int32_t* offsets,
                  const uint8_t* w, const uint16_t* s, const uint16_t* z, const q2_epilogue* epi, void* y, int64_t R,
                  int64_t E, int64_t N, int64_t K, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (E < 0 || x_rows < 0) return fail(Q2_ERR_ARG, "negative size (E=%lld x_rows=%lld)", (long long)E, (long long)x_rows);
  int st = check_sizes(R, N, K);
  if (st || (st = check_linear_k(K))) return st;
  if (E > 65536) return fail(Q2_ERR_SHAPE, "E=%lld exceeds 65536", (long long)E);
  if (R > 0x7fffffff || x_rows > 0x7fffffff) return fail(Q2_ERR_SHAPE, "more than 2^31 - 1 rows");
  if (E > 0 && (st = check_sizes(0, E * N, K))) return st;       // E * N stays far below 2^63: N <= 2^46
  if (row_index == nullptr && x_rows != R && R > 0)      // an index of no rows may be NULL
    return fail(Q2_ERR_ARG, "x_rows=%lld must be R=%lld without a row index", (long long)x_rows, (long long)R);
  const q2_epilogue& e = epi ? *epi : kPlain;
  if ((st = check_epilogue(e, R, N, true))) return st;
  const bool work = R > 0 && E > 0 && N > 0;
  if ((st = check_ptr(x, work && x_rows > 0 && K > 0, 16, "x")) ||
      (st = check_ptr(row_index, false, 4, "row_index")) || (st = check_ptr(offsets, work, 4, "offsets")) ||
      (st = check_ptr(w, work && K > 0, 16, "weights")) || (st = check_ptr(s, work && K > 0, 2, "scales")) ||
      (fmt == 1 && (st = check_ptr(z, work && K > 0, 2, "zero points"))) ||
      (st = check_ptr(y, work, (e.flags & Q2_EPI_OUT_BF16) ? 2 : 4, "y")))
    return st;
  if (!work) return ok();
  const size_t need = fmt == 0 ? q2_linear_grouped_workspace_bytes(R, E, N, K) : 0;
  if ((st = check_workspace(workspace, workspace_bytes, need))) return st;
  const int64_t n_out = (e.flags & Q2_EPI_GATED) ? N / 2 : N;
  if ((st = check_overlap(y, (e.flags & Q2_EPI_OUT_BF16) != 0, R * n_out, x, x_rows * K * 2, "x", nullptr, 0))) return st;
  if ((st = check_device())) return st;
  q2dev::FusedArgs a = {};
  a.x = x; a.x_rows = x_rows; a.row_index = row_index; a.w = w; a.s = s; a.z = z; a.offsets = offsets;
  a.E = E; a.M = R; a.N = N; a.K = K;
  set_epilogue(a, e);
  a.y = y;
  return launch(a, fmt, need ? workspace : nullptr, stream, "grouped linear launch");
}

// Sizes that a linear takes, for the workspace queries: no error, no message.
bool sizes_ok(int64_t M, int64_t N, int64_t K) {
  return M > 0 && N > 0 && K > 0 && K % 128 == 0 && K <= kMostK && sizes_fit(M, N, K);
}

bool route_sizes_ok(int64_t T, int64_t E, int64_t k) {
  return T >= 0 && E >= 1 && E <= 1024 && k >= 1 && k <= E && k <= 64 && T <= 0x7fffffff / k && T <= (1 << 26);
}

}  // namespace

extern "C" {

size_t q2_linear_fused_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t r) {
  if (M <= 0 || N <= 0 || r < 0 || r > 65535) return 0;
  const size_t limbs = r > 0 ? q2_lowrank_workspace_bytes(M, r) : 0;
  const size_t rest = sizes_ok(M, N, K) ? q2dev::fused_workspace_bytes(M, N, K, 0, 0) : 0;
  return limbs > SIZE_MAX - rest ? SIZE_MAX : limbs + rest;
}

int q2_linear_fused(const uint16_t* x_bf16, const uint8_t* packed, const uint16_t* scales_f16, const uint16_t* A_f16,
                    const uint16_t* B_f16, int64_t r, const q2_epilogue* epi, void* y, int64_t M, int64_t N, int64_t K,
                    void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return fused_entry(0, x_bf16, packed, scales_f16, nullptr, A_f16, B_f16, r, epi, y, M, N, K, workspace,
                     workspace_bytes, stream);
}

int q4_linear_fused(const uint16_t* x_bf16, const uint8_t* packed4, const uint16_t* scale_f16,
                    const uint16_t* zero_f16, const q2_epilogue* epi, void* y, int64_t M, int64_t N, int64_t K,
                    hipStream_t stream) {
  return fused_entry(1, x_bf16, packed4, scale_f16, zero_f16, nullptr, nullptr, 0, epi, y, M, N, K, nullptr, 0, stream);
}

size_t q2_linear_grouped_workspace_bytes(int64_t R, int64_t E, int64_t N, int64_t K) {
  if (E <= 0 || E > 65536 || R > 0x7fffffff || !sizes_ok(R, N, K) || !sizes_fit(0, E * N, K)) return 0;
  return q2dev::fused_workspace_bytes(R, N, K, E, 0);
}

int q2_linear_grouped(const uint16_t* x_bf16, int64_t x_rows, const int32_t* row_index, const int32_t* offsets,
                      const uint8_t* packed, const uint16_t* scales_f16, const q2_epilogue* epi, void* y, int64_t R,
                      int64_t E, int64_t N, int64_t K, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return grouped_entry(0, x_bf16, x_rows, row_index, offsets, packed, scales_f16, nullptr, epi, y, R, E, N, K,
                       workspace, workspace_bytes, stream);
}

int q4_linear_grouped(const uint16_t* x_bf16, int64_t x_rows, const int32_t* row_index, const int32_t* offsets,
                      const uint8_t* packed4, const uint16_t* scale_f16, const uint16_t* zero_f16,
                      const q2_epilogue* epi, void* y, int64_t R, int64_t E, int64_t N, int64_t K,
                      hipStream_t stream) {
  return grouped_entry(1, x_bf16, x_rows, row_index, offsets, packed4, scale_f16, zero_f16, epi, y, R, E, N, K,
                       nullptr, 0, stream);
}

size_t q2_route_workspace_bytes(int64_t T, int64_t E, int64_t k) {
  return T > 0 && route_sizes_ok(T, E, k) ? q2dev::route_workspace_bytes(T, E) : 0;
}

int q2_route(const void* logits, int64_t T, int64_t E, int64_t k, uint32_t flags, int32_t* expert, float* weight,
             int32_t* offsets, int32_t* row_token, int32_t* slot, void* workspace, size_t workspace_bytes,
             hipStream_t stream) {
  if (T < 0 || E < 0 || k < 0)
    return fail(Q2_ERR_ARG, "negative size (T=%lld E=%lld k=%lld)", (long long)T, (long long)E, (long long)k);
  const uint32_t known = Q2_ROUTE_LOGITS_BF16 | Q2_ROUTE_RENORM;
  if (flags & ~known) return fail(Q2_ERR_ARG, "unknown route flag bits 0x%x", flags & ~known);
  if (!route_sizes_ok(T, E, k))
    return fail(Q2_ERR_SHAPE, "T=%lld E=%lld k=%lld: 1 <= k <= min(E, 64), E <= 1024, T <= 2^26, T * k < 2^31", (long long)T,
                (long long)E, (long long)k);
  int st;
  const bool ne = T > 0;
  if ((st = check_ptr(logits, ne, (flags & Q2_ROUTE_LOGITS_BF16) ? 2 : 4, "logits")) ||
      (st = check_ptr(expert, ne, 4, "expert")) || (st = check_ptr(weight, ne, 4, "weight")) ||
      (st = check_ptr(offsets, true, 4, "offsets")) || (st = check_ptr(row_token, ne, 4, "row_token")) ||
      (st = check_ptr(slot, ne, 4, "slot")))
    return st;
  if ((st = check_workspace(workspace, workspace_bytes, q2_route_workspace_bytes(T, E, k)))) return st;
  if ((st = check_device())) return st;
  return hip_status(q2dev::launch_route(logits, (flags & Q2_ROUTE_LOGITS_BF16) ? 1 : 0, T, E, (int)k,
                                        (flags & Q2_ROUTE_RENORM) ? 1 : 0, expert, weight, offsets, row_token, slot,
                                        workspace, stream),
                    "route launch");
}

int q2_combine(const void* z, int64_t R, const int32_t* slot, const float* weight, const void* residual, void* y,
               int64_t T, int64_t k, int64_t N, uint32_t flags, hipStream_t stream) {
  if (R < 0 || T < 0 || k < 0 || N < 0)
    return fail(Q2_ERR_ARG, "negative size (R=%lld T=%lld k=%lld N=%lld)", (long long)R, (long long)T, (long long)k,
                (long long)N);
  const uint32_t known = Q2_COMBINE_Z_BF16 | Q2_COMBINE_OUT_BF16 | Q2_COMBINE_RESIDUAL_BF16;
  if (flags & ~known) return fail(Q2_ERR_ARG, "unknown combine flag bits 0x%x", flags & ~known);
  if (k > 64) return fail(Q2_ERR_SHAPE, "k=%lld exceeds 64", (long long)k);
  const int64_t lim = (int64_t)1 << 46;
  if (R > 0x7fffffff || T > lim || N > lim || (T > 0 && N > lim / T) || (R > 0 && N > lim / R))
    return fail(Q2_ERR_SHAPE, "sizes too large");
  int st;
  const bool ne = T > 0 && N > 0;
  if ((st = check_ptr(z, ne && R > 0 && k > 0, (flags & Q2_COMBINE_Z_BF16) ? 2 : 4, "z")) ||
      (st = check_ptr(slot, ne && k > 0, 4, "slot")) || (st = check_ptr(weight, ne && k > 0, 4, "weight")) ||
      (st = check_ptr(residual, false, (flags & Q2_COMBINE_RESIDUAL_BF16) ? 2 : 4, "residual")) ||
      (st = check_ptr(y, ne, (flags & Q2_COMBINE_OUT_BF16) ? 2 : 4, "y")))
    return st;
  if (!ne) return ok();
  if ((st = check_overlap(y, (flags & Q2_COMBINE_OUT_BF16) != 0, T * N, k > 0 ? z : nullptr,
                          R * N * ((flags & Q2_COMBINE_Z_BF16) ? 2 : 4), "z", residual,
                          (flags & Q2_COMBINE_RESIDUAL_BF16) != 0)))
    return st;
  if ((st = check_device())) return st;
  return hip_status(q2dev::launch_combine(z, (flags & Q2_COMBINE_Z_BF16) ? 1 : 0, R, slot, weight, residual,
                                          (flags & Q2_COMBINE_RESIDUAL_BF16) ? 1 : 0, y,
                                          (flags & Q2_COMBINE_OUT_BF16) ? 1 : 0, T, (int)k, N, stream),
                    "combine launch");
}

}  // extern "C"
