// q2_token_api.hip - the C ABI of the 4-bit products with scales per group and of the
// sampler: argument validation, device check, launch.  Every argument check runs
// before the first HIP call.
#include "q2.h"
#include "q2_fused_host.h"
#include "q2_token.h"

namespace {

using namespace q2host;

bool sample_sizes_ok(int64_t B, int64_t V) { return B >= 0 && B <= (1 << 30) && V >= 1 && V <= (1 << 24); }

// An output of B 4-byte elements against B rows of row_bytes, pitch bytes apart: what lies
// between the rows is not theirs.
bool overlaps_rows(const void* out, int64_t B, const void* rows, int64_t row_bytes, int64_t pitch) {
  if (!overlap(out, 4 * B, rows, (B - 1) * pitch + row_bytes)) return false;
  const uintptr_t o = reinterpret_cast<uintptr_t>(out), r = reinterpret_cast<uintptr_t>(rows);
  if (o < r) return true;                                // reaches the first row
  const int64_t row = (int64_t)(o - r) / pitch, at = (int64_t)(o - r) % pitch;
  return at < row_bytes || (row + 1 < B && at + 4 * B > pitch);
}

// Outputs are written while other rows' inputs are read.  u may be an output itself: a
// row's is read before its token and probability are written.
int check_outputs(const q2_sampling& c, const void* logits, int64_t row_bytes, int64_t pitch, int64_t B, const float* u,
                  const int32_t* token, const float* prob) {
  if (overlap(token, 4 * B, prob, 4 * B)) return fail(Q2_ERR_ARG, "token overlaps prob");
  const struct {
    const void* p;
    const char* name;
  } outs[] = {{token, "token"}, {prob, "prob"}},
    ins[] = {{c.temperature_rows, "temperature"}, {c.top_k_rows, "top_k"}, {c.top_p_rows, "top_p"}, {c.min_p_rows, "min_p"}};
  for (const auto& out : outs) {
    if (overlaps_rows(out.p, B, logits, row_bytes, pitch)) return fail(Q2_ERR_ARG, "%s overlaps the logits", out.name);
    if (out.p != u && overlap(out.p, 4 * B, u, 4 * B)) return fail(Q2_ERR_ARG, "%s overlaps u without being it", out.name);
    for (const auto& in : ins)
      if (in.p && overlap(out.p, 4 * B, in.p, 4 * B)) return fail(Q2_ERR_ARG, "%s overlaps %s", out.name, in.name);
  }
  return Q2_OK;
}

}  // namespace

extern "C" {

int q4_matvec(const uint16_t* x_bf16, const uint8_t* packed4, const uint16_t* scale_f16, const void* zero,
              int64_t group, uint32_t flags, const q2_epilogue* epi, void* y, int64_t M, int64_t N, int64_t K,
              hipStream_t stream) {
  if (M < 0 || N < 0 || K < 0)
    return fail(Q2_ERR_ARG, "negative size (M=%lld N=%lld K=%lld)", (long long)M, (long long)N, (long long)K);
  if (flags & ~Q4_ZERO_CODES) return fail(Q2_ERR_ARG, "unknown flag bits 0x%x", flags & ~Q4_ZERO_CODES);
  if (group <= 0 || (group != 32 && group != 64 && group % 128 != 0))
    return fail(Q2_ERR_SHAPE, "group=%lld is not 32, 64 or a multiple of 128", (long long)group);
  if (K % group != 0) return fail(Q2_ERR_SHAPE, "K=%lld is not a multiple of the group %lld", (long long)K, (long long)group);
  if (!sizes_fit(M, N, K)) return fail(Q2_ERR_ARG, "sizes too large");
  int st = check_linear_k(K);
  if (st) return st;
  const q2_epilogue& e = epi ? *epi : kPlain;
  if ((st = check_epilogue(e, M, N, false))) return st;
  const bool codes = (flags & Q4_ZERO_CODES) != 0, out16 = (e.flags & Q2_EPI_OUT_BF16) != 0;
  if (codes && zero == nullptr && N > 0 && K > 0) return fail(Q2_ERR_ARG, "zero points are NULL");
  if ((st = check_ptr(x_bf16, M > 0 && K > 0, 16, "x")) || (st = check_ptr(packed4, N > 0 && K > 0, 16, "weights")) ||
      (st = check_ptr(scale_f16, N > 0 && K > 0, 2, "scales")) ||
      (st = check_ptr(zero, false, codes ? 1 : 2, "zero points")) ||
      (st = check_ptr(y, M > 0 && N > 0, out16 ? 2 : 4, "y")))
    return st;
  if (M == 0 || N == 0) return ok();
  const int64_t n_out = (e.flags & Q2_EPI_GATED) ? N / 2 : N;
  if ((st = check_overlap(y, out16, M * n_out, x_bf16, M * K * 2, "x", e.residual,
                          (e.flags & Q2_EPI_RESIDUAL_BF16) != 0)))
    return st;
  if ((st = check_device())) return st;
  q2dev::MatvecArgs a = {};
  a.f.x = x_bf16; a.f.x_rows = M; a.f.w = packed4; a.f.s = scale_f16;
  a.f.E = 1; a.f.M = M; a.f.N = N; a.f.K = K;
  a.group = group;
  a.zero = zero == nullptr ? q2dev::ZERO_8 : codes ? q2dev::ZERO_CODES : q2dev::ZERO_F16;
  if (codes) a.zero_codes = static_cast<const uint8_t*>(zero);
  else a.f.z = static_cast<const uint16_t*>(zero);
  set_epilogue(a.f, e);
  a.f.y = y;
  return hip_status(q2dev::launch_q4_matvec(a, stream), "4-bit product launch");
}

size_t q2_sample_workspace_bytes(int64_t B, int64_t V) {
  return B > 0 && sample_sizes_ok(B, V) ? q2dev::sample_workspace_bytes(B, V) : 0;
}

int q2_sample(const void* logits, int64_t B, int64_t V, int64_t ld, uint32_t flags, const q2_sampling* settings,
              const float* u, int32_t* token, float* prob, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (B < 0 || V < 0) return fail(Q2_ERR_ARG, "negative size (B=%lld V=%lld)", (long long)B, (long long)V);
  if (flags & ~Q2_SAMPLE_LOGITS_BF16) return fail(Q2_ERR_ARG, "unknown sample flag bits 0x%x", flags & ~Q2_SAMPLE_LOGITS_BF16);
  if (!sample_sizes_ok(B, V)) return fail(Q2_ERR_SHAPE, "B=%lld V=%lld: 1 <= V <= 2^24, B <= 2^30",
                                                           (long long)B, (long long)V);
  if (B > 1 && (ld < V || ld > ((int64_t)1 << 46) / B))
    return fail(Q2_ERR_ARG, "ld=%lld: rows of V=%lld logits overlap or lie too far apart", (long long)ld, (long long)V);
  const q2_sampling none = {1.f, 0, 1.f, 0.f, nullptr, nullptr, nullptr, nullptr};
  const q2_sampling& c = settings ? *settings : none;
  const bool bf16 = (flags & Q2_SAMPLE_LOGITS_BF16) != 0;
  int st;
  if ((st = check_ptr(logits, B > 0, bf16 ? 2 : 4, "logits")) || (st = check_ptr(u, B > 0, 4, "u")) ||
      (st = check_ptr(c.temperature_rows, false, 4, "temperature")) || (st = check_ptr(c.top_k_rows, false, 4, "top_k")) ||
      (st = check_ptr(c.top_p_rows, false, 4, "top_p")) || (st = check_ptr(c.min_p_rows, false, 4, "min_p")) ||
      (st = check_ptr(token, B > 0, 4, "token")) || (st = check_ptr(prob, B > 0, 4, "prob")))
    return st;
  if (B == 0) return ok();
  if ((st = check_workspace(workspace, workspace_bytes, q2_sample_workspace_bytes(B, V)))) return st;
  const int64_t size = bf16 ? 2 : 4;
  if ((st = check_outputs(c, logits, V * size, (B > 1 ? ld : V) * size, B, u, token, prob))) return st;
  if ((st = check_device())) return st;
  q2dev::SampleArgs a = {};
  a.logits = logits;
  a.bf16 = bf16;
  a.B = B; a.V = V; a.ld = ld;
  a.u = u;
  a.temperature = c.temperature_rows; a.temperature_all = c.temperature;
  a.top_k = c.top_k_rows; a.top_k_all = c.top_k;
  a.top_p = c.top_p_rows; a.top_p_all = c.top_p;
  a.min_p = c.min_p_rows; a.min_p_all = c.min_p;
  a.token = token;
  a.prob = prob;
  return hip_status(q2dev::launch_sample(a, workspace, stream), "sample launch");
}

}  // extern "C"
