// q2_fused_host.h - argument checks shared by the host files of the entry points
// that take an epilogue, a workspace or a residual that may be the output.
#pragma once
#include "q2_fused.h"
#include "q2_host.h"

namespace q2host {

inline const q2_epilogue kPlain = {Q2_ACT_NONE, 0u, nullptr, nullptr, nullptr};

inline int check_epilogue(const q2_epilogue& e, int64_t M, int64_t N, bool grouped) {
  if (e.activation > Q2_ACT_SILU) return fail(Q2_ERR_ARG, "unknown activation %u", e.activation);
  const uint32_t known = Q2_EPI_GATED | Q2_EPI_OUT_BF16 | Q2_EPI_RESIDUAL_BF16;
  if (e.flags & ~known) return fail(Q2_ERR_ARG, "unknown epilogue flag bits 0x%x", e.flags & ~known);
  if ((e.flags & Q2_EPI_GATED) && N % 2 != 0)
    return fail(Q2_ERR_SHAPE, "N=%lld is odd: a gated weight has two equal halves", (long long)N);
  if (grouped && (e.gate || e.residual)) return fail(Q2_ERR_ARG, "a grouped linear takes no gate and no residual");
  int st = check_ptr(e.bias, false, 4, "bias");
  if (st || (st = check_ptr(e.gate, false, 4, "gate"))) return st;
  return check_ptr(e.residual, false, (e.flags & Q2_EPI_RESIDUAL_BF16) ? 2 : 4, "residual");
}

inline void set_epilogue(q2dev::FusedArgs& a, const q2_epilogue& e) {
  a.act = (int)e.activation;
  a.gated = (e.flags & Q2_EPI_GATED) ? 1 : 0;
  a.out_bf16 = (e.flags & Q2_EPI_OUT_BF16) ? 1 : 0;
  a.res_bf16 = (e.flags & Q2_EPI_RESIDUAL_BF16) ? 1 : 0;
  a.bias = e.bias;
  a.gate = e.gate;
  a.residual = e.residual;
}

inline int check_workspace(const void* ws, size_t bytes, size_t need) {
  if (bytes < need) return fail(Q2_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", bytes, need);
  if (need > 0 && ws == nullptr) return fail(Q2_ERR_ARG, "workspace is NULL");
  if (need > 0 && !aligned(ws, 256)) return fail(Q2_ERR_ALIGN, "workspace is not 256-byte aligned");
  return Q2_OK;
}

inline bool overlap(const void* p, int64_t bytes_p, const void* q, int64_t bytes_q) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return bytes_p > 0 && bytes_q > 0 && (a < b ? b - a < (uintptr_t)bytes_p : a - b < (uintptr_t)bytes_q);
}

// y of `count` elements against an input that other workgroups read, and against
// the residual, which may be y itself.
inline int check_overlap(const void* y, int y_bf16, int64_t count, const void* in, int64_t in_bytes, const char* name,
                  const void* residual, int res_bf16) {
  const int64_t bytes = count * (y_bf16 ? 2 : 4);
  if (in && overlap(y, bytes, in, in_bytes)) return fail(Q2_ERR_ARG, "y overlaps %s", name);
  if (residual && !(residual == y && res_bf16 == y_bf16) && overlap(y, bytes, residual, count * (res_bf16 ? 2 : 4)))
    return fail(Q2_ERR_ARG, "y overlaps the residual without being it, address and type");
  return Q2_OK;
}

}  // namespace q2host
