// q2_token.h - arguments of the 4-bit products with scales per group and of the
// sampler of tokens.
#pragma once
#include "q2_fused.h"

namespace q2dev {

// y = epilogue(x W^T) with weights (q - zero) * scale.  f.s: f16 scales [N, K / group];
// the zero point of a group is 8 (ZERO_8), a 4-bit code of zero_codes [N, ceil(K / group / 2)]
// (ZERO_CODES) or f.z, f16 [N, K / group] (ZERO_F16).  f has one group of rows and no branch.
enum { ZERO_8 = 0, ZERO_CODES = 1, ZERO_F16 = 2 };
struct MatvecArgs {
  FusedArgs f;
  const uint8_t* zero_codes;
  int64_t group;
  int zero;
};
hipError_t launch_q4_matvec(const MatvecArgs& a, hipStream_t stream);

// One draw for each of B rows of V logits, ld elements apart.  A setting is the
// array's element of the row or, without an array, the value.
struct SampleArgs {
  const void* logits;
  int bf16;
  int64_t B, V, ld;
  const float* u;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  float temperature_all, top_p_all, min_p_all;
  int32_t top_k_all;
  int32_t* token;
  float* prob;
};
size_t sample_workspace_bytes(int64_t B, int64_t V);
hipError_t launch_sample(const SampleArgs& a, void* workspace, hipStream_t stream);

}  // namespace q2dev
