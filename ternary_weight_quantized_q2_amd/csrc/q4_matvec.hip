// q4_matvec.hip - the launch of the 4-bit products with scales per group, and the plain
// kernel for weights of few inputs.
#include "q4_matvec.h"

namespace q2dev {

constexpr int MV_BM = 16, MV_BN = 64;

// A workgroup owns 16 rows x 64 weight columns; each of its four waves 16 of the
// columns, 32 inputs at a time, straight from global memory.  For what the other
// kernel's loads and grid do not take: one row, K = 2560, N = 2 x 9728 took 40 us here.
__global__ __launch_bounds__(256) void matvec_tile_kernel(MatvecArgs m, int tiles_n) {
  const FusedArgs& a = m.f;
  __shared__ float out[MV_BM][MV_BN + 4];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int c = lane & 15, g = lane >> 4;
  RowTile rt;
  int tn;
  if (!find_tile(a, MV_BM, tiles_n, 1, rt, tn)) return;
  const int64_t n_out = fused_n_out(a), K = a.K;
  const int out_cols = a.gated ? MV_BN / 2 : MV_BN;
  const int64_t n0 = (int64_t)tn * out_cols;
  // Sums of x are of up to 128 inputs, of which a group may have many.
  const int groups = (int)(K / m.group), blocks = m.group > BLOCK_K ? (int)(m.group / BLOCK_K) : 1;
  const int steps = (int)(m.group / blocks / 32);
  const NatConsts kc = q4_nat_consts();

  const int cb = 16 * wv + c;
  const bool up = a.gated && cb >= MV_BN / 2;
  int64_t n = n0 + (up ? cb - MV_BN / 2 : cb);
  n = n < n_out ? n : n_out - 1;
  if (up) n += n_out;
  const uint8_t* wp = a.w + n * (K / 2) + 4 * g;
  const uint16_t* sp = a.s + n * groups;
  const int64_t row = std::min<int64_t>(rt.m0 + c, rt.mend - 1);
  const uint16_t* xp = a.x + row * K + 8 * g;

  const uint32_t sone = m.zero == ZERO_8 ? 0x3FC03FC0u : 0x3F803F80u;     // bf16 1.5 / 1 pairs
  const q2_u32x4 sones = q2_u32x4{sone, sone, sone, sone};
  q2_f32x4 acc = q2_f32x4{0.f, 0.f, 0.f, 0.f};
  for (int gr = 0; gr < groups; ++gr) {
    float z = 8.f;
    if (m.zero == ZERO_CODES) z = (float)((m.zero_codes[n * ((groups + 1) / 2) + gr / 2] >> (4 * (gr & 1))) & 15);
    if (m.zero == ZERO_F16) z = f16_to_f32(a.z[n * groups + gr]);
    const float z16 = m.zero == ZERO_8 ? 0.f : z * 0.0625f;   // ZERO_8: off with the sum already
    for (int b = 0; b < blocks; ++b) {
      q2_f32x4 tmp = q2_f32x4{0.f, 0.f, 0.f, 0.f}, sum = tmp;
      uint64_t pz = ~0ull;
      for (int t = 0; t < steps; ++t) {
        const int64_t k0 = gr * m.group + BLOCK_K * b + 32 * t;
        const uint32_t w[1] = {*reinterpret_cast<const uint32_t*>(wp + k0 / 2)};
        const q2_u32x4 av = *reinterpret_cast<const q2_u32x4*>(xp + k0);
        pz &= q4_part_zero(w, z);
        tmp = mfma(av, q4_frag(w[0], kc), tmp);
        sum = mfma(av, sones, sum);
      }
      const float d = f16_to_f32((uint16_t)zero_where(sp[gr], column_all(pz)));
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(d, __builtin_fmaf(-z16, sum[e], tmp[e] - sum[e]), acc[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) out[4 * g + e][cb] = acc[e] * 16.f;
  __syncthreads();
  for (int idx = threadIdx.x; idx < MV_BM * out_cols; idx += 256) {
    const int r = idx / out_cols, col = idx - r * out_cols;
    const int64_t mm = rt.m0 + r, nn = n0 + col;
    if (mm >= rt.mend || nn >= n_out) continue;
    store_out(a, a.bias, n_out, mm, nn, out[r][col], a.gated ? out[r][MV_BN / 2 + col] : 0.f);
  }
}

hipError_t launch_q4_matvec(const MatvecArgs& m, hipStream_t stream) {
  // less than a unit of inputs, more rows than the grid's second dimension, columns beyond 32 bits
  if (m.f.K < 256 || m.f.N > 0x7fffffff || m.f.M > 65535 * MV_ROWS) {
    const int64_t cols = m.f.gated ? MV_BN / 2 : MV_BN;
    const int64_t tiles_n = (fused_n_out(m.f) + cols - 1) / cols, tiles_m = max_row_tiles(m.f, MV_BM);
    if (tiles_n > 0x7fffffff || tiles_m > 0x7fffffff / tiles_n) return hipErrorInvalidValue;
    hipLaunchKernelGGL(matvec_tile_kernel, grid_of(tiles_m * tiles_n), dim3(256), 0, stream, m, (int)tiles_n);
    return hipGetLastError();
  }
  if (m.group == 32) return launch_matvec<GROUP_32>(m, stream);
  if (m.group == 64) return launch_matvec<GROUP_64>(m, stream);
  return launch_matvec<GROUP_128>(m, stream);
}

}  // namespace q2dev
