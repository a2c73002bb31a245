// q2_fused.hip - the Q2_0 and 4-bit linears with an epilogue (bias, activation,
// gate, residual) and over rows grouped by expert.
//
// y = epilogue(x W^T): products of bf16 activations and weights decoded to bf16
// by a magic-number OR (q2_device.h) on the matrix cores, one fp32 FMA per
// output and 128-weight block for the block's f16 scale, the epilogue on the
// finished fp32 sums, one rounding to the output type.
#include "q2_fused.h"
#include "q2_internal.h"
#include <algorithm>
#include <cmath>

namespace q2dev {

constexpr int F_BM = 32, F_BN = 64;

// Weight row of tile column cb: with a gated epilogue the tile's first half
// holds columns of the first N / 2 weight rows and the second half the same
// columns of the others, so both factors of an output meet in one tile.
__device__ __forceinline__ int64_t tile_wrow(const FusedArgs& a, int64_t n_out, int64_t n0, int cb, int bn) {
  int64_t n;
  if (a.gated) {
    const int half = bn / 2;
    const bool up = cb >= half;
    n = n0 + (up ? cb - half : cb);
    n = n < n_out ? n : n_out - 1;
    return up ? n + n_out : n;
  }
  n = n0 + cb;
  return n < n_out ? n : n_out - 1;
}

// A workgroup owns 32 rows x 64 weight columns; each of its four waves 16 of
// the columns, straight from global memory.  Bound by the latency of those loads:
// M = 1024, K = 384, N = 4096 33 us, 99 TFLOP/s (the kernel of q2_fused_mid.hip
// needs 14 at K = 512); it takes what the others' addressing does not reach.
template <int FMT>
__global__ __launch_bounds__(256) void fused_tile_kernel(FusedArgs a, int tiles_n) {
  constexpr int DW = (FMT == 0) ? 2 : 4;
  __shared__ float out[F_BM][F_BN + 4];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int c = lane & 15, g = lane >> 4;
  RowTile rt;
  int tn;
  if (!find_tile(a, F_BM, tiles_n, 1, rt, tn)) return;
  const int64_t n_out = fused_n_out(a);
  const int out_cols = a.gated ? F_BN / 2 : F_BN;
  const int64_t n0 = (int64_t)tn * out_cols;
  const int64_t KB = a.K / BLOCK_K, row_bytes = (FMT == 0) ? a.K / 4 : a.K / 2;
  const NatConsts kc = (FMT == 0) ? q2_nat_consts() : q4_nat_consts();

  const int64_t wn = tile_wrow(a, n_out, n0, 16 * wv + c, F_BN);
  const int64_t wrow = rt.expert * a.N + wn;
  const uint8_t* wp = a.w + wrow * row_bytes + g * (4 * DW);
  const uint16_t* sp = a.s + wrow * KB;
  const uint16_t* zp = (FMT == 1) ? a.z + wrow * KB : nullptr;
  const uint16_t* xp[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t m = rt.m0 + 16 * i + c;
    int64_t src = m < rt.mend ? m : -1;
    if (src >= 0 && a.row_index) src = a.row_index[m];
    xp[i] = (src >= 0 && src < a.x_rows) ? a.x + src * a.K + 32 * g : nullptr;
  }

  const uint32_t sone = (FMT == 0) ? 0xBFA0BFA0u : 0xBF80BF80u;   // bf16 -1.25 / -1 pairs
  const q2_u32x4 sones = q2_u32x4{sone, sone, sone, sone};
  q2_f32x4 acc[2] = {q2_f32x4{0.f, 0.f, 0.f, 0.f}, q2_f32x4{0.f, 0.f, 0.f, 0.f}};
  for (int64_t b = 0; b < KB; ++b) {
    uint32_t w[DW];
#pragma unroll
    for (int d = 0; d < DW; ++d) w[d] = reinterpret_cast<const uint32_t*>(wp + b * (16 * DW))[d];
    q2_u32x4 bf[4];
    float zc = 0.f;
    uint64_t pz;
    if constexpr (FMT == 0) {
      bf[0] = q2_frag<0>(w[0], kc);
      bf[1] = q2_frag<1>(w[0], kc);
      bf[2] = q2_frag<0>(w[1], kc);
      bf[3] = q2_frag<1>(w[1], kc);
      pz = q2_part_zero(w);
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t) bf[t] = q4_frag(w[t], kc);
      zc = f16_to_f32(zp[b]);
      pz = q4_part_zero(w, zc);
    }
    const float dc = f16_to_f32((uint16_t)zero_where(sp[b], column_all(pz)));
    const float k4 = 1.f + zc * 0.0625f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      q2_u32x4 av[4];
      q2_f32x4 sum = q2_f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        av[t] = q2_u32x4{0u, 0u, 0u, 0u};
        if (xp[i]) av[t] = *reinterpret_cast<const q2_u32x4*>(xp[i] + b * BLOCK_K + 8 * t);
        sum = mfma(av[t], sones, sum);
      }
      if constexpr (FMT == 1) sum = q2_f32x4{k4 * sum[0], k4 * sum[1], k4 * sum[2], k4 * sum[3]};
#pragma unroll
      for (int t = 0; t < 4; ++t) sum = mfma(av[t], bf[t], sum);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = __builtin_fmaf(dc, sum[e], acc[i][e]);
    }
  }
  const float fin = (FMT == 0) ? 4.f : 16.f;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) out[16 * i + 4 * g + e][16 * wv + c] = acc[i][e] * fin;
  __syncthreads();
  const float* bias = a.bias ? a.bias + rt.expert * a.N : nullptr;
  const int r8 = (a.r + 7) & ~7;
  for (int idx = threadIdx.x; idx < F_BM * out_cols; idx += 256) {
    const int row = idx / out_cols, col = idx - row * out_cols;
    const int64_t m = rt.m0 + row, n = n0 + col;
    if (m >= rt.mend || n >= n_out) continue;
    float v = out[row][col], u = a.gated ? out[row][F_BN / 2 + col] : 0.f;
    for (int j = 0; j < a.r; ++j) {                      // the rank-r branch, from the limbs of x A^T
      const float t = bf16_to_f32(a.lr_t[m * 2 * r8 + j]) + bf16_to_f32(a.lr_t[m * 2 * r8 + r8 + j]);
      v = __builtin_fmaf(t, f16_to_f32(a.lr_b[n * a.r + j]), v);
      if (a.gated) u = __builtin_fmaf(t, f16_to_f32(a.lr_b[(n + n_out) * a.r + j]), u);
    }
    store_out(a, bias, n_out, m, n, v, u);
  }
}

// The f16 kernel for Q2_0 weights, from the sizes alone (the workspace goes by
// them too).  Its 128 x 256 tiles must cover half of the chip's 256 CUs, the
// columns must be enough to pay for converting x, and groups must fill their
// tiles.  Measured, this kernel / the one of q2_fused_mid.hip, in us: K = 4096,
// N = 12288: M = 320 (120 tiles) 54 / 48, M = 384 (144) 55 / 65, M = 1024 (384)
// 111 / 132; M = 1536, N = 4096 64 / 71; M = 4096, N = 2048 80 / 91; M = 4096,
// K = 12288, N = 1536 192 / 190; M = 8192, K = 2048, N = 1024 53 / 50.  32 groups,
// K = 2048, N = 2 x 1408: 2048 rows (half of the tiles' rows) 62 / 56, 4096 rows
// (two thirds) 89 / 91, 6400 rows 98 / 123; K = 1408, N = 2048: 4096 rows 55 / 49,
// 8192 rows 80 / 83.
static bool use_f16(int64_t M, int64_t N, int64_t K, int64_t E, int fmt) {
  if (fmt != 0 || !fused_f16_takes(M, N, K)) return false;
  // groups add half a tile each
  const double tiles = (M / 128.0 + (E > 0 ? 0.5 * std::min(E, M) : 0.0)) * std::ceil(N / 256.0);
  const double fill = E > 0 ? (double)M / ((double)M + 64.0 * (double)E) : 1.0;          // rows that are not padding
  return tiles >= 140.0 && fill >= 0.7 && N >= 1536;
}

size_t fused_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t E, int fmt) {
  return use_f16(M, N, K, E, fmt) ? f16_workspace_bytes(M, K) : 0;
}

hipError_t launch_fused(const FusedArgs& a, int fmt, void* ws, hipStream_t stream) {
  const int64_t groups = a.offsets ? a.E : 0;
  const bool f16 = use_f16(a.M, a.N, a.K, groups, fmt) && a.x_rows > 0 && a.x_rows <= a.M;
  if (a.r > 0 && !(f16 && a.r <= 64)) {                  // else converted and multiplied in one pass over x
    const hipError_t e = launch_lowrank_t(a.x, a.lr_a, a.lr_t, a.M, a.K, a.r, stream);
    if (e != hipSuccess) return e;
  }
  if (f16) return launch_fused_f16(a, ws, stream);
  // Few rows, or few tiles of them: up to 256 workgroups without groups, up to four
  // rows per group.  There / in the next one, us: 16 rows, K = 4096, N = 12288 13.1 /
  // 13.6; N = 4096 (256 workgroups) 32 rows 11.2 / 12.7, 4-bit 13.0 / 15.1; N = 6144
  // (384) 13.5 / 12.9; 128 rows, K = 2560, N = 1024 8.4 / 11.6; over 32 experts,
  // K = 2048, 2 x 1408, 128 rows 24.3 / 25.9, 256 rows 32.1 / 25.8.
  if (a.M <= 16 || (a.offsets ? a.M <= 4 * a.E : few_tiles(a) <= 256)) return launch_fused_few(a, fmt, stream);
  if (fused_mid_takes(a, fmt)) return launch_fused_mid(a, fmt, stream);
  // Short K (less than four blocks) or a weight beyond 4 GB: the plain kernel.
  const int64_t cols = a.gated ? F_BN / 2 : F_BN;
  const int64_t tiles_n = (fused_n_out(a) + cols - 1) / cols, slots = max_row_tiles(a, F_BM);
  if (tiles_n > 0x7fffffff || slots > 0x7fffffff / tiles_n) return hipErrorInvalidValue;
  const dim3 grid = grid_of(slots * tiles_n);
  if (fmt == 0) hipLaunchKernelGGL((fused_tile_kernel<0>), grid, dim3(256), 0, stream, a, (int)tiles_n);
  else hipLaunchKernelGGL((fused_tile_kernel<1>), grid, dim3(256), 0, stream, a, (int)tiles_n);
  return hipGetLastError();
}

}  // namespace q2dev
