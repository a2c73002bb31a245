// q2_fused_few.hip - the fused and grouped linears for up to 16 rows per tile:
// single tokens, decode batches, experts with a few rows each.
//
// What counts here is the read of the packed weights and the latency of one
// pass: every wave has all loads of its blocks in flight before it computes on
// any of them, in pieces of at least 64 bytes of a weight row.  One row, K = 2560,
// N = 2 x 9728: 10 us Q2_0 (13 MB, 1.3 TB/s), 11.9 us 4-bit (26 MB, 2.2 TB/s) with the
// weights from memory; 16 rows, K = 4096, N = 4096: 10.2 us.
#include "q2_fused.h"
#include <algorithm>

namespace q2dev {

// The half-words b, b + 1, ... of a row of n (four of them from element
// min(b, n - 4) on): one 8-byte load, or, for rows of less than four (SHORT),
// single ones.  A run-time branch between the two would make every later load
// wait for this one.
template <bool SHORT>
__device__ __forceinline__ uint64_t load4h(const uint16_t* p, int b, int n) {
  uint64_t v;
  if constexpr (SHORT) {
    v = p[0] | (uint32_t)p[min(1, n - 1)] << 16 | (uint64_t)p[min(2, n - 1)] << 32;
  } else {
    __builtin_memcpy(&v, p + min(b, n - 4), 8);
  }
  return v;
}

constexpr int FEW_COLS = 32;                             // weight columns of a workgroup, two 16-column tiles
constexpr int FEW_WAVES = 16;                            // at most
constexpr int FEW_BLOCKS = 2;                            // of a wave in a pass

// LDS bytes of one row of x over `blocks` blocks, copied 1 KB at a time: 16 bytes
// of padding put the 16 rows that a fragment read touches into different banks.
__host__ __device__ constexpr int few_row_bytes(int blocks) { return (blocks + 3) / 4 * 1024 + 16; }

// A workgroup of kg waves owns up to 16 rows x 32 weight columns (with a gated
// epilogue the second tile holds the other factors of the first one's
// outputs).  In each pass wave w takes two consecutive 128-wide blocks.  In the
// matrix-core layout lane (c, g) = (lane % 16, lane / 16) holds inputs 32 g ..
// 32 g + 31 of weight column c and of row c.  A 4-bit block's 64 bytes per
// column are loaded that way; of 2-bit codes a lane loads 16 of the 64 bytes
// that two blocks have per column, and two lane-row swaps bring both blocks
// into the layout (8 bytes per lane and block would touch 32-byte pieces).  The
// rows of x are staged in LDS, only those that exist.
template <int FMT, bool SHORT, bool BRANCH>
__global__ __launch_bounds__(64 * FEW_WAVES) void fused_few_kernel(FusedArgs a, int bm, int tiles_n) {
  constexpr int DW = (FMT == 0) ? 2 : 4, D = FEW_BLOCKS;
  extern __shared__ __align__(16) uint8_t xs[];
  const int lane = threadIdx.x & 63, kg = blockDim.x >> 6;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  RowTile rt;
  int tn;
  if (!find_tile(a, bm, tiles_n, 1, rt, tn)) return;
  const int64_t n_out = fused_n_out(a), K = a.K;
  const int out_cols = a.gated ? FEW_COLS / 2 : FEW_COLS;
  const int64_t n0 = (int64_t)tn * out_cols;
  const int KB = (int)(K / BLOCK_K);
  const int rows = (int)std::min<int64_t>(rt.mend - rt.m0, bm);
  const int64_t row_bytes = (FMT == 0) ? K / 4 : K / 2;
  const NatConsts kc = (FMT == 0) ? q2_nat_consts() : q4_nat_consts();

  const uint8_t* wp[2];
  const uint16_t *sp[2], *zp[2];
  int64_t wrow[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    int64_t n = n0 + c + (a.gated ? 0 : 16 * j);
    n = n < n_out ? n : n_out - 1;
    if (a.gated && j) n += n_out;
    wrow[j] = n;
    const int64_t row = rt.expert * a.N + n;
    wp[j] = a.w + row * row_bytes;
    sp[j] = a.s + row * KB;
    zp[j] = (FMT == 1) ? a.z + row * KB : nullptr;
  }

  // Lane i: the row of x that tile row i reads, -1 for an index outside x.
  int xsrc = -1;
  if (lane < rows) {
    const int64_t src = a.row_index ? (int64_t)a.row_index[rt.m0 + lane] : rt.m0 + lane;
    xsrc = src >= 0 && src < a.x_rows ? (int)src : -1;
  }

  const int span = kg * D;                               // blocks of a pass
  const int rstride = few_row_bytes(span);
  const uint8_t* const xrow = xs + min(c, rows - 1) * rstride + 64 * g;   // rows past the last one repeat it
  const uint32_t sone = (FMT == 0) ? 0x3FA03FA0u : 0x3F803F80u;           // bf16 1.25 / 1 pairs
  const q2_u32x4 sones = q2_u32x4{sone, sone, sone, sone};
  q2_f32x4 acc[2] = {q2_f32x4{0.f, 0.f, 0.f, 0.f}, q2_f32x4{0.f, 0.f, 0.f, 0.f}};

  for (int p0 = 0; p0 < KB; p0 += span) {
    const int bb = p0 + wv * D;                          // this wave's first block
    uint32_t w[2][D][DW];
    uint64_t s[2], z[2];
    if (bb < KB) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if constexpr (FMT == 0) {
#pragma unroll
          for (int p = 0; p < D / 2; ++p) {
            const int b = min(bb + 2 * p + (g >> 1), KB - 1);             // past the end: a valid block, dropped below
            const q2_u32x4 v = *reinterpret_cast<const q2_u32x4*>(wp[j] + (int64_t)b * 32 + 16 * (g & 1));
            w[j][2 * p][0] = v[0]; w[j][2 * p][1] = v[1];
            w[j][2 * p + 1][0] = v[2]; w[j][2 * p + 1][1] = v[3];
          }
        } else {
#pragma unroll
          for (int d = 0; d < D; ++d) {
            const int b = min(bb + d, KB - 1);
            const q2_u32x4 v = *reinterpret_cast<const q2_u32x4*>(wp[j] + (int64_t)b * 64 + 16 * g);
#pragma unroll
            for (int q = 0; q < 4; ++q) w[j][d][q] = v[q];
          }
        }
        s[j] = load4h<SHORT>(sp[j], bb, KB);
        z[j] = (FMT == 1) ? load4h<SHORT>(zp[j], bb, KB) : 0;
      }
    }
    if (p0 > 0) __syncthreads();                         // the last pass's rows are read
    const int nb = min(span, KB - p0), pieces = (nb + 3) / 4;
    for (int i = wv; i < rows * pieces; i += kg) {
      const int row = i / pieces, q = i - row * pieces;
      const int src = __builtin_amdgcn_readlane(xsrc, row);
      uint8_t* const dst = xs + row * rstride + q * 1024;
      if (src >= 0) {                                    // past the pass: its last chunk again
        const uint16_t* p = a.x + (int64_t)src * K + (int64_t)p0 * BLOCK_K + 8 * min(64 * q + lane, 16 * nb - 1);
        __builtin_amdgcn_global_load_lds(p, (lds_void*)dst, 16, 0, 0);
      } else {
        *reinterpret_cast<q2_u32x4*>(dst + 16 * lane) = q2_u32x4{0u, 0u, 0u, 0u};
      }
    }
    if (BRANCH && p0 == 0) {
      // The rank-r branch while the weights are on their way: T_hi B_hi + T_hi B_lo +
      // T_lo B_hi in bf16, 32 of r per wave, in the block sums' units (a fourth).  In
      // a kernel of its own: its 16 registers cost linears without one up to 17 %.
      const int r8 = (a.r + 7) & ~7;
      for (int k0 = 32 * wv; k0 < r8; k0 += 32 * kg) {
        const int64_t m = rt.m0 + min(c, rows - 1);
        const q2_u32x4 hi = branch_afrag(a, m, k0 + 8 * g, false), lo = branch_afrag(a, m, k0 + 8 * g, true);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const BranchB bq = branch_bfrag(a, wrow[j], k0 + 8 * g);
          q2_f32x4 br = mfma(hi, bq.hi, q2_f32x4{0.f, 0.f, 0.f, 0.f});
          br = mfma(hi, bq.lo, br);
          br = mfma(lo, bq.hi, br);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[j][e] = __builtin_fmaf(0.25f, br[e], acc[j][e]);
        }
      }
    }
    stage_barrier<0>();                                  // all copies have landed
    if (bb < KB) {
      const int sh = 16 * (SHORT ? bb : bb - min(bb, KB - 4));
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        s[j] >>= sh;
        z[j] >>= sh;
      }
      if constexpr (FMT == 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int p = 0; p < D / 2; ++p)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              auto r = __builtin_amdgcn_permlane16_swap(w[j][2 * p][q], w[j][2 * p + 1][q], false, false);
              r = __builtin_amdgcn_permlane32_swap(r[0], r[1], false, false);
              w[j][2 * p][q] = r[0];
              w[j][2 * p + 1][q] = r[1];
            }
      }
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (bb + d < KB) {
          q2_u32x4 av[4];
          q2_f32x4 sum = q2_f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            av[t] = *reinterpret_cast<const q2_u32x4*>(xrow + (wv * D + d) * 256 + 16 * t);
            sum = mfma(av[t], sones, sum);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            q2_u32x4 bf[4];
            if constexpr (FMT == 0) {
              bf[0] = q2_frag<0>(w[j][d][0], kc);
              bf[1] = q2_frag<1>(w[j][d][0], kc);
              bf[2] = q2_frag<0>(w[j][d][1], kc);
              bf[3] = q2_frag<1>(w[j][d][1], kc);
            } else {
#pragma unroll
              for (int t = 0; t < 4; ++t) bf[t] = q4_frag(w[j][d][t], kc);
            }
            q2_f32x4 tmp = q2_f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int t = 0; t < 4; ++t) tmp = mfma(av[t], bf[t], tmp);
            const uint32_t sb = (uint32_t)(s[j] >> (16 * d)) & 0xFFFFu;
            if constexpr (FMT == 0) {
              // A column of codes 1 is the row sums' operand, 1.25 everywhere, in the
              // same instructions: the same bits, so zero weights add exactly nothing.
              const float dc = f16_to_f32((uint16_t)sb);
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[j][e] = __builtin_fmaf(dc, tmp[e] - sum[e], acc[j][e]);
            } else {
              const float zc = f16_to_f32((uint16_t)(z[j] >> (16 * d)));
              const float dc = f16_to_f32((uint16_t)zero_where(sb, column_all(q4_part_zero(w[j][d], zc))));
              const float k4 = 1.f + zc * 0.0625f;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                acc[j][e] = __builtin_fmaf(dc, __builtin_fmaf(-k4, sum[e], tmp[e]), acc[j][e]);
            }
          }
        }
      }
    }
  }
  __syncthreads();                                       // the rows' space takes the partial sums
  float (*const red)[16][FEW_COLS + 1] = reinterpret_cast<float (*)[16][FEW_COLS + 1]>(xs);
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[wv][4 * g + e][16 * j + c] = acc[j][e];
  __syncthreads();

  const float* bias = a.bias ? a.bias + rt.expert * a.N : nullptr;
  const float fin = (FMT == 0) ? 4.f : 16.f;
  for (int idx = threadIdx.x; idx < rows * out_cols; idx += blockDim.x) {
    const int row = idx / out_cols, col = idx - row * out_cols;
    const int64_t m = rt.m0 + row, n = n0 + col;
    if (n >= n_out) continue;
    float v = 0.f, u = 0.f;
    for (int q = 0; q < kg; ++q) v += red[q][row][col];  // wave order
    if (a.gated)
      for (int q = 0; q < kg; ++q) u += red[q][row][FEW_COLS / 2 + col];
    v *= fin;
    u *= fin;
    store_out(a, bias, n_out, m, n, v, u);
  }
}

// Waves of a workgroup, two blocks each per pass: four once that gives the chip
// a thousand waves, eight, sixteen for fewer workgroups.  Short passes keep few
// rows of x in LDS and few registers, so more workgroups share a CU.  Measured
// against four blocks per wave and all of K in one pass where the waves reach, us:
// 23 tokens to 4 of 32 experts, K = 2560, N = 1408 16.0 / 20.7 (4-bit 20.0 /
// 22.3); 16 rows, K = 4096, N = 12288 13.3 / 16.6; one row, K = 2560, 2 x 9728
// 10.0 / 9.8 (4-bit 11.9 / 13.1); K = 4096, N = 4096 (128 workgroups, eight waves)
// 6.2 / 6.4; K = 9728, N = 2560 (80, sixteen) 10.1 / 10.0.
template <int FMT, bool SHORT, bool BRANCH>
static hipError_t run_few(const FusedArgs& a, int bm, int64_t slots, int64_t tiles_n, hipStream_t stream) {
  const int KB = (int)(a.K / BLOCK_K);
  const int rows = (int)std::min<int64_t>(a.M, bm);      // at most 64 KB of them in LDS
  const int64_t wgs = slots * tiles_n;
  int kg = wgs >= 256 ? 4 : wgs >= 128 ? 8 : FEW_WAVES;
  kg = std::clamp((KB + FEW_BLOCKS - 1) / FEW_BLOCKS, 1, kg);
  while (kg > 1 && rows * few_row_bytes(kg * FEW_BLOCKS) > 64 * 1024) --kg;
  const size_t lds = std::max<size_t>((size_t)rows * few_row_bytes(kg * FEW_BLOCKS),
                                      (size_t)kg * 16 * (FEW_COLS + 1) * 4);
  hipLaunchKernelGGL((fused_few_kernel<FMT, SHORT, BRANCH>), grid_of(wgs), dim3(64 * kg), lds, stream, a, bm,
                     (int)tiles_n);
  return hipGetLastError();
}

template <int FMT>
static hipError_t pick_few(const FusedArgs& a, int bm, int64_t slots, int64_t tiles_n, hipStream_t stream) {
  const bool is_short = a.K < 4 * BLOCK_K;
  if constexpr (FMT == 0)
    if (a.r > 0)
      return is_short ? run_few<FMT, true, true>(a, bm, slots, tiles_n, stream)
                      : run_few<FMT, false, true>(a, bm, slots, tiles_n, stream);
  return is_short ? run_few<FMT, true, false>(a, bm, slots, tiles_n, stream)
                  : run_few<FMT, false, false>(a, bm, slots, tiles_n, stream);
}

static int64_t few_columns(const FusedArgs& a) {         // output columns of a workgroup
  return a.gated ? FEW_COLS / 2 : FEW_COLS;
}
int64_t few_tiles(const FusedArgs& a) {
  return ((a.M + 15) / 16) * ((fused_n_out(a) + few_columns(a) - 1) / few_columns(a));
}

hipError_t launch_fused_few(const FusedArgs& a, int fmt, hipStream_t stream) {
  // Rows per tile: groups of a few rows take eight (half the LDS, fewer idle tiles
  // in the launch; 92 rows over 32 experts, K = 2560, N = 1408 4-bit: 20.0 us, 22.1
  // with sixteen); a group with more reads its weights again, from the caches.
  const int bm = a.offsets != nullptr ? 8 : 16;
  const int64_t cols = few_columns(a);
  const int64_t tiles_n = (fused_n_out(a) + cols - 1) / cols, slots = max_row_tiles(a, bm);
  if (tiles_n > 0x7fffffff || slots > 0x7fffffff / tiles_n) return hipErrorInvalidValue;
  return fmt == 0 ? pick_few<0>(a, bm, slots, tiles_n, stream) : pick_few<1>(a, bm, slots, tiles_n, stream);
}

}  // namespace q2dev
