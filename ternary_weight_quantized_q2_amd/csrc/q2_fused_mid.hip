// q2_fused_mid.hip - the fused and grouped linears between few tiles and the f16
// kernel's many rows, and of the 4-bit format, whose weights (q - z) s have no exact
// f16 value, everything beyond few tiles.
//
// Weights decode to bf16 1 + c / 4 or 1 + q / 16 (q2_device.h); per 128-wide
// block the row sums of x take the 1 back and one FMA per output applies the
// block's scale.
#include "q2_fused.h"
#include "q2_internal.h"
#include <algorithm>

namespace q2dev {

// Position of chunk q of row r: q ^ mid_swz(r).  The 16-byte fragment reads of a
// pass then touch 16 different bank groups (a bit rotation of r mod 16).
__device__ __forceinline__ int mid_swz(int r) { return ((r >> 2) & 3) | ((r & 3) << 2); }

// A workgroup of KG groups of NW waves owns 16 MT rows x 64 NW weight columns;
// wave (kg, wn) computes the 64 columns wn from every KG-th unit of blocks (a
// unit is what one 16-byte load of a lane holds: two 2-bit blocks, one 4-bit
// block), so a block is decoded once per workgroup.  Rows go to LDS by direct
// copies, a set of KG blocks per stage, two stages; one barrier per stage waits
// for them.  Codes of the next unit are loaded to registers of their own while
// this one is computed (ROLL = false), or, in tiles of 64 rows, which have no
// room for them, column tile by column tile as this one's are decoded: 64 x 160
// tiles then fit 256 registers but for three of Q2_0 and one of 4-bit, spilled outside
// the loop, and 64 x 128 ones gained 3 %, 32-row ones lost 4 %.
// x and the codes are addressed with a scalar block offset (buffer loads): 8 % less
// time for 20 rows per expert than 64-bit addresses.  Each wave sums its rows on the
// matrix cores itself (a quarter of its products; sharing the sums would need a second
// barrier).
template <int FMT, int MT, int NT, int NW, int KG, int OCC>
__global__ __launch_bounds__(64 * NW * KG, OCC) void fused_mid_kernel(FusedArgs a, int tiles_n, int group_m) {
  constexpr int W = NW * KG, BM = 16 * MT, BN = 16 * NT * NW;
  constexpr int U = (FMT == 0) ? 2 : 1;                  // blocks per unit
  constexpr bool ROLL = MT > 2;
  constexpr int STAGE = KG * BM * 256;
  constexpr int STRIDE = BN + 4;                         // floats per row of the output tile
  constexpr int RG = BM / 4;                             // copies of four rows per block
  constexpr int RPW = RG / NW;                           // of a wave: its group's block, a share of the rows
  constexpr int CHUNK = 16;                              // blocks of scales in LDS at a time
  constexpr int OFF_S = 2 * STAGE;
  constexpr int PIECES = (BN * (CHUNK / 4) + 64 * W - 1) / (64 * W);      // 8-byte loads per thread and chunk
  constexpr int SMEM = OFF_S + 2 * CHUNK * BN * 4;
  static_assert(BM * STRIDE * 4 <= OFF_S && (KG / 2) * NW * MT * NT * 1024 <= OFF_S, "output tile and partial sums");
  static_assert(RG % NW == 0 && BM % W == 0, "rows divide over the waves");
  __shared__ __align__(16) uint8_t smem[SMEM];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wv % NW, kg = wv / NW;
  const int c = lane & 15, g = lane >> 4;
  RowTile rt;
  int tn;
  if (!find_tile(a, BM, tiles_n, group_m, rt, tn)) return;
  const int64_t n_out = fused_n_out(a), K = a.K, m0 = rt.m0;
  const int rows = (int)std::min<int64_t>(rt.mend - m0, BM);
  const int KB = a.x_rows > 0 ? (int)(K / BLOCK_K) : 0;  // no row to read: every product is an empty sum
  const int64_t row_bytes = (FMT == 0) ? K / 4 : K / 2;
  const NatConsts kc = (FMT == 0) ? q2_nat_consts() : q4_nat_consts();
  const int64_t n0 = (int64_t)tn * (a.gated ? BN / 2 : BN);
  // Weight row of tile column `col`: with a gated epilogue the tile's second
  // half holds the other factors of the first half's outputs.
  auto wrow = [&](int col) -> int64_t {
    const bool up = a.gated && col >= BN / 2;
    int64_t n = n0 + (up ? col - BN / 2 : col);
    n = n < n_out ? n : n_out - 1;
    return up ? n + n_out : n;
  };
  // Offsets from the expert's weight fit 32 bits (checked by the launcher).
  const uint8_t* const wbase = a.w + rt.expert * a.N * row_bytes;
  const uint16_t* const sbase = a.s + rt.expert * a.N * (K / BLOCK_K);
  const uint16_t* const zbase = (FMT == 1) ? a.z + rt.expert * a.N * (K / BLOCK_K) : nullptr;
  uint32_t woff[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) woff[j] = (uint32_t)(wrow(16 * (NT * wn + j) + c) * row_bytes) + 16u * g;
  // Scales (low half) and zero points (high half) of CHUNK blocks and the tile's
  // columns sit in LDS as [block][column], two chunks in turn: a half-word per
  // lane, column and block straight from global memory cost up to a sixth of the
  // kernel.  A thread loads 8 bytes, four blocks of one row, PIECES times; blocks
  // past the end load the last four again.
  uint32_t* const sz = reinterpret_cast<uint32_t*>(smem + OFF_S);
  uint64_t sreg[PIECES], zreg[PIECES];
  auto piece_start = [&](int chunk, int idx) { return min(CHUNK * chunk + 4 * (idx % (CHUNK / 4)), KB - 4); };
  auto load_scales = [&](int chunk) {
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
      const int idx = min(tid + p * 64 * W, BN * (CHUNK / 4) - 1);
      const uint32_t off = (uint32_t)(wrow(idx / (CHUNK / 4)) * KB + piece_start(chunk, idx));
      __builtin_memcpy(&sreg[p], sbase + off, 8);
      if constexpr (FMT == 1) __builtin_memcpy(&zreg[p], zbase + off, 8);
    }
  };
  auto store_scales = [&](int chunk) {
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
      const int idx = min(tid + p * 64 * W, BN * (CHUNK / 4) - 1);
      const int slot = piece_start(chunk, idx) - CHUNK * chunk;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t v = (uint32_t)(sreg[p] >> (16 * e)) & 0xFFFFu;
        const uint32_t u = FMT == 1 ? (uint32_t)(zreg[p] >> (16 * e)) << 16 : 0u;
        if (slot + e >= 0) sz[((chunk & 1) * CHUNK + slot + e) * BN + idx / (CHUNK / 4)] = v | u;
      }
    }
  };
  const uint32_t* const szl = sz + 16 * NT * wn + c;     // this lane's column of tile j at + 16 j

  // Copy r of this wave: rows 4 (RPW wn + r) .. + 3 of its group's block, lane l
  // row l / 16 of them and position l % 16.
  uint32_t xoff[RPW];
#pragma unroll
  for (int r = 0; r < RPW; ++r) {
    const int row = 4 * (RPW * wn + r) + (lane >> 4);
    const int64_t m = m0 + (row < rows ? row : rows - 1);
    int64_t src = a.row_index ? (int64_t)a.row_index[m] : m;
    if (src < 0 || src >= a.x_rows) src = 0;             // read row 0; the result is cleared at the end
    xoff[r] = (uint32_t)((a.row_index ? src : src - m0) * K * 2) + 16u * ((lane & 15) ^ mid_swz(row & 15));
  }
  const __amdgpu_buffer_rsrc_t rx = a.row_index ? buf_rsrc(a.x, (uint32_t)(a.x_rows * K * 2))
                                                : buf_rsrc(a.x + m0 * K, (uint32_t)(rows * K * 2));
  const __amdgpu_buffer_rsrc_t rw = buf_rsrc(wbase, (uint32_t)(a.N * row_bytes));
  const int units = (KB + U - 1) / U, NS = (units + KG - 1) / KG * U;     // stages
  auto block_of = [&](int s) { return (KG * (s / U) + kg) * U + s % U; };
  auto copy_stage = [&](int s) {
    const int blk = min(block_of(s), KB - 1);            // past the end: the last block again, never used
#pragma unroll
    for (int r = 0; r < RPW; ++r) {
      const uint32_t xo = xoff[r];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rx, (lds_void*)(smem + (s & 1) * STAGE + kg * BM * 256 + (RPW * wn + r) * 1024), 16, xo,
          (uint32_t)blk * 256u, 0, 0);
    }
  };
  q2_u32x4 w[NT], wnext[ROLL ? 1 : NT];                  // this lane's 16 bytes of a unit's codes
  auto load_codes = [&](int j, int n) {                  // past the last unit: that one again, never used
    const int u = KG * n + kg;
    const q2_u32x4 v = __builtin_bit_cast(
        q2_u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, woff[j] - unit_back(u, KB, U, g), unit_start(u, KB, U), 0));
    if constexpr (ROLL) w[j] = v;
    else wnext[j] = v;
  };

  q2_f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = q2_f32x4{0.f, 0.f, 0.f, 0.f};
  int aoff[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) aoff[t] = c * 256 + (((4 * g + t) ^ mid_swz(c)) << 4);
  const uint32_t sone = (FMT == 0) ? 0xBFA0BFA0u : 0x3F803F80u;   // bf16 -1.25 / 1 pairs
  const q2_u32x4 sones = q2_u32x4{sone, sone, sone, sone};

  auto compute = [&](const uint8_t* st, int half, int blk, int next) {
    const uint32_t* const sp = szl + (blk & (2 * CHUNK - 1)) * BN;
    q2_u32x4 av[MT][4];
    q2_f32x4 sum[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
#pragma unroll
      for (int t = 0; t < 4; ++t) av[i][t] = *reinterpret_cast<const q2_u32x4*>(st + i * 4096 + aoff[t]);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) sum[i] = q2_f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < MT; ++i) sum[i] = mfma(av[i][t], sones, sum[i]);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const uint32_t sv = sp[16 * j];                    // scale | zero point << 16
      q2_u32x4 bf[4];
      float zc = 0.f;
      uint64_t pz;
      if constexpr (FMT == 0) {
        const uint32_t w2[2] = {w[j][2 * half], w[j][2 * half + 1]};
        bf[0] = q2_frag<0>(w2[0], kc);
        bf[1] = q2_frag<1>(w2[0], kc);
        bf[2] = q2_frag<0>(w2[1], kc);
        bf[3] = q2_frag<1>(w2[1], kc);
        pz = q2_part_zero(w2);
      } else {
        const uint32_t w4[4] = {w[j][0], w[j][1], w[j][2], w[j][3]};
#pragma unroll
        for (int t = 0; t < 4; ++t) bf[t] = q4_frag(w4[t], kc);
        zc = f16_to_f32((uint16_t)(sv >> 16));
        pz = q4_part_zero(w4, zc);
      }
      if (ROLL && next >= 0) load_codes(j, next);
      const float dc = f16_to_f32((uint16_t)zero_where(sv & 0xFFFFu, column_all(pz)));
      const float k4 = -dc * (1.f + zc * 0.0625f);
      q2_f32x4 tmp[MT];
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < MT; ++i)
          tmp[i] = mfma(av[i][t], bf[t], t > 0 ? tmp[i] : FMT == 0 ? sum[i] : q2_f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[i][j][e] = __builtin_fmaf(dc, tmp[i][e], acc[i][j][e]);
          if constexpr (FMT == 1) acc[i][j][e] = __builtin_fmaf(k4, sum[i][e], acc[i][j][e]);
        }
    }
  };

  // A chunk's scales are loaded two stages before its first block and written
  // one stage before, so a stage's barrier lies between the writes and the reads.
  constexpr int PER = CHUNK / (KG * U) * U;              // stages per chunk
  static_assert(PER >= 2 && CHUNK % (KG * U) == 0, "scale chunks");
  auto stage_scales = [&](int s) {                       // after stage s's barrier
    const int in = s % PER, next = s / PER + 1;
    if (CHUNK * next < KB) {
      if (in == PER - 2) load_scales(next);
      if (in == PER - 1) store_scales(next);
    }
  };
  if (KB > 0) {
    load_scales(0);
    copy_stage(0);
#pragma unroll
    for (int j = 0; j < NT; ++j) load_codes(j, 0);
    store_scales(0);
  }
  for (int n = 0; n * U < NS; ++n) {
    const int b0 = (KG * n + kg) * U;
    stage_barrier<ROLL ? NT : 0>();                      // the unit's codes may still be in flight
    stage_scales(U * n);
    if constexpr (!ROLL)
#pragma unroll
      for (int j = 0; j < NT; ++j) w[j] = wnext[j];
    if constexpr (FMT == 0) {
      copy_stage(2 * n + 1);
      // two stages per unit; the swaps bring 64 bytes per column into the matrix layout of two blocks
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          auto r = __builtin_amdgcn_permlane16_swap(w[j][q], w[j][2 + q], false, false);
          r = __builtin_amdgcn_permlane32_swap(r[0], r[1], false, false);
          w[j][q] = r[0];
          w[j][2 + q] = r[1];
        }
      if (b0 < KB) compute(smem + kg * BM * 256, 0, b0, -1);
      stage_barrier<0>();
      stage_scales(2 * n + 1);
      if (2 * n + 2 < NS) {
        copy_stage(2 * n + 2);
        if constexpr (!ROLL)
#pragma unroll
          for (int j = 0; j < NT; ++j) load_codes(j, n + 1);
      }
      if (b0 + 1 < KB) compute(smem + STAGE + kg * BM * 256, 1, b0 + 1, n + 1);
    } else {
      if (n + 1 < NS) {
        copy_stage(n + 1);
        if constexpr (!ROLL)
#pragma unroll
          for (int j = 0; j < NT; ++j) load_codes(j, n + 1);
      }
      if (b0 < KB) compute(smem + (n & 1) * STAGE + kg * BM * 256, 0, b0, n + 1);
    }
  }
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();

  // Partial sums of the groups, halving: the upper half's tiles go through LDS
  // and are added by the lower half, in a fixed order.
  float* const part = reinterpret_cast<float*>(smem);
  constexpr int PART = MT * NT * 4 * 64;
#pragma unroll
  for (int half = KG / 2; half >= 1; half /= 2) {
    if (kg >= half && kg < 2 * half) {
      float* p = part + ((kg - half) * NW + wn) * PART + lane;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) p[((i * NT + j) * 4 + e) * 64] = acc[i][j][e];
    }
    __syncthreads();
    if (kg < half) {
      const float* p = part + (kg * NW + wn) * PART + lane;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] += p[((i * NT + j) * 4 + e) * 64];
    }
    __syncthreads();
  }
  float* const out = part;
  if (kg == 0) {
    const float fin = (FMT == 0) ? 4.f : 16.f;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] *= fin;
    if (FMT == 0 && a.r > 0) {
      // (x A^T) B^T as T_hi B_hi + T_hi B_lo + T_lo B_hi in bf16
      const int r8 = (a.r + 7) & ~7;
      for (int k0 = 0; k0 < r8; k0 += 32) {
        const int q0 = k0 + 8 * g;
        q2_u32x4 aq[MT][2];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int l = 0; l < 2; ++l) aq[i][l] = branch_afrag(a, m0 + 16 * i + c, q0, l != 0);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const BranchB bq = branch_bfrag(a, wrow(16 * (NT * wn + j) + c), q0);
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            acc[i][j] = mfma(aq[i][0], bq.hi, acc[i][j]);
            acc[i][j] = mfma(aq[i][0], bq.lo, acc[i][j]);
            acc[i][j] = mfma(aq[i][1], bq.hi, acc[i][j]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) out[(16 * i + 4 * g + e) * STRIDE + 16 * (NT * wn + j) + c] = acc[i][j][e];
  }
  __syncthreads();
  // Each wave stores a share of the rows.
  constexpr int SR = BM / W;
  if (a.row_index) {
    for (int row = wv * SR; row < min((wv + 1) * SR, rows); ++row) {
      const int64_t src = a.row_index[m0 + row];
      if (src < 0 || src >= a.x_rows)                    // a row of zeros of x
        for (int col = lane; col < BN; col += 64) out[row * STRIDE + col] = 0.f;
    }
    __builtin_amdgcn_wave_barrier();
  }
  const float* bias = a.bias ? a.bias + rt.expert * a.N : nullptr;
  store_strip(a, bias, n_out, out + wv * SR * STRIDE, STRIDE, BN / 2, a.gated ? BN / 2 : BN, m0 + wv * SR,
              min(rows - wv * SR, SR), n0, lane);
}

template <int FMT, int MT, int NT, int NW, int KG, int OCC>
static hipError_t run_mid(const FusedArgs& a, hipStream_t stream) {
  constexpr int BM = 16 * MT, BN = 16 * NT * NW;
  const int64_t cols = a.gated ? BN / 2 : BN;
  const int64_t tiles_n = (fused_n_out(a) + cols - 1) / cols, slots = max_row_tiles(a, BM);
  if (tiles_n > 0x7fffffff || slots > 0x7fffffff / tiles_n) return hipErrorInvalidValue;
  const int group_m = tile_group_rows(slots, tiles_n, 2.0 * BM * (double)a.K,
                                      (double)BN * a.K * (FMT == 0 ? 0.265625 : 0.53125), KG > 2 ? 32 : 64);
  hipLaunchKernelGGL((fused_mid_kernel<FMT, MT, NT, NW, KG, OCC>), grid_of(slots * tiles_n), dim3(64 * NW * KG), 0,
                     stream, a, (int)tiles_n, group_m);
  return hipGetLastError();
}

// Offsets of 32 bits: from an expert's weight; from a tile's first row of x, with
// a row index from the first row.
bool fused_mid_takes(const FusedArgs& a, int fmt) {
  const int64_t most = ((int64_t)1 << 32) - 1;
  return a.K >= 4 * BLOCK_K && a.K <= ((int64_t)1 << 24) && a.N <= most / (fmt == 0 ? a.K / 4 : a.K / 2) &&
         (!a.row_index || a.x_rows <= most / (2 * a.K));
}

// The tile.  K split over four or eight groups of waves makes a workgroup take a
// CU for itself, so 256 of them are a round; two of K split over two share a CU.
// Of the sizes below the one with the least rounds times the time of a round is
// taken, as measured at one K in one format; other K and Q2_0 are taken to stretch all
// of them alike (K = 2560, 4-bit, us per round: 32 x 64 over eight groups 12.6; over four
// 32 x 96 14.5, 64 x 64 17.0, 64 x 96 20.5, 64 x 128 23.4, 64 x 160 26.4; over two
// 64 x 128 28 up to 256 workgroups and 36 up to 512).  So 128 rows, N = 2 x 9728
// take 64 x 160 (29 us, 36 with 64 x 128 over two), N = 8192 64 x 64, N = 2560
// 32 x 64 (12.6, 18 over two), 384 rows N = 2 x 9728 64 x 128 over two (69, 75 with
// 64 x 160).
// Groups of rows, whose number of tiles is not known here, take K over two, with
// 64 rows per tile once the mean group fills two of them (128 rows each, K = 2048,
// 2 x 1408 4-bit: 114 us against 116), else 32 (64 rows each: 69 against 98 with K
// over four); a launch that can make few tiles only takes 32 x 64.
template <int FMT>
static hipError_t pick_mid(const FusedArgs& a, hipStream_t stream) {
  if (a.offsets) {
    if (max_row_tiles(a, 32) * ((a.N + 127) / 128) <= 128) return run_mid<FMT, 2, 4, 1, 8, 2>(a, stream);
    if (a.M >= 128 * a.E) return run_mid<FMT, 4, 4, 2, 2, 2>(a, stream);
    return run_mid<FMT, 2, 4, 2, 2, 2>(a, stream);
  }
  auto tiles = [&](int64_t bm, int64_t bn) {
    const int64_t cols = a.gated ? bn / 2 : bn;
    return ((a.M + bm - 1) / bm) * ((fused_n_out(a) + cols - 1) / cols);
  };
  const int64_t pairs = tiles(64, 128), rest = pairs % 512;
  double least = (double)(pairs / 512) * 36. + (rest == 0 ? 0. : rest <= 256 ? 28. : 36.);
  int pick = 0;
  auto offer = [&](int id, int64_t bm, int64_t bn, double round) {
    const double t = (double)((tiles(bm, bn) + 255) / 256) * round;
    if (t < least) least = t, pick = id;
  };
  offer(1, 32, 64, 12.6);
  offer(2, 32, 96, 14.5);
  offer(3, 64, 64, 17.0);
  offer(4, 64, 96, 20.5);
  offer(5, 64, 128, 23.4);
  offer(6, 64, 160, 26.4);
  switch (pick) {
    case 1: return run_mid<FMT, 2, 4, 1, 8, 2>(a, stream);
    case 2: return run_mid<FMT, 2, 3, 2, 4, 2>(a, stream);
    case 3: return run_mid<FMT, 4, 2, 2, 4, 2>(a, stream);
    case 4: return run_mid<FMT, 4, 3, 2, 4, 2>(a, stream);
    case 5: return run_mid<FMT, 4, 4, 2, 4, 2>(a, stream);
    case 6: return run_mid<FMT, 4, 5, 2, 4, 2>(a, stream);
    default: return run_mid<FMT, 4, 4, 2, 2, 2>(a, stream);
  }
}

hipError_t launch_fused_mid(const FusedArgs& a, int fmt, hipStream_t stream) {
  return fmt == 0 ? pick_mid<0>(a, stream) : pick_mid<1>(a, stream);
}

}  // namespace q2dev
