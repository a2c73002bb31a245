// q2_fused.h - arguments, epilogue and row-group lookup shared by the kernels of
// the fused and grouped linears.
#pragma once
#include "q2.h"
#include "q2_device.h"
#include <algorithm>

namespace q2dev {

// One fused or grouped linear.  Rows of x and y are numbered over all experts;
// without experts (offsets == nullptr) there is one group of M rows.
struct FusedArgs {
  const uint16_t* x;          // bf16 [x_rows, K]
  const int32_t* row_index;   // row of x that row i reads, or nullptr (i); outside [0, x_rows): zeros
  int64_t x_rows;
  const uint8_t* w;           // codes [E, N, K/4] or [E, N, K/2]
  const uint16_t* s;          // f16 scales [E, N, K/128]
  const uint16_t* z;          // f16 zero points, 4-bit only
  const int32_t* offsets;     // [E + 1] or nullptr
  int64_t E, M, N, K;         // N counts weight rows
  const uint16_t* lr_a;       // f16 [r, K]; r > 0 only without groups
  uint16_t* lr_t;             // bf16 limbs [M, 2 r8] of x A^T, written by the launch
  const uint16_t* lr_b;       // f16 [N, r]
  int r;
  int act, gated, out_bf16, res_bf16;
  const float* bias;          // [E, N] or nullptr
  const float* gate;          // [n_out] or nullptr
  const void* residual;       // [M, n_out] or nullptr
  void* y;                    // [M, n_out]
};

__host__ __device__ __forceinline__ int64_t fused_n_out(const FusedArgs& a) { return a.gated ? a.N / 2 : a.N; }

// ---- decode --------------------------------------------------------------------
// q2_bfrag_nat and q4_bfrag_nat of q2_device.h without inline assembly: the
// compiler spaces a matrix instruction from the vector instruction that writes
// its operand, but not from one it does not see as such.  (Written with inline
// assembly, a fragment whose last dword was followed by one scalar instruction
// and then its matrix instruction came out wrong on every run.)
typedef uint16_t q2_u16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t shr16(uint32_t v, uint32_t sh) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(q2_u16x2, v) >> __builtin_bit_cast(q2_u16x2, sh));
}
template <int H>
__device__ __forceinline__ q2_u32x4 q2_frag(uint32_t w, const NatConsts& k) {
  const uint32_t u0 = byte_to_halves<2 * H>(w), u1 = byte_to_halves<2 * H + 1>(w);
  return q2_u32x4{(shr16(u0, k.sh01) & k.mask) | k.one, (shr16(u0, k.sh23) & k.mask) | k.one,
                  (shr16(u1, k.sh01) & k.mask) | k.one, (shr16(u1, k.sh23) & k.mask) | k.one};
}
__device__ __forceinline__ q2_u32x4 q4_frag(uint32_t w, const NatConsts& k) { return q4_bfrag_nat(w, k); }

// ---- the codes of a row, 64 bytes at a time --------------------------------------
// A unit is four 16-byte pieces of a row: `per` blocks, two of 2-bit codes or one
// of 4-bit codes.  Prefetches run past the last unit and, with an odd number of
// 2-bit blocks, past the row inside it; what they load there is never used, but the
// scalar offset of a buffer load is no part of its bounds check, so they stay in the
// row: piece p of unit u lies at unit_start + 16 p - unit_back.
__host__ __device__ constexpr int last_unit(int blocks, int per) { return (blocks + per - 1) / per - 1; }
__host__ __device__ constexpr uint32_t unit_start(int u, int blocks, int per) {
  return 64u * (uint32_t)(u < last_unit(blocks, per) ? u : last_unit(blocks, per));
}
__host__ __device__ constexpr uint32_t unit_back(int u, int blocks, int per, int piece) {
  return per == 2 && (blocks & 1) && u >= last_unit(blocks, per) && piece >= 2 ? 32u : 0u;
}

// ---- the rank-r branch -----------------------------------------------------------
// Its matrix-core operands: x A^T as limbs [M, 2 r8] (hi | lo), B split exactly
// into bf16 hi + lo, added up as T_hi B_hi + T_hi B_lo + T_lo B_hi (the dropped
// T_lo B_lo is 2^-16 of the branch).  Eight elements from q0 on.
__device__ __forceinline__ q2_u32x4 branch_afrag(const FusedArgs& a, int64_t m, int q0, bool low) {
  const int r8 = (a.r + 7) & ~7;
  m = m < a.M ? m : a.M - 1;
  if (q0 >= r8) return q2_u32x4{0u, 0u, 0u, 0u};
  return *reinterpret_cast<const q2_u32x4*>(a.lr_t + m * 2 * r8 + (low ? r8 : 0) + q0);
}
// Eight elements of B as hi and lo: one load where r is a multiple of eight and
// B 16-byte aligned, else one by one.
struct BranchB {
  q2_u32x4 hi, lo;
};
__device__ __forceinline__ BranchB branch_bfrag(const FusedArgs& a, int64_t n, int q0) {
  uint16_t h[8] = {};
  const uint16_t* const p = a.lr_b + n * a.r + q0;
  if (a.r % 8 == 0 && (reinterpret_cast<uintptr_t>(a.lr_b) & 15) == 0) {
    if (q0 < a.r) __builtin_memcpy(h, __builtin_assume_aligned(p, 16), 16);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (q0 + k < a.r) h[k] = p[k];
  }
  BranchB b;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    uint16_t hi0, lo0, hi1, lo1;
    f16_split_bf16(h[2 * d], hi0, lo0);
    f16_split_bf16(h[2 * d + 1], hi1, lo1);
    b.hi[d] = hi0 | ((uint32_t)hi1 << 16);
    b.lo[d] = lo0 | ((uint32_t)lo1 << 16);
  }
  return b;
}

// ---- epilogue ----------------------------------------------------------------
// exp and the reciprocal are the hardware's (about one ulp each); both GELU and
// SiLU are v times a logistic or normal distribution function, so a large |v|
// gives v or a zero, never inf / inf.
// The normal distribution function of -a, a >= 0, is exp(-a^2 / 2) q(1 / (1 + 0.23 a))
// with a polynomial q fitted on 0 <= a <= 13.3 for the least relative error, 4.8e-8:
// relative, as the rest of a gated pair multiplies it, where (1 + erf) / 2 keeps
// nothing below 2^-25.  It takes less time too (M = 1536, K = 4096, N = 12288: 151.6 us, 159.7).
__device__ __forceinline__ float normal_tail(float a) {
  const float s = __builtin_amdgcn_rcpf(__builtin_fmaf(0.23f, a, 1.0f));
  float q = -0.078409999609f;
  q = __builtin_fmaf(q, s, 0.290122002363f);
  q = __builtin_fmaf(q, s, -0.277491927147f);
  q = __builtin_fmaf(q, s, 0.300703167915f);
  q = __builtin_fmaf(q, s, -0.032352376729f);
  q = __builtin_fmaf(q, s, 0.119253337383f);
  q = __builtin_fmaf(q, s, 0.085835561156f);
  q = __builtin_fmaf(q, s, 0.092367239296f);
  q = __builtin_fmaf(q, s, -2.7028827390e-05f);
  return q * __builtin_amdgcn_exp2f(-0.72134752044448170f * (a * a));        // log2(e) / 2
}
__device__ __forceinline__ float logistic(float v) { return __builtin_amdgcn_rcpf(1.0f + __expf(-v)); }

__device__ __forceinline__ float activate(int act, float v) {
  switch (act) {
    case Q2_ACT_RELU: return v < 0.0f ? 0.0f : v;         // a NaN stays one (fmaxf would drop it)
    case Q2_ACT_GELU: {
      const float tail = normal_tail(fabsf(v));
      return v * (v < 0.0f ? tail : 1.0f - tail);
    }
    // (1 + tanh u) / 2 is the logistic function of 2 u
    case Q2_ACT_GELU_TANH: return v * logistic(1.5957691216057308f * (v + 0.044715f * v * v * v));
    case Q2_ACT_SILU: return v * logistic(v);
    default: return v;
  }
}

// The same for eight values, with one choice of the activation.
__device__ __forceinline__ void activate8(int act, float (&v)[8]) {
  auto all = [&](auto f) {
#pragma unroll
    for (int d = 0; d < 8; ++d) v[d] = f(v[d]);
  };
  switch (act) {
    case Q2_ACT_RELU: return all([](float t) { return activate(Q2_ACT_RELU, t); });
    case Q2_ACT_GELU: return all([](float t) { return activate(Q2_ACT_GELU, t); });
    case Q2_ACT_GELU_TANH: return all([](float t) { return activate(Q2_ACT_GELU_TANH, t); });
    case Q2_ACT_SILU: return all([](float t) { return activate(Q2_ACT_SILU, t); });
    default: return;
  }
}

__device__ __forceinline__ float load_elem(const void* p, int64_t i, int bf16) {
  return bf16 ? bf16_to_f32(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

// bf16 bits of v, nearest even, NaN kept (the hardware's conversion).
__device__ __forceinline__ uint16_t to_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// One output element from its product v (and, gated, the product u of the
// second half's row): row m, output column n, of an expert with bias `bias`.
__device__ __forceinline__ void store_out(const FusedArgs& a, const float* bias, int64_t n_out, int64_t m, int64_t n,
                                          float v, float u) {
  if (bias) v += bias[n];
  v = activate(a.act, v);
  if (a.gated) v *= bias ? u + bias[n_out + n] : u;
  if (a.gate) v *= a.gate[n];
  const int64_t i = m * n_out + n;
  if (a.residual) v += load_elem(a.residual, i, a.res_bf16);
  if (a.out_bf16) static_cast<uint16_t*>(a.y)[i] = to_bf16(v);
  else static_cast<float*>(a.y)[i] = v;
}

// ROWS x (64 or 32 output columns) of finished products in LDS (row stride
// `stride` floats; with a gated epilogue the second factor of column n at
// `half` + n) to y, by the 64 lanes of one wave: pieces of eight columns
// where y, the residual and the column count allow it.
__device__ __forceinline__ bool vec_rows(const FusedArgs& a, int64_t n_out) {
  // a grouped bias starts E * N floats in: with n_out % 8 == 0 every expert's is aligned with the first
  const uintptr_t p = reinterpret_cast<uintptr_t>(a.y) | reinterpret_cast<uintptr_t>(a.residual) |
                      reinterpret_cast<uintptr_t>(a.bias) | reinterpret_cast<uintptr_t>(a.gate);
  return n_out % 8 == 0 && (p & 15) == 0;
}

struct Eight {
  float v[8];
};
__device__ __forceinline__ Eight load8f(const float* p) {
  const q2_f32x4 a = reinterpret_cast<const q2_f32x4*>(p)[0], b = reinterpret_cast<const q2_f32x4*>(p)[1];
  return Eight{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
}
// Eight elements of the residual, as they lie in memory and as floats.
struct EightRaw {
  q2_u32x4 w[2];
};
__device__ __forceinline__ EightRaw load8raw(const void* p, int64_t i, int bf16) {
  EightRaw r = {};
  if (bf16) {
    r.w[0] = *reinterpret_cast<const q2_u32x4*>(static_cast<const uint16_t*>(p) + i);
  } else {
    const q2_u32x4* q = reinterpret_cast<const q2_u32x4*>(static_cast<const float*>(p) + i);
    r.w[0] = q[0];
    r.w[1] = q[1];
  }
  return r;
}
__device__ __forceinline__ Eight raw_floats(const EightRaw& r, int bf16) {
  Eight f;
#pragma unroll
  for (int d = 0; d < 8; ++d) {
    const uint32_t h = r.w[0][d >> 1], lo = (d & 1) ? h & 0xFFFF0000u : h << 16;
    f.v[d] = __builtin_bit_cast(float, bf16 ? lo : r.w[d >> 2][d & 3]);
  }
  return f;
}

// The residual of four pieces is loaded before the first is finished, and the
// bias and gate of a lane's columns once where every piece of it has the same
// ones: a wave that waits for each in turn spends most of the epilogue waiting
// (M = 4093, N = 4096 with a residual in 32 bits: 55 us of every tile's time).
__device__ __forceinline__ void store_strip(const FusedArgs& a, const float* bias, int64_t n_out, const float* strip,
                                            int stride, int half, int cols, int64_t m0, int rows, int64_t n0,
                                            int lane) {
  if (vec_rows(a, n_out)) {
    constexpr int BATCH = 4;
    const int per = cols / 8, total = rows * per;        // pieces of eight columns per row
    const bool fixed = 64 % per == 0;
    Eight b = {}, bu = {}, g = {};
    auto columns = [&](int64_t n) {
      if (bias) b = load8f(bias + n);
      if (bias && a.gated) bu = load8f(bias + n_out + n);
      if (a.gate) g = load8f(a.gate + n);
    };
    if (fixed && n0 + lane % per * 8 < n_out) columns(n0 + lane % per * 8);
    for (int base = lane; base < total; base += 64 * BATCH) {
      EightRaw res[BATCH] = {};
      if (a.residual) {
#pragma unroll
        for (int p = 0; p < BATCH; ++p) {
          const int idx = base + 64 * p, row = idx / per;
          const int64_t n = n0 + (idx - row * per) * 8;
          if (idx < total && n < n_out) res[p] = load8raw(a.residual, (m0 + row) * n_out + n, a.res_bf16);
        }
      }
#pragma unroll 1                                          // the code once: unrolled it was 4 % of a gated layer's time
      for (int p = 0; p < BATCH; ++p) {
        const EightRaw now = res[0];
#pragma unroll
        for (int q = 1; q < BATCH; ++q) res[q - 1] = res[q];
        const int idx = base + 64 * p, row = idx / per, col = (idx - row * per) * 8;
        const int64_t n = n0 + col;
        if (idx >= total || n >= n_out) continue;
        if (!fixed) columns(n);
        const float* s = strip + row * stride + col;
        Eight v = load8f(s);
        if (bias) {
#pragma unroll
          for (int d = 0; d < 8; ++d) v.v[d] += b.v[d];
        }
        activate8(a.act, v.v);
        if (a.gated) {
          const Eight u = load8f(s + half);
#pragma unroll
          for (int d = 0; d < 8; ++d) v.v[d] *= bias ? u.v[d] + bu.v[d] : u.v[d];
        }
        if (a.gate) {
#pragma unroll
          for (int d = 0; d < 8; ++d) v.v[d] *= g.v[d];
        }
        if (a.residual) {
          const Eight r = raw_floats(now, a.res_bf16);
#pragma unroll
          for (int d = 0; d < 8; ++d) v.v[d] += r.v[d];
        }
        const int64_t i = (m0 + row) * n_out + n;
        if (a.out_bf16) {
          q2_u32x4 o;
#pragma unroll
          for (int d = 0; d < 4; ++d)
            o[d] = (uint32_t)to_bf16(v.v[2 * d]) | ((uint32_t)to_bf16(v.v[2 * d + 1]) << 16);
          *reinterpret_cast<q2_u32x4*>(static_cast<uint16_t*>(a.y) + i) = o;
        } else {
          q2_f32x4* y = reinterpret_cast<q2_f32x4*>(static_cast<float*>(a.y) + i);
          y[0] = q2_f32x4{v.v[0], v.v[1], v.v[2], v.v[3]};
          y[1] = q2_f32x4{v.v[4], v.v[5], v.v[6], v.v[7]};
        }
      }
    }
  } else {
    // A lane keeps its column (and with narrow strips a share of the rows), eight
    // rows at a time: M = 1536, K = 4096, N = 12289 with a residual 209 us, an
    // element at a time 373 (N = 12288: 168).
    constexpr int ROWS = 8;
    const int share = cols < 64 && 64 % cols == 0 ? 64 / cols : 1;
    const int lrow = share > 1 ? lane / cols : 0, lcol = lane - lrow * cols * (share > 1);
    for (int c0 = 0; c0 < cols; c0 += 64) {
      const int col = c0 + lcol;
      const int64_t n = n0 + col;
      const bool live = col < cols && n < n_out;
      const float b = bias && live ? bias[n] : 0.f, bu = bias && a.gated && live ? bias[n_out + n] : 0.f;
      const float g = a.gate && live ? a.gate[n] : 1.f;
      if (!live) continue;
      for (int r0 = lrow; r0 < rows; r0 += ROWS * share) {
        float v[ROWS], u[ROWS], res[ROWS];
#pragma unroll
        for (int q = 0; q < ROWS; ++q) {
          const int row = min(r0 + q * share, rows - 1); // past the end: the last row again, not stored
          res[q] = a.residual ? load_elem(a.residual, (m0 + row) * n_out + n, a.res_bf16) : 0.f;
          v[q] = strip[row * stride + col];
          u[q] = a.gated ? strip[row * stride + half + col] : 0.f;
        }
        if (bias) {
#pragma unroll
          for (int q = 0; q < ROWS; ++q) v[q] += b, u[q] += bu;
        }
        activate8(a.act, v);
#pragma unroll
        for (int q = 0; q < ROWS; ++q) {
          if (a.gated) v[q] *= u[q];
          if (a.gate) v[q] *= g;
          if (a.residual) v[q] += res[q];
          const int row = r0 + q * share;
          const int64_t i = (m0 + row) * n_out + n;
          if (row >= rows) continue;
          if (a.out_bf16) static_cast<uint16_t*>(a.y)[i] = to_bf16(v[q]);
          else static_cast<float*>(a.y)[i] = v[q];
        }
      }
    }
  }
}

// ---- grids -----------------------------------------------------------------------
// A launch of 2^32 or more threads along one dimension runs without an error, but
// not all of it.  Workgroups past GRID_X go along the second dimension, which may
// reach past the last one.
constexpr int GRID_X = 1 << 21;
inline dim3 grid_of(int64_t workgroups) {
  return workgroups <= GRID_X ? dim3((unsigned)workgroups)
                              : dim3(GRID_X, (unsigned)((workgroups + GRID_X - 1) / GRID_X));
}
__device__ __forceinline__ int workgroup_id() { return (int)(blockIdx.x + blockIdx.y * (unsigned)GRID_X); }

// ---- row groups ----------------------------------------------------------------
// Offsets are clamped to [0, M] and to not decrease within a group, so whatever
// they hold, the rows lie inside x and y.
struct RowTile {
  int64_t m0, mend;           // rows m0 .. min(m0 + bm, mend) - 1
  int64_t expert;
};

__device__ __forceinline__ int64_t clamp_offset(int32_t v, int64_t lo, int64_t hi) {
  return v < lo ? lo : v > hi ? hi : v;
}

// Tiles of bm rows of group e (offsets clamped) for the lane that asks.
__device__ __forceinline__ int group_tiles(const FusedArgs& a, int64_t e, int bm, int& lo, int& hi) {
  lo = hi = 0;
  if (e < a.E) {
    lo = (int)clamp_offset(a.offsets[e], 0, a.M);
    hi = (int)clamp_offset(a.offsets[e + 1], lo, a.M);
  }
  return (int)(((int64_t)hi - lo + bm - 1) / bm);
}

// The tile of this workgroup; false when there is none for it (the launch covers
// the most tiles that the offsets can make).  Each XCD gets a contiguous range
// of tile numbers.  Without groups they run over blocks of group_m row tiles,
// row-fastest inside (see tile_group_rows) and from another row in each column, so
// that a row's tiles are not all on the same CUs of an XCD; with groups over the
// column tiles of a row tile, so an XCD meets few experts and reads their weights once.
// Every wave of the workgroup calls it together; the results are scalars
// (readlane), so that buffer resources built on them stay in scalar registers.
__device__ __forceinline__ bool find_tile(const FusedArgs& a, int bm, int tiles_n, int group_m, RowTile& rt, int& tn) {
  const int wg = workgroup_id();
  rt.expert = 0;
  rt.mend = a.M;
  if (a.offsets == nullptr) {
    const int tiles_m = a.M <= bm ? 1 : (int)((a.M + bm - 1) / bm);
    if (wg >= tiles_m * tiles_n) return false;
    const int tile = xcd_tile(wg, tiles_m * tiles_n);
    if (tiles_m == 1) {
      rt.m0 = 0;
      tn = tile;
      return true;
    }
    const int grp = tile / (group_m * tiles_n), gi = tile - grp * group_m * tiles_n;
    const int gm = min(group_m, tiles_m - grp * group_m);
    tn = gi / gm;
    rt.m0 = (int64_t)(grp * group_m + (gi + tn) % gm) * bm;
    return true;
  }
  const int lane = threadIdx.x & 63;
  int lo, hi, mine = group_tiles(a, lane, bm, lo, hi), total = mine;
  for (int64_t e = lane + 64; e - lane < a.E; e += 64) {
    int l, h;
    total += group_tiles(a, e, bm, l, h);
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) total += __shfl_xor(total, d);
  total = __builtin_amdgcn_readfirstlane(total);
  // bad offsets can count more tiles than the launch covers
  const int tiles = (int)min((int64_t)total * tiles_n, (int64_t)min(gridDim.x * gridDim.y, 0x7fffffffu));
  if (wg >= tiles) return false;
  const int tile = xcd_tile(wg, tiles);
  int slot = tile / tiles_n;
  tn = tile - slot * tiles_n;
  for (int64_t e0 = 0; e0 < a.E; e0 += 64) {             // slot < total: found before the last group's end
    if (e0 > 0) mine = group_tiles(a, e0 + lane, bm, lo, hi);
    int sum = mine;                                      // inclusive sum over the lanes
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(sum, d);
      if (lane >= d) sum += v;
    }
    const uint64_t past = __builtin_amdgcn_ballot_w64(sum > slot);
    if (past != 0) {
      const int l = __builtin_ctzll(past);
      rt.m0 = __builtin_amdgcn_readlane(lo, l) + (int64_t)(slot - __builtin_amdgcn_readlane(sum - mine, l)) * bm;
      rt.mend = __builtin_amdgcn_readlane(hi, l);
      rt.expert = e0 + l;
      return true;
    }
    slot -= __builtin_amdgcn_readlane(sum, 63);
  }
  return false;                                          // bad offsets whose tiles overflow their sum
}

// At most this many row tiles of bm rows over all groups: each of the at most
// min(E, M) groups with rows adds less than one tile to M / bm.
inline int64_t max_row_tiles(const FusedArgs& a, int bm) {
  if (a.offsets == nullptr) return (a.M + bm - 1) / bm;
  const int64_t groups = a.E < a.M ? a.E : a.M;
  return (a.M + groups * (bm - 1)) / bm;
}

// Row tiles per block of the tile order.  Cutting the tile grid into p row parts
// times 8 / p column parts, one block per XCD, makes the XCDs together read the
// weights p times and x 8 / p times; once an XCD runs its block in several
// rounds (`resident` tiles at a time) its rows of x are read again in each,
// unless they stay in its 4 MB L2.  p is the power of two with the least sum.
inline int tile_group_rows(int64_t tiles_m, int64_t tiles_n, double xtile, double wtile, int resident) {
  const double rounds = std::max(1.0, (double)tiles_m * (double)tiles_n / 8.0 / resident);
  auto cost = [&](int p) {
    const double xpart = (double)((tiles_m + p - 1) / p) * xtile;
    return 8.0 * xpart * (xpart <= 2.5e6 ? 1.0 : rounds) + p * wtile * (double)tiles_n;
  };
  int best = 1;
  for (int p = 2; p <= 8 && p <= tiles_m; p *= 2)
    if (cost(p) < cost(best)) best = p;
  return (int)((tiles_m + best - 1) / best);
}

// ---- host side -------------------------------------------------------------------
// Workspace beside the limbs of a rank-r branch; 0 where none is needed.
size_t fused_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t E, int fmt);
// fmt 0 = Q2_0, 1 = 4-bit.  ws: that many bytes.
hipError_t launch_fused(const FusedArgs& a, int fmt, void* ws, hipStream_t stream);

bool fused_mid_takes(const FusedArgs& a, int fmt);
hipError_t launch_fused_mid(const FusedArgs& a, int fmt, hipStream_t stream);
int64_t few_tiles(const FusedArgs& a);                   // workgroups of launch_fused_few without groups
hipError_t launch_fused_few(const FusedArgs& a, int fmt, hipStream_t stream);
size_t f16_workspace_bytes(int64_t rows, int64_t K);
bool fused_f16_takes(int64_t rows, int64_t N, int64_t K);
hipError_t launch_fused_f16(const FusedArgs& a, void* ws, hipStream_t stream);

hipError_t launch_route(const void* logits, int logits_bf16, int64_t T, int64_t E, int k, int renorm, int32_t* expert,
                        float* weight, int32_t* offsets, int32_t* row_token, int32_t* slot, void* ws,
                        hipStream_t stream);
size_t route_workspace_bytes(int64_t T, int64_t E);
hipError_t launch_combine(const void* z, int z_bf16, int64_t R, const int32_t* slot, const float* weight,
                          const void* residual, int res_bf16, void* y, int out_bf16, int64_t T, int k, int64_t N,
                          hipStream_t stream);

}  // namespace q2dev
