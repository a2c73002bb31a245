// q2_fused_f16.hip - the fused and grouped Q2_0 linears for many rows.
//
// A Q2_0 weight is -d, 0 or d with an f16 scale d, so it is an f16 value as it
// stands; what keeps the product off the f16 matrix cores is the range of the
// bf16 activations.  Here each row of x is first multiplied by a power of two
// that puts its largest element into [2^15, 2^16) and converted to f16.  A bf16
// value has 8 significant bits, so every element down to 2^-32 of its row's
// largest is exact.  Then the sum over all of K runs in the matrix cores' fp32
// accumulators with exact products, without a block's start value, row sums or
// a rescale per block; the power of two is taken back by an exact ldexp.
//
// What the conversion rounds off smaller elements is at most 2^-40 of the row's
// largest one, but that is the whole result of an output whose weights at the larger
// elements are zero.  So a row that loses something in one element has that
// element's place and remainder listed, and its outputs get the remainder times
// their weight at the end (among 5e7 normal numbers there is such an element now and
// then).  A row that loses in more (a wide row) stays bf16, and a tile that holds
// one runs on the bf16 matrix cores with each weight as the exact sum of two bf16
// values, at twice the products.
#include "q2_fused.h"
#include "q2_internal.h"
#include <algorithm>
#include <type_traits>

namespace q2dev {

typedef _Float16 q2_f16x8 __attribute__((ext_vector_type(8)));
typedef float q2_f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ q2_f32x16 mfma32(q2_u32x4 a, q2_u32x4 b, q2_f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(q2_f16x8, a), __builtin_bit_cast(q2_f16x8, b), c, 0,
                                                0, 0);
}
__device__ __forceinline__ q2_f32x16 mfma32_bf16(q2_u32x4 a, q2_u32x4 b, q2_f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(q2_bf16x8, a), __builtin_bit_cast(q2_bf16x8, b), c,
                                                 0, 0, 0);
}

// ============================================================================
// x as f16: row i of the output is row i of x times 2^-(rowinfo[i] >> 2)
// ============================================================================
// Each group of 16 elements is stored as a transposed 4 x 4 matrix (position
// 4 j + b holds element 4 b + j), the order in which a dword of sixteen codes
// decodes.

// The largest and the smallest nonzero |x| of the elements so far, as bf16 bits in
// each half of a word, the smallest less one: zeros count as 0xFFFF.  An infinity or
// a NaN is the largest; its row has no finite product whatever its exponent is.
struct Span {
  q2_u16x2 top = {0, 0}, low = {0xFFFF, 0xFFFF};
  __device__ __forceinline__ void add(const q2_u32x4& v) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const q2_u16x2 m = __builtin_bit_cast(q2_u16x2, v[d] & 0x7FFF7FFFu);
      top = __builtin_elementwise_max(top, m);
      low = __builtin_elementwise_min(low, (q2_u16x2)(m - q2_u16x2{1, 1}));
    }
  }
  // Both in one word of which a maximum per half joins two: top, low's complement.
  __device__ __forceinline__ uint32_t word() const {
    return (uint32_t)max(top[0], top[1]) << 16 | (0xFFFFu - min(low[0], low[1]));
  }
};
__device__ __forceinline__ uint32_t join_span(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(
      uint32_t, __builtin_elementwise_max(__builtin_bit_cast(q2_u16x2, a), __builtin_bit_cast(q2_u16x2, b)));
}
// Whether a row may lose something: its smallest nonzero element lies below 2^-32
// times the power of two of its largest.  (Every bf16 is a multiple of 2^-133, which
// is exact as long as the largest element lies below 2^-93.)
__device__ __forceinline__ bool may_lose(uint32_t span) {
  const int limit = (int)(span >> 23) - 32;              // exponent of 2^-32 times the largest
  return limit > 1 && span >> 16 < 0x7F80u && 0x10000u - (span & 0xFFFFu) < (uint32_t)limit << 7;
}
// What a row's info word says below its exponent.
constexpr int ROW_LOST = 1, ROW_WIDE = 2;
__device__ __forceinline__ int row_word(int shift, int lost) { return lost > 1 ? ROW_WIDE : -4 * shift | lost; }
// The input and the remainder of a row with ROW_LOST.
struct Lost {
  int32_t k;
  float r;
};
// Adds up how many of sixteen elements from input k on the conversion rounds; the last of them is kept.
__device__ __forceinline__ void find_lost(const q2_u32x4& v0, const q2_u32x4& v1, int shift, int k, int& n, Lost& l) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t w = (i < 8 ? v0[(i & 7) >> 1] : v1[(i & 7) >> 1]);
    const float x = __builtin_bit_cast(float, (i & 1) ? w & 0xFFFF0000u : w << 16);
    const float r = x - __builtin_amdgcn_ldexpf((float)(_Float16)__builtin_amdgcn_ldexpf(x, shift), -shift);
    if (r != 0.f) {
      ++n;
      l = Lost{k + i, r};
    }
  }
}

// The shift that puts the largest into [2^15, 2^16): floor(log2 |x|) from the bits (a
// subnormal bf16 is bits * 2^-133); 0 for a row of zeros.
__device__ __forceinline__ int top_shift(uint32_t top) {
  const int e = top >= 0x80u ? (int)(top >> 7) - 127 : top ? 31 - __builtin_clz(top) - 133 : 15;
  return 15 - e;
}
// Sixteen elements as f16 pairs in their own order.
__device__ __forceinline__ void to_f16(const q2_u32x4& v0, const q2_u32x4& v1, int shift, uint32_t (&h)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = i < 4 ? v0[i] : v1[i - 4];
    const _Float16 lo = (_Float16)__builtin_amdgcn_ldexpf(__builtin_bit_cast(float, w << 16), shift);
    const _Float16 hi = (_Float16)__builtin_amdgcn_ldexpf(__builtin_bit_cast(float, w & 0xFFFF0000u), shift);
    h[i] = (uint32_t)__builtin_bit_cast(uint16_t, lo) | ((uint32_t)__builtin_bit_cast(uint16_t, hi) << 16);
  }
}
// The stored order: positions 2 p, 2 p + 1 hold elements 4 b + j and 4 b + 4 + j
// with j = p / 2, b = 2 (p % 2), i.e. halves j % 2 of dwords 2 b + j / 2 and + 2.
__device__ __forceinline__ void store_f16(q2_u32x4* dst, const uint32_t (&h)[8]) {
  q2_u32x4 o[2];
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int j = p >> 1, b = 2 * (p & 1), d = 2 * b + (j >> 1);
    o[p >> 2][p & 3] = __builtin_amdgcn_perm(h[d + 2], h[d], (j & 1) ? 0x07060302u : 0x05040100u);
  }
  dst[0] = o[0];
  dst[1] = o[1];
}

// The elements of a wide row, kept: bf16 bits.
__device__ __forceinline__ void keep_bf16(const q2_u32x4& v0, const q2_u32x4& v1, uint32_t (&h)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = i < 4 ? v0[i] : v1[i - 4];
}

// Rows without a branch: one wave per row, which stays in registers up to
// 1024 NCH elements between the search for its largest element and the
// conversion (NCH = 0: longer rows, read twice).  Rows between 4096 and 12288 take
// the form for 12288, which loads their last elements again in the rest of its
// places.  Row M (of M + 1) is a row of zeros that indexes outside x are pointed to.
constexpr int CV_ROWS = 4;

template <int NCH>
__global__ __launch_bounds__(64 * CV_ROWS) void x_to_f16_kernel(const uint16_t* x, uint16_t* out, int32_t* rowinfo,
                                                                Lost* lost, int64_t M, int64_t K) {
  const int lane = threadIdx.x & 63;
  const int64_t m = (int64_t)blockIdx.x * CV_ROWS + (threadIdx.x >> 6);
  if (m > M) return;
  const int64_t chunks = K / 16;
  q2_u32x4* const dst = reinterpret_cast<q2_u32x4*>(out + m * K);
  if (m == M) {
    for (int64_t q = lane; q < 2 * chunks; q += 64) dst[q] = q2_u32x4{0u, 0u, 0u, 0u};
    if (lane == 0) rowinfo[m] = 0;
    return;
  }
  const q2_u32x4* const xr = reinterpret_cast<const q2_u32x4*>(x + m * K);
  constexpr int N = NCH > 0 ? NCH : 1;
  q2_u32x4 v[N][2];
  Span sp;
  if constexpr (NCH > 0) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int64_t q = std::min<int64_t>(lane + 64 * i, chunks - 1);     // past the row: its last elements again
      v[i][0] = xr[2 * q];
      v[i][1] = xr[2 * q + 1];
    }
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      sp.add(v[i][0]);
      sp.add(v[i][1]);
    }
  } else {
    for (int64_t q = lane; q < 2 * chunks; q += 64) sp.add(xr[q]);
  }
  uint32_t span = sp.word();
#pragma unroll
  for (int d = 32; d; d >>= 1) span = join_span(span, (uint32_t)__shfl_xor((int)span, d));
  const int shift = top_shift(span >> 16);
  uint32_t h[8];
  if (__builtin_amdgcn_readfirstlane((int)may_lose(span)) != 0) {        // rare: from memory again, in short loops
    int n = 0;
    Lost l = {};
#pragma unroll 1
    for (int64_t q = lane; q < chunks; q += 64) find_lost(xr[2 * q], xr[2 * q + 1], shift, (int)(16 * q), n, l);
    const uint64_t lanes = __builtin_amdgcn_ballot_w64(n > 0);
    const bool wide = __builtin_popcountll(lanes) > 1 || __builtin_amdgcn_ballot_w64(n > 1) != 0;
    if (n == 1 && !wide) lost[m] = l;
    if (lane == 0) rowinfo[m] = row_word(shift, wide ? 2 : lanes != 0);
#pragma unroll 1
    for (int64_t q = lane; q < chunks; q += 64) {
      if (wide) keep_bf16(xr[2 * q], xr[2 * q + 1], h);
      else to_f16(xr[2 * q], xr[2 * q + 1], shift, h);
      store_f16(dst + 2 * q, h);
    }
    return;
  }
  if (lane == 0) rowinfo[m] = row_word(shift, 0);
  if constexpr (NCH > 0) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int64_t q = lane + 64 * i;
      if (q < chunks) {
        to_f16(v[i][0], v[i][1], shift, h);
        store_f16(dst + 2 * q, h);
      }
    }
  } else {
    for (int64_t q = lane; q < chunks; q += 64) {
      to_f16(xr[2 * q], xr[2 * q + 1], shift, h);
      store_f16(dst + 2 * q, h);
    }
  }
}

// Rows with a rank-r branch, r <= 64: sixteen rows per workgroup of sixteen
// waves, each wave every sixteenth run of 64 inputs (lane (c, g): row c, inputs
// 16 g .. + 15 of the run).  x is read once up to K = 12288 (8192 for r > 32), converted, stored
// and multiplied by A (f16 as it is: exact products) while it is in registers;
// the waves' sums of x A^T meet in LDS and leave as the branch's bf16 limbs.
// Reading x once for both took a call at M = 4093, K = 12288, N = 4096, r = 32
// from 487 us to 445; this kernel is 70 us of it, 200 MB at 2.9 TB/s: sixteen
// rows fill a CU's registers, so its loads and its stores take turns.  There is one
// form per rank: shorter rows load their last run again in the places they do not fill.
constexpr int XA_WAVES = 16, XA_MAX_RANK = 64;

__device__ __forceinline__ q2_f32x4 mfma16_f16(q2_u32x4 a, q2_u32x4 b, q2_f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(q2_f16x8, a), __builtin_bit_cast(q2_f16x8, b), c, 0,
                                                0, 0);
}

template <int CT>
__global__ __launch_bounds__(64 * XA_WAVES) void x_to_f16_branch_kernel(const uint16_t* x, const uint16_t* A,
                                                                        uint16_t* out, int32_t* rowinfo, Lost* lost,
                                                                        uint16_t* limbs, int64_t M, int64_t K, int r) {
  constexpr int XA_RUNS = CT <= 2 ? 12 : 8;              // of a wave, in registers
  __shared__ uint32_t spans[XA_WAVES][16];
  __shared__ int lost_n[16];
  __shared__ q2_f32x4 red[XA_WAVES][CT][64];
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = (int64_t)blockIdx.x * 16;
  const int64_t m = std::min<int64_t>(m0 + c, M - 1);    // rows past the end repeat the last one, not stored
  const bool live = m0 + c < M;
  const int runs = (int)(K / 64);
  const uint16_t* const xr = x + m * K + 16 * g;
  q2_u32x4 v[XA_RUNS][2];
  Span sp;
#pragma unroll
  for (int i = 0; i < XA_RUNS; ++i) {
    const int s = min(wv + XA_WAVES * i, runs - 1);
    const q2_u32x4* p = reinterpret_cast<const q2_u32x4*>(xr + (int64_t)s * 64);
    v[i][0] = p[0];
    v[i][1] = p[1];
  }
#pragma unroll
  for (int i = 0; i < XA_RUNS; ++i) {
    sp.add(v[i][0]);
    sp.add(v[i][1]);
  }
  for (int s = wv + XA_WAVES * XA_RUNS; s < runs; s += XA_WAVES) {
    const q2_u32x4* p = reinterpret_cast<const q2_u32x4*>(xr + (int64_t)s * 64);
    sp.add(p[0]);
    sp.add(p[1]);
  }
  uint32_t span = sp.word();
  span = join_span(span, (uint32_t)__shfl_xor((int)span, 16));
  span = join_span(span, (uint32_t)__shfl_xor((int)span, 32));
  if (g == 0) spans[wv][c] = span;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < XA_WAVES; ++w) span = join_span(span, spans[w][c]);
  const int shift = top_shift(span >> 16);
  const bool any =                                       // of the sixteen rows; readfirstlane: a scalar branch
      __builtin_amdgcn_readfirstlane((int)(__builtin_amdgcn_ballot_w64(may_lose(span)) != 0)) != 0;
  bool wide = false;
  if (any) {
    if (threadIdx.x < 16) lost_n[threadIdx.x] = 0;
    __syncthreads();
    int n = 0;
    Lost l = {};
    if (may_lose(span)) {
#pragma unroll 1
      for (int s = wv; s < runs; s += XA_WAVES) {
        const q2_u32x4* p = reinterpret_cast<const q2_u32x4*>(xr + (int64_t)s * 64);
        find_lost(p[0], p[1], shift, s * 64 + 16 * g, n, l);
      }
    }
    if (n > 0) atomicAdd(&lost_n[c], n);
    __syncthreads();
    wide = lost_n[c] > 1;
    if (n == 1 && !wide && live) lost[m] = l;            // one lane of the workgroup holds it
  }
  if (wv == 0 && g == 0 && live) rowinfo[m] = row_word(shift, any ? lost_n[c] : 0);

  const uint16_t* ar[CT];
#pragma unroll
  for (int t = 0; t < CT; ++t) ar[t] = A + (int64_t)min(16 * t + c, r - 1) * K + 16 * g;   // columns past r: not stored
  q2_f32x4 acc[CT];
#pragma unroll
  for (int t = 0; t < CT; ++t) acc[t] = q2_f32x4{0.f, 0.f, 0.f, 0.f};
  // With a row among them that loses something, all sixteen are multiplied as bf16, A as two bf16 values.
  auto product = [&](auto as_bf16, int s, const q2_u32x4& v0, const q2_u32x4& v1) {
    uint32_t h[8], raw[8];
    to_f16(v0, v1, shift, h);
    q2_u32x4* const dst = reinterpret_cast<q2_u32x4*>(out + m * K + (int64_t)s * 64 + 16 * g);
    if constexpr (decltype(as_bf16)::value) {
      keep_bf16(v0, v1, raw);
#pragma unroll
      for (int i = 0; i < 8; ++i) raw[i] = wide ? raw[i] : h[i];
      if (live) store_f16(dst, raw);
    } else {
      if (live) store_f16(dst, h);
    }
#pragma unroll
    for (int t = 0; t < CT; ++t) {
      const q2_u32x4* p = reinterpret_cast<const q2_u32x4*>(ar[t] + (int64_t)s * 64);
      if constexpr (decltype(as_bf16)::value) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const q2_u32x4 av = p[i], xv = i ? v1 : v0;
          q2_u32x4 hi, lo;
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            hi[d] = f16x2_bf16_hi(av[d]);
            lo[d] = f16x2_bf16_lo(av[d]);
          }
          acc[t] = mfma(xv, hi, acc[t]);
          acc[t] = mfma(xv, lo, acc[t]);
        }
      } else {
        acc[t] = mfma16_f16(q2_u32x4{h[0], h[1], h[2], h[3]}, p[0], acc[t]);
        acc[t] = mfma16_f16(q2_u32x4{h[4], h[5], h[6], h[7]}, p[1], acc[t]);
      }
    }
  };
  auto reread = [&](auto as_bf16, int s) {
    const q2_u32x4* p = reinterpret_cast<const q2_u32x4*>(xr + (int64_t)s * 64);
    product(as_bf16, s, p[0], p[1]);
  };
  if (!any) {
#pragma unroll
    for (int i = 0; i < XA_RUNS; ++i) {
      const int s = wv + XA_WAVES * i;
      if (s < runs) product(std::false_type{}, s, v[i][0], v[i][1]);
    }
    for (int s = wv + XA_WAVES * XA_RUNS; s < runs; s += XA_WAVES) reread(std::false_type{}, s);
  } else {                                               // rare: from memory again, in a short loop
#pragma unroll 1
    for (int s = wv; s < runs; s += XA_WAVES) reread(std::true_type{}, s);
  }
#pragma unroll
  for (int t = 0; t < CT; ++t) red[wv][t][lane] = acc[t];
  __syncthreads();
  const int r8 = (r + 7) & ~7;
  if (wv < CT) {                                         // one wave per column tile, waves in order
    q2_f32x4 sum = red[0][wv][lane];
#pragma unroll
    for (int w = 1; w < XA_WAVES; ++w) sum += red[w][wv][lane];
    const int col = 16 * wv + c;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = 4 * g + e;
      uint32_t rs = 0;
#pragma unroll
      for (int w = 0; w < XA_WAVES; ++w) rs = join_span(rs, spans[w][row]);
      if (m0 + row < M && col < r8) {
        const float t = col < r ? __builtin_amdgcn_ldexpf(sum[e], any ? 0 : -top_shift(rs >> 16)) : 0.f;
        const uint16_t hi = f32_to_bf16_rn(t), lo = f32_to_bf16_rn(t - bf16_to_f32(hi));
        limbs[(m0 + row) * 2 * r8 + col] = hi;
        limbs[(m0 + row) * 2 * r8 + r8 + col] = lo;
      }
    }
  }
}

// ============================================================================
// The product
// ============================================================================
// Decode: with c at the low two bits of a byte, a byte permute looks up the low
// and the high byte of c's weight in two four-entry tables, four codes at a
// time, and two more permutes join them to f16 pairs: 3 VALU operations per pair.
struct WTable {
  uint32_t lo, hi;
};
// Of the weight with 16-bit pattern v and its double v2 (the code 3).
__device__ __forceinline__ WTable weight_table(uint32_t v, uint32_t v2) {
  const uint32_t pair = v | (v2 << 16);                  // bytes lo, hi, lo2, hi2
  WTable t;
  t.lo = __builtin_amdgcn_perm(pair, pair, 0x02000C00u);                       // lo, 0, lo, lo2
  t.hi = __builtin_amdgcn_perm(pair, pair, 0x03010C01u) ^ 0x00000080u;         // -hi, 0, hi, hi2
  return t;
}
__device__ __forceinline__ WTable weight_table(uint16_t dbits) {
  const _Float16 d = __builtin_bit_cast(_Float16, dbits);
  return weight_table(dbits, __builtin_bit_cast(uint16_t, (_Float16)(d + d)));
}
// The two bf16 values that add up to the weight.
__device__ __forceinline__ void weight_tables_bf16(uint16_t dbits, WTable& hi, WTable& lo) {
  const float d = f16_to_f32(dbits);
  const float dh = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, d) & 0xFFFF0000u), dl = d - dh;
  auto top = [](float v) { return __builtin_bit_cast(uint32_t, v) >> 16; };
  hi = weight_table(top(dh), top(dh + dh));
  lo = weight_table(top(dl), top(dl + dl));
}
// K step t (0..3) of a 64-wide half block from the lane's two code dwords.
template <int T>
__device__ __forceinline__ q2_u32x4 decode_step(const q2_u32x2& w, const WTable& tab) {
  constexpr int I = T >> 1, J = 2 * (T & 1);
  q2_u32x4 r;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint32_t sel = (w[I] >> (2 * (J + u))) & 0x03030303u;
    const uint32_t lo = __builtin_amdgcn_perm(0u, tab.lo, sel), hi = __builtin_amdgcn_perm(0u, tab.hi, sel);
    r[2 * u] = __builtin_amdgcn_perm(hi, lo, 0x05010400u);
    r[2 * u + 1] = __builtin_amdgcn_perm(hi, lo, 0x07030602u);
  }
  return r;
}

// Row of x16 that row m reads: x_rows (zeros) for an index outside x.
__device__ __forceinline__ int64_t source_row(const FusedArgs& a, int64_t m) {
  const int64_t src = a.row_index[m];
  return src >= 0 && src < a.x_rows ? src : a.x_rows;
}

// M = 4093, K = 12288, N = 4096 1.25 PFLOP/s in this kernel, 8192 x 8192 x 8192
// 1.28 with the conversion, M = 1536, K = 4096, N = 12288 1.10.  The matrix cores are
// busy 70 % of the time at the 1.7 GHz that the power limit leaves them; 256-row
// tiles with half of the decode, deeper prefetch and other orders of the same
// instructions moved a call by at most 4 %.
constexpr int FX_BN = 256;                               // weight columns of a workgroup
constexpr int FX_MAX_BM = 128;
constexpr int FX_WBUF = 64 * 64;                         // codes of a wave's 64 columns, two blocks
constexpr int FX_STRIP = 64 + 4;                         // floats per row of a wave's output strip

// A workgroup of four waves owns 128 or 96 rows x 256 weight columns, each wave
// all the rows of 64 columns, so a column's weights are decoded once.  Two
// workgroups share a CU and overlap each other's waits.  Per half block (64 of
// K, half-stage hs) a wave copies a quarter of the tile's rows and a sixteenth
// of its own columns' codes to LDS:
//  - rows: two half blocks; those of hs + 1 are issued at hs (a third buffer and
//    issuing them at hs - 1 made no difference);
//  - codes: two buffers of two blocks (64 bytes of a row at a time: reading a
//    block's 32 bytes from 32 rows per instruction cost 16 % of the kernel);
//    piece q of the buffer that is used from half-stage 4 S + 4 on is issued at
//    4 S - 1 + q, after that buffer's last codes went to registers at 4 S - 2;
//  - scales: four blocks at a time in registers.
// One barrier per half-stage, at which every copy issued before it has landed.
// A half block is four steps of 16 inputs.  A step reads its rows and decodes its
// weights while the matrix cores run the step before it, one product, four
// vector instructions, one LDS read in turn: 2 - 4 % less time than reading and
// decoding ahead of a step's products.
template <int MT>
__global__ __launch_bounds__(256, 2) void fused_f16_kernel(FusedArgs a, const uint16_t* x16, const int32_t* rowinfo,
                                                           const Lost* lost, int tiles_n, int group_m) {
  constexpr int FX_BM = 32 * MT;                         // rows of a workgroup
  constexpr int FX_HALF = FX_BM * 128;                   // bytes of a 64-wide half block of the rows
  constexpr int FX_OFF_W = 2 * FX_HALF;
  constexpr int FX_SMEM = FX_OFF_W + 4 * 2 * FX_WBUF;    // 56 or 64 KB: two workgroups per CU
  static_assert(FX_SMEM <= 80 * 1024 && 4 * 32 * FX_STRIP * 4 <= FX_SMEM && FX_BM <= FX_MAX_BM, "LDS");
  __shared__ __align__(16) uint8_t smem[FX_SMEM];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 31, h = lane >> 5;

  RowTile rt;
  int tn;
  if (!find_tile(a, FX_BM, tiles_n, group_m, rt, tn)) return;
  const int64_t m0 = rt.m0, n_out = fused_n_out(a), K = a.K;
  const int KB = (int)(K / BLOCK_K), NH = 2 * KB;
  // Columns of the wave's two 32-column tiles: neighbours, or with a gated
  // epilogue both factors of the same outputs.
  const int64_t n0 = (int64_t)tn * (a.gated ? FX_BN / 2 : FX_BN) + wv * (a.gated ? 32 : 64);
  auto wcol = [&](int col) -> int64_t {                  // weight row of the wave's column 0 .. 63
    int64_t n = n0 + (a.gated ? (col & 31) : col);
    n = n < n_out ? n : n_out - 1;
    return a.gated && col >= 32 ? n + n_out : n;
  };

  // Rows: copy kk fills tile rows 32 kk + 8 wv .. + 7, lane l row l / 8 of them
  // and 16-byte position l % 8, which holds chunk (l % 8) ^ (row / 2 % 8): the
  // sixteen rows that one pass of a 16-byte read touches lie in different
  // banks.  Rows past the last one are padding of the workspace, never stored.
  // With a row index the four copies' rows lie anywhere in x16.
  const int crow = 8 * wv + (lane >> 3);
  const uint32_t chunk = (uint32_t)(((lane & 7) ^ ((crow >> 1) & 7)) << 4);
  uint32_t xoff[MT];
#pragma unroll
  for (int kk = 0; kk < MT; ++kk) {
    int64_t row = crow + 32 * kk;
    if (a.row_index) row = source_row(a, std::min<int64_t>(m0 + row, rt.mend - 1));
    xoff[kk] = (uint32_t)(row * K * 2) + chunk;
  }
  const __amdgpu_buffer_rsrc_t rx =
      a.row_index ? buf_rsrc(x16, (uint32_t)((a.x_rows + 1) * K * 2)) : buf_rsrc(x16 + m0 * K, (uint32_t)(FX_BM * K * 2));
  auto copy_rows = [&](int hs, int buf) {
#pragma unroll
    for (int kk = 0; kk < MT; ++kk) {
      const uint32_t xo = xoff[kk];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void*)(smem + buf * FX_HALF + (32 * kk + 8 * wv) * 128), 16, xo,
                                               (uint32_t)hs * 128u, 0, 0);
    }
  };
  // Info words of the rows, lane l's of rows l and l + 64 (past the last row: its own).
  auto load_info = [&](int row) {
    const int64_t m = std::min<int64_t>(m0 + std::min(row, FX_BM - 1), rt.mend - 1);
    return rowinfo[a.row_index ? source_row(a, m) : m];
  };
  const int info_lo = load_info(lane), info_hi = load_info(64 + lane);
  int aoff[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) aoff[t] = c * 128 + (((4 * h + t) ^ ((c >> 1) & 7)) << 4);

  // Codes: piece q holds columns 16 q .. + 15, lane l column l / 4 of them and
  // 16-byte position l % 4, which holds unit (l % 4) ^ (column / 4 % 4).
  const __amdgpu_buffer_rsrc_t rw = buf_rsrc(a.w + rt.expert * a.N * (K / 4), (uint32_t)(a.N * (K / 4)));
  const int unit = (lane & 3) ^ ((lane >> 4) & 3);
  auto code_off = [&](int q) { return (uint32_t)(wcol(16 * q + (lane >> 2)) * (K / 4)) + 16u * unit; };
  const uint32_t woff0 = code_off(0), woff1 = code_off(1), woff2 = code_off(2), woff3 = code_off(3);
  auto copy_codes = [&](int set, int q) {                // past the last set: that one again, never used
    const uint32_t wo = q == 0 ? woff0 : q == 1 ? woff1 : q == 2 ? woff2 : woff3;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rw, (lds_void*)(smem + FX_OFF_W + ((set & 1) * 4 + wv) * FX_WBUF + q * 1024), 16,
        wo - unit_back(set, KB, 2, unit), unit_start(set, KB, 2), 0, 0);
  };
  const uint8_t* const wbase = smem + FX_OFF_W + wv * FX_WBUF + c * 64 + 8 * h;
  auto read_codes = [&](int hs, q2_u32x2 (&w)[2]) {
    const int off = ((hs >> 2) & 1) * 4 * FX_WBUF + (((hs & 3) ^ ((c >> 2) & 3)) << 4);
#pragma unroll
    for (int j = 0; j < 2; ++j) w[j] = *reinterpret_cast<const q2_u32x2*>(wbase + off + j * 32 * 64);
  };

  // Scales of four blocks, a half-word each, from block min(4 q, KB - 4) on.
  const uint16_t* sp[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) sp[j] = a.s + (rt.expert * a.N + wcol(32 * j + c)) * KB;
  auto load_scales = [&](int q, uint64_t (&sc)[2]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) __builtin_memcpy(&sc[j], sp[j] + min(4 * q, KB - 4), 8);
  };

  q2_f32x16 acc[MT][2];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  q2_u32x2 w[2] = {};
  uint64_t scn[2];
  load_scales(0, scn);
#pragma unroll
  for (int q = 0; q < 4; ++q) copy_codes(0, q);
  copy_codes(1, 0);                                      // half-stage -1's piece
  copy_rows(0, 0);
  __builtin_amdgcn_s_waitcnt(0);
  read_codes(0, w);
  const uint64_t wide_lo = __builtin_amdgcn_ballot_w64((info_lo & ROW_WIDE) != 0);
  const uint64_t wide_hi = __builtin_amdgcn_ballot_w64((info_hi & ROW_WIDE) != 0);
  const uint64_t lost_lo = __builtin_amdgcn_ballot_w64((info_lo & ROW_LOST) != 0);
  const uint64_t lost_hi = __builtin_amdgcn_ballot_w64((info_hi & ROW_LOST) != 0);
  if ((wide_lo | wide_hi) == 0) {
    // Operands of a step and of the one before it, whose products are still to come:
    // zeros at first.
    q2_u32x4 av[2][MT], bf[2][2];
#pragma unroll
    for (int i = 0; i < MT; ++i) av[1][i] = q2_u32x4{0u, 0u, 0u, 0u};
    bf[1][0] = bf[1][1] = q2_u32x4{0u, 0u, 0u, 0u};
    for (int quad = 0; 4 * quad < KB; ++quad) {
      const uint64_t sc[2] = {scn[0], scn[1]};
      load_scales(quad + 1, scn);                        // past the end: the last four again, never used
      const int b0 = min(4 * quad, KB - 4), bend = min(4 * quad + 4, KB);
      for (int blk = 4 * quad; blk < bend; ++blk) {
        const int sh = 16 * (blk - b0);
        const WTable tab[2] = {weight_table((uint16_t)(sc[0] >> sh)), weight_table((uint16_t)(sc[1] >> sh))};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int hs = 2 * blk + half;
          stage_barrier<0>();
          copy_codes((hs + 1) / 4 + 1, (hs + 1) & 3);
          copy_rows(hs + 1 < NH ? hs + 1 : NH - 1, half ^ 1);      // past the end: the last one again, never read
          const uint8_t* st = smem + half * FX_HALF;
          q2_u32x2 wn[2];
#define Q2_STEP(T)                                                                                     \
  {                                                                                                    \
    constexpr int P = (T) & 1;                                                                         \
    _Pragma("unroll") for (int i = 0; i < MT; ++i)                                                     \
        av[P][i] = *reinterpret_cast<const q2_u32x4*>(st + i * 4096 + aoff[T]);                        \
    if ((T) == 1) read_codes(hs + 1, wn);                                                              \
    bf[P][0] = decode_step<T>(w[0], tab[0]);                                                           \
    bf[P][1] = decode_step<T>(w[1], tab[1]);                                                           \
    _Pragma("unroll") for (int i = 0; i < MT; ++i)                                                     \
        _Pragma("unroll") for (int j = 0; j < 2; ++j)                                                  \
            acc[i][j] = mfma32(av[P ^ 1][i], bf[P ^ 1][j], acc[i][j]);                                 \
    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);       /* LDS reads */                           \
    _Pragma("unroll") for (int i = 0; i < 2 * MT; ++i) {                                               \
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);     /* product */                             \
      __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);     /* decode */                              \
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                                               \
    }                                                                                                  \
    __builtin_amdgcn_sched_barrier(0);                                                                 \
  }
      Q2_STEP(0) Q2_STEP(1) Q2_STEP(2) Q2_STEP(3)
#undef Q2_STEP
          w[0] = wn[0];
          w[1] = wn[1];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = mfma32(av[1][i], bf[1][j], acc[i][j]);
  } else {
    // A tile with a wide row: all its rows as bf16, the others' f16 values exactly, in
    // the same order of steps; twice the products, four times the vector instructions.
    // M = 1536, K = 4096, N = 12288: 270 us for 141 when every tile holds a wide row,
    // 198 when one row of tiles does (first in its CU, as it ends last, and spread over
    // the CUs by find_tile's order: 252 without either); M = 4093, K = 12288, N = 4096
    // with rank 32: 732 for 392.
    __builtin_amdgcn_s_setprio(3);
    uint32_t kept[MT];                                   // all ones where row 32 i + c is bf16 already; a branch would cost more
#pragma unroll
    for (int i = 0; i < MT; ++i) kept[i] = 0u - ((uint32_t)((i < 2 ? wide_lo : wide_hi) >> (32 * (i & 1))) >> c & 1u);
    q2_u32x4 av[2][MT], bh[2][2], bl[2][2];
#pragma unroll
    for (int i = 0; i < MT; ++i) av[1][i] = q2_u32x4{0u, 0u, 0u, 0u};
    bh[1][0] = bh[1][1] = bl[1][0] = bl[1][1] = q2_u32x4{0u, 0u, 0u, 0u};
    for (int quad = 0; 4 * quad < KB; ++quad) {
      const uint64_t sc[2] = {scn[0], scn[1]};
      load_scales(quad + 1, scn);                        // past the end: the last four again, never used
      const int b0 = min(4 * quad, KB - 4), bend = min(4 * quad + 4, KB);
      for (int blk = 4 * quad; blk < bend; ++blk) {
        const int sh = 16 * (blk - b0);
        WTable hi[2], lo[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) weight_tables_bf16((uint16_t)(sc[j] >> sh), hi[j], lo[j]);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int hs = 2 * blk + half;
          stage_barrier<0>();
          copy_codes((hs + 1) / 4 + 1, (hs + 1) & 3);
          copy_rows(hs + 1 < NH ? hs + 1 : NH - 1, half ^ 1);      // past the end: the last one again, never read
          const uint8_t* st = smem + half * FX_HALF;
          q2_u32x2 wn[2];
#define Q2_STEP(T)                                                                                     \
  {                                                                                                    \
    constexpr int P = (T) & 1;                                                                         \
    if ((T) == 1) read_codes(hs + 1, wn);                                                              \
    _Pragma("unroll") for (int i = 0; i < MT; ++i) {                                                   \
      av[P][i] = *reinterpret_cast<const q2_u32x4*>(st + i * 4096 + aoff[T]);                          \
      _Pragma("unroll") for (int d = 0; d < 4; ++d)                                                    \
          av[P][i][d] = (av[P][i][d] & kept[i]) | (f16x2_bf16_hi(av[P][i][d]) & ~kept[i]);             \
    }                                                                                                  \
    _Pragma("unroll") for (int j = 0; j < 2; ++j) {                                                    \
      bh[P][j] = decode_step<T>(w[j], hi[j]);                                                          \
      bl[P][j] = decode_step<T>(w[j], lo[j]);                                                          \
    }                                                                                                  \
    _Pragma("unroll") for (int i = 0; i < MT; ++i)                                                     \
        _Pragma("unroll") for (int j = 0; j < 2; ++j)                                                  \
            acc[i][j] = mfma32_bf16(av[P ^ 1][i], bh[P ^ 1][j], acc[i][j]);                            \
    _Pragma("unroll") for (int i = 0; i < MT; ++i)                                                     \
        _Pragma("unroll") for (int j = 0; j < 2; ++j)                                                  \
            acc[i][j] = mfma32_bf16(av[P ^ 1][i], bl[P ^ 1][j], acc[i][j]);                            \
    __builtin_amdgcn_sched_group_barrier(0x100, MT + 2, 0);  /* LDS reads */                           \
    _Pragma("unroll") for (int i = 0; i < 4 * MT; ++i) {                                               \
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);     /* product */                             \
      __builtin_amdgcn_sched_group_barrier(0x002, 7, 0);     /* conversion and decode */               \
    }                                                                                                  \
    __builtin_amdgcn_sched_barrier(0);                                                                 \
  }
          Q2_STEP(0) Q2_STEP(1) Q2_STEP(2) Q2_STEP(3)
#undef Q2_STEP
          w[0] = wn[0];
          w[1] = wn[1];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        acc[i][j] = mfma32_bf16(av[1][i], bh[1][j], acc[i][j]);
        acc[i][j] = mfma32_bf16(av[1][i], bl[1][j], acc[i][j]);
      }
    __builtin_amdgcn_s_setprio(0);
  }
  __builtin_amdgcn_s_waitcnt(0);                         // no copy may still write this workgroup's LDS
  __syncthreads();

  // The rows' powers of two: element 4 q + e of a tile is row 8 q + 4 h + e.
  int* const exps = reinterpret_cast<int*>(smem);
  if (tid < FX_BM) exps[tid] = (wv == 0 ? info_lo : info_hi) >> 2;        // row 64 wv + lane
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int s = exps[32 * i + 8 * q + 4 * h + e];
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j][4 * q + e] = __builtin_amdgcn_ldexpf(acc[i][j][4 * q + e], s);
      }
  __syncthreads();                                       // read before the strips overwrite them

  if (a.r > 0) {
    const int r8 = (a.r + 7) & ~7;
    for (int k0 = 0; k0 < r8; k0 += 16) {
      const int q0 = k0 + 8 * h;
      BranchB bq[2];
      q2_u32x4 aq[MT][2];
#pragma unroll
      for (int j = 0; j < 2; ++j) bq[j] = branch_bfrag(a, wcol(32 * j + c), q0);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int l = 0; l < 2; ++l) aq[i][l] = branch_afrag(a, m0 + 32 * i + c, q0, l != 0);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          acc[i][j] = mfma32_bf16(aq[i][0], bq[j].hi, acc[i][j]);
          acc[i][j] = mfma32_bf16(aq[i][0], bq[j].lo, acc[i][j]);
          acc[i][j] = mfma32_bf16(aq[i][1], bq[j].hi, acc[i][j]);
        }
    }
  }

  // Out through a strip of 32 rows x 64 columns per wave.
  const float* bias = a.bias ? a.bias + rt.expert * a.N : nullptr;
  float* strip = reinterpret_cast<float*>(smem) + wv * 32 * FX_STRIP;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        strip[(8 * (e >> 2) + 4 * h + (e & 3)) * FX_STRIP + 32 * j + c] = acc[i][j][e];
    __builtin_amdgcn_wave_barrier();
    const int rows = (int)std::min<int64_t>(rt.mend - m0 - 32 * i, 32);
    // Remainders of rows that lost something in one element; lane l's column is l.
    // Nothing to see with one such row (M = 1536, K = 4096, N = 12288: 152 us), 251 us
    // with every row: 128 cache lines of codes and scales for a wave and row, whatever
    // the order of the loads.
    for (uint32_t left = (uint32_t)((i < 2 ? lost_lo : lost_hi) >> (32 * (i & 1))); left != 0; left &= left - 1) {
      const int row = __builtin_ctz(left);
      if (row >= rows) break;
      const int64_t m = m0 + 32 * i + row;
      const Lost l = lost[a.row_index ? source_row(a, m) : m];
      const int64_t wr = rt.expert * a.N + wcol(lane);
      const int code = a.w[wr * (K / 4) + (l.k >> 2)] >> (2 * (l.k & 3)) & 3;
      const float w = (float)(code - 1) * f16_to_f32(a.s[wr * KB + l.k / BLOCK_K]);
      strip[row * FX_STRIP + lane] = __builtin_fmaf(l.r, w, strip[row * FX_STRIP + lane]);
    }
    __builtin_amdgcn_wave_barrier();
    store_strip(a, bias, n_out, strip, FX_STRIP, 32, a.gated ? 32 : 64, m0 + 32 * i, rows, n0, lane);
    __builtin_amdgcn_wave_barrier();
  }
}

// ============================================================================
// launch
// ============================================================================
static size_t pad256(size_t v) { return (v + 255) & ~(size_t)255; }

// `rows` rows of x, their info words and what they lost.  The last tile's rows run up
// to FX_MAX_BM - 1 past them, a row index needs one row of zeros behind them.
static size_t x16_bytes(int64_t rows, int64_t K) { return pad256((size_t)(rows + FX_MAX_BM) * (size_t)K * 2); }
static size_t info_bytes(int64_t rows) { return pad256((size_t)(rows + FX_MAX_BM) * 4); }
size_t f16_workspace_bytes(int64_t rows, int64_t K) {
  return x16_bytes(rows, K) + info_bytes(rows) + pad256((size_t)rows * sizeof(Lost));
}

// Rows of x are addressed with 32 bits from a tile's first row, and with a row
// index from the first row of x; codes from an expert's weight.
bool fused_f16_takes(int64_t rows, int64_t N, int64_t K) {
  return K >= 4 * BLOCK_K && K <= (1 << 22) && N <= ((int64_t)1 << 33) / K && rows <= ((int64_t)1 << 30) / K;
}

// Rows of a workgroup.  The chip holds 512 workgroups, and one that has a CU for
// itself runs about twice as fast, so a launch takes its full rounds of 512 plus
// half a round for up to 256 more tiles.  A round of 96-row tiles takes 0.85 of
// one of 128-row tiles (each decode serves fewer rows).  Measured, 128 / 96 rows:
// 1536 rows K = 4096 N = 12288 182 / 157 us (576 and 768 tiles), N = 8192 121 /
// 108; 1024 rows N = 12288 116 / 139; 4093 rows K = 12288 N = 4096 371 / 417.
// Groups of rows, whose tiles are not known here: 128; both were within 2 %.
static int rows_per_tile(const FusedArgs& a, int64_t cols) {
  if (a.offsets) return 128;
  auto rounds = [&](int64_t bm) {
    const int64_t tiles = ((a.M + bm - 1) / bm) * ((fused_n_out(a) + cols - 1) / cols), rest = tiles % 512;
    return (double)(tiles / 512) + (rest == 0 ? 0.0 : rest <= 256 ? 0.5 : 1.0);
  };
  return 0.85 * rounds(96) < rounds(128) ? 96 : 128;
}

hipError_t launch_fused_f16(const FusedArgs& a, void* ws, hipStream_t stream) {
  const int64_t rows = a.x_rows, K = a.K;
  uint8_t* const w8 = static_cast<uint8_t*>(ws);
  uint16_t* x16 = reinterpret_cast<uint16_t*>(w8);
  int32_t* rowinfo = reinterpret_cast<int32_t*>(w8 + x16_bytes(a.M, K));
  Lost* lost = reinterpret_cast<Lost*>(w8 + x16_bytes(a.M, K) + info_bytes(a.M));
  const int64_t cols = a.gated ? FX_BN / 2 : FX_BN;
  const int bm = rows_per_tile(a, cols);
  const int64_t tiles_n = (fused_n_out(a) + cols - 1) / cols, slots = max_row_tiles(a, bm);
  if (tiles_n > 0x7fffffff || slots > 0x7fffffff / tiles_n) return hipErrorInvalidValue;
  if (a.r > 0 && a.r <= XA_MAX_RANK) {
    const dim3 grid((unsigned)((rows + 15) / 16)), block(64 * XA_WAVES);
#define Q2_XA(CT)                                                                                                  \
  hipLaunchKernelGGL((x_to_f16_branch_kernel<CT>), grid, block, 0, stream, a.x, a.lr_a, x16, rowinfo, lost, a.lr_t, \
                     rows, K, a.r)
    if (a.r <= 16) Q2_XA(1);
    else if (a.r <= 32) Q2_XA(2);
    else Q2_XA(4);
#undef Q2_XA
  } else {
    const dim3 grid((unsigned)(rows / CV_ROWS + 1)), block(64 * CV_ROWS);
#define Q2_CV(NCH) hipLaunchKernelGGL((x_to_f16_kernel<NCH>), grid, block, 0, stream, a.x, x16, rowinfo, lost, rows, K)
    if (K <= 2048) Q2_CV(2);
    else if (K <= 4096) Q2_CV(4);
    else if (K <= 12288) Q2_CV(12);
    else Q2_CV(0);
#undef Q2_CV
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int group_m = tile_group_rows(slots, tiles_n, 2.0 * bm * (double)K, (double)FX_BN * K * 0.265625, 64);
  const dim3 grid = grid_of(slots * tiles_n);
#define Q2_FX(MT) \
  hipLaunchKernelGGL((fused_f16_kernel<MT>), grid, dim3(256), 0, stream, a, x16, rowinfo, lost, (int)tiles_n, group_m)
  if (bm == 96) Q2_FX(3);
  else Q2_FX(4);
#undef Q2_FX
  return hipGetLastError();
}

}  // namespace q2dev
