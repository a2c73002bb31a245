// q2_route.hip - the experts' router (top-k choice, softmax weights, row plan)
// and the combination of the experts' rows.
#include "q2_fused.h"
#include <algorithm>

namespace q2dev {

// ============================================================================
// Router
// ============================================================================
// A workgroup of sixteen waves takes 64 tokens.  Logits are held as
// order-preserving bits, 0 for a masked expert or one already chosen, and k steps
// each take the largest and, among equal ones, the lowest expert.  Up to 16
// choices among up to 256 experts, sixteen lanes work on a token (choose16): a
// step takes 65 vector instructions for four tokens at E = 128, where a wave per
// token (choose: lane l holds every 64th logit, a maximum over the lanes by six
// data-parallel-primitive moves and a ballot of the lanes that hold it) takes 45
// for one.  The steps' instructions bound the kernel, not the logits' 4 MB.
//
// Row plan: each token chooses an expert at most once, so 64 tokens' choices
// are one 64-bit mask per expert, and a choice's place among the rows of its
// expert is the number of mask bits below its token.  The rows of earlier
// workgroups and experts come from the workgroups' counts: up to 64 tokens one
// launch has everything; beyond, the first launch leaves its counts in the
// workspace and every workgroup of the second adds them up.  That sum is
// (workgroups)^2, so past 1024 workgroups each takes several chunks of 64
// tokens instead.  Integer counts: the plan is exact, the same on every run.
// T = 16384, E = 128, k = 8, bf16 logits: choice 9.5 us (14.8 with a wave per
// token), plan 6.2; T = 4096, E = 256 both 19 us (23); one token, E = 64: 3.7.
constexpr int RT_TOK = 64, RT_THREADS = 1024, RT_WAVES = RT_THREADS / 64;
constexpr int RT_GROUPS = 1024, RT_CHUNKS = 1023;       // workgroups, while a workgroup's chunks are at most so many
static_assert(RT_TOK * RT_CHUNKS <= 0xFFFF, "a workgroup's count of an expert has 16 bits");

constexpr int route_pad(int64_t E) { return (int)((E + 1) & ~(int64_t)1); }     // counts per workgroup, u16 pairs
static int route_chunks(int64_t T) {
  return (int)std::min<int64_t>((T + RT_TOK * RT_GROUPS - 1) / (RT_TOK * RT_GROUPS), RT_CHUNKS);
}
static int64_t route_groups(int64_t T) {
  const int64_t per = (int64_t)RT_TOK * route_chunks(T);
  return (T + per - 1) / per;
}

__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);          // -0 counts as +0
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float from_order_bits(uint32_t o) {
  return __builtin_bit_cast(float, o ^ ((o >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// Logits of experts e0 + step i of a token as order-preserving bits; 0, below
// every other, for masked experts and past the last one.
template <int NE>
__device__ __forceinline__ void load_keys(const void* logits, int bf16, int64_t t, int E, int e0, int step,
                                          uint32_t (&key)[NE]) {
  float v[NE];
  if (bf16) {
    const uint16_t* p = static_cast<const uint16_t*>(logits) + t * E;
#pragma unroll
    for (int i = 0; i < NE; ++i) v[i] = bf16_to_f32(p[min(e0 + step * i, E - 1)]);
  } else {
    const float* p = static_cast<const float*>(logits) + t * E;
#pragma unroll
    for (int i = 0; i < NE; ++i) v[i] = p[min(e0 + step * i, E - 1)];
  }
#pragma unroll
  for (int i = 0; i < NE; ++i) key[i] = e0 + step * i < E && v[i] > -__builtin_inff() ? order_bits(v[i]) : 0u;
}

// v from the lane that CTRL names, 0 where there is none.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp0(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
// Largest v (0 at least) and sum over the 64 lanes: shifts by 1, 2, 4, 8 within
// rows of 16, then rows 0, 2 onto 1, 3 and the lower half onto the upper.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, dpp0<0x111, 0xF>(v));
  v = max(v, dpp0<0x112, 0xF>(v));
  v = max(v, dpp0<0x114, 0xF>(v));
  v = max(v, dpp0<0x118, 0xF>(v));
  v = max(v, dpp0<0x142, 0xA>(v));
  v = max(v, dpp0<0x143, 0xC>(v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __builtin_bit_cast(float, dpp0<CTRL, ROWS>(__builtin_bit_cast(uint32_t, v)));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = add_dpp<0x111, 0xF>(v);
  v = add_dpp<0x112, 0xF>(v);
  v = add_dpp<0x114, 0xF>(v);
  v = add_dpp<0x118, 0xF>(v);
  v = add_dpp<0x142, 0xA>(v);
  v = add_dpp<0x143, 0xC>(v);
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// exp(v - top) of a logit, 1 for the largest itself (also when that is +inf).
__device__ __forceinline__ float route_exp(float v, float top) { return v == top ? 1.0f : __expf(v - top); }

// Choice and weights of one token: lane j < k returns choice j (-1 for none).
template <int NE>
__device__ __forceinline__ void choose(const void* logits, int bf16, int64_t t, int E, int k, int renorm, int lane,
                                       int& ex, float& wt) {
  uint32_t key[NE];
  load_keys<NE>(logits, bf16, t, E, lane, 64, key);
  ex = -1;
  float mine = 0.f, top = 0.f, total = 0.f;
  for (int j = 0; j < k; ++j) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < NE; ++i) m = max(m, key[i]);
    m = wave_max(m);
    if (m == 0) break;                                   // nothing left but masked experts
    const float v = from_order_bits(m);
    if (j == 0) {
      top = v;
      if (!renorm) {                                     // every unmasked expert, before any key is taken out
#pragma unroll
        for (int i = 0; i < NE; ++i)
          if (key[i] != 0) total += route_exp(from_order_bits(key[i]), top);
        total = wave_sum(total);
      }
    }
    const float p = route_exp(v, top);
    if (renorm) total += p;                              // largest first
    int e = -1;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const uint64_t b = __builtin_amdgcn_ballot_w64(key[i] == m);
      if (e < 0 && b != 0) {
        const int l = __builtin_ctzll(b);
        e = 64 * i + l;
        if (lane == l) key[i] = 0;
      }
    }
    if (lane == j) {
      ex = e;
      mine = p;
    }
  }
  wt = ex >= 0 ? mine / total : 0.f;
}

// Up to 16 choices among up to 256 experts: sixteen lanes per token, four tokens
// of a wave together.  Lane l of a token holds experts NK l .. NK l + NK - 1, so
// the lowest expert among equal logits is in the lowest lane.  Rotations within
// the sixteen lanes leave the maximum (and the sum, whose four additions are the
// same pairs in every lane) in all of them.
template <int N>
__device__ __forceinline__ uint32_t ror16(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 | N, 0xF, 0xF, true);
}
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = max(v, ror16<8>(v));
  v = max(v, ror16<4>(v));
  v = max(v, ror16<2>(v));
  return max(v, ror16<1>(v));
}
__device__ __forceinline__ float sum16(float v) {
  auto add = [](float a, uint32_t b) { return a + __builtin_bit_cast(float, b); };
  v = add(v, ror16<8>(__builtin_bit_cast(uint32_t, v)));
  v = add(v, ror16<4>(__builtin_bit_cast(uint32_t, v)));
  v = add(v, ror16<2>(__builtin_bit_cast(uint32_t, v)));
  return add(v, ror16<1>(__builtin_bit_cast(uint32_t, v)));
}

// Lane l < k of the token's sixteen returns choice l.
template <int NK>
__device__ __forceinline__ void choose16(const void* logits, int bf16, int64_t t, int E, int k, int renorm, int l,
                                         int& ex, float& wt) {
  uint32_t key[NK];
  load_keys<NK>(logits, bf16, t, E, NK * l, 1, key);
  ex = -1;
  float mine = 0.f, top = 0.f, total = 0.f;
  for (int j = 0; j < k; ++j) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < NK; ++i) m = max(m, key[i]);
    m = max16(m);
    if (__builtin_amdgcn_ballot_w64(m != 0) == 0) break; // nothing left in any of the four tokens
    const float v = from_order_bits(m);
    if (j == 0) {
      top = v;
      if (!renorm) {
#pragma unroll
        for (int i = 0; i < NK; ++i)
          if (key[i] != 0) total += route_exp(from_order_bits(key[i]), top);
        total = sum16(total);
      }
    }
    const float p = m != 0 ? route_exp(v, top) : 0.f;
    if (renorm) total += p;                              // largest first
    // the complement of the lowest expert that holds m; a token with none left has every key 0
    uint32_t at = 0;
#pragma unroll
    for (int i = NK - 1; i >= 0; --i) at = key[i] == m ? ~(uint32_t)(NK * l + i) : at;
    const int e = (int)~max16(at), own = e - NK * l;
#pragma unroll
    for (int i = 0; i < NK; ++i) key[i] = i == own ? 0u : key[i];
    if (l == j && m != 0) {
      ex = e;
      mine = p;
    }
  }
  wt = ex >= 0 ? mine / total : 0.f;
}

// Offsets of the experts from their totals in tot[] (replaced), by one wave.
__device__ __forceinline__ void scan_experts(int* tot, int E, int lane) {
  int run = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    const int v = e < E ? tot[e] : 0;
    int s = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(s, d);
      if (lane >= d) s += o;
    }
    if (e < E) tot[e] = run + s - v;
    run += __shfl(s, 63);
  }
  if (lane == 0) tot[E] = run;
}

template <int NE, int LANES, bool ONE>
__global__ __launch_bounds__(RT_THREADS) void route_choose_kernel(const void* logits, int bf16, int64_t T, int E, int k,
                                                                  int renorm, int chunks, int32_t* expert,
                                                                  float* weight, int32_t* offsets, int32_t* row_token,
                                                                  int32_t* slot, uint16_t* counts, int pad) {
  __shared__ unsigned long long mask[LANES * NE];
  __shared__ int off[LANES * NE + 1];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t first = (int64_t)blockIdx.x * RT_TOK * chunks;
  if constexpr (!ONE)
    for (int e = threadIdx.x; e < E; e += RT_THREADS) off[e] = 0;
  int nt = 0;
  for (int ch = 0; ch < chunks; ++ch) {
    const int64_t t0 = first + (int64_t)ch * RT_TOK;
    nt = (int)std::min<int64_t>(T - t0, RT_TOK);
    for (int e = threadIdx.x; e < E; e += RT_THREADS) mask[e] = 0;
    __syncthreads();
    constexpr int AT_ONCE = 64 / LANES;                  // tokens of a wave
    const int l = lane % LANES;
    for (int i0 = wv * AT_ONCE; i0 < nt; i0 += RT_WAVES * AT_ONCE) {
      const int i = i0 + lane / LANES;
      const int64_t t = t0 + min(i, nt - 1);             // past the last token: the last one again, not stored
      int ex;
      float wt;
      if constexpr (LANES == 16) choose16<NE>(logits, bf16, t, E, k, renorm, l, ex, wt);
      else choose<NE>(logits, bf16, t, E, k, renorm, l, ex, wt);
      if (l < k && i < nt) {
        expert[t * k + l] = ex;
        weight[t * k + l] = wt;
        if (ex >= 0) atomicOr(&mask[ex], 1ull << i);
      }
    }
    __syncthreads();
    if constexpr (!ONE)
      for (int e = threadIdx.x; e < E; e += RT_THREADS) off[e] += __popcll(mask[e]);
  }
  if constexpr (!ONE) {
    for (int e = threadIdx.x; e < pad; e += RT_THREADS)   // off[e] was added up by this thread
      counts[(int64_t)blockIdx.x * pad + e] = e < E ? (uint16_t)off[e] : (uint16_t)0;
  } else {
    for (int e = threadIdx.x; e < E; e += RT_THREADS) off[e] = __popcll(mask[e]);
    __syncthreads();
    if (wv == 0) scan_experts(off, E, lane);
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += RT_THREADS) offsets[e] = off[e];
    for (int i = threadIdx.x; i < nt * k; i += RT_THREADS) {
      const int ex = expert[i];                          // written by this workgroup before the barrier
      const int tok = i / k;
      int row = -1;
      if (ex >= 0) {
        row = off[ex] + __popcll(mask[ex] & ((1ull << tok) - 1));
        row_token[row] = tok;
      }
      slot[i] = row;
      if (i >= off[E]) row_token[i] = -1;
    }
  }
}

// Second launch: workgroup b adds up the counts of all workgroups and of those
// before it, and places its tokens' choices.
__global__ __launch_bounds__(RT_THREADS) void route_place_kernel(const int32_t* expert, int64_t T, int E, int k,
                                                                 int chunks, const uint16_t* counts, int pad,
                                                                 int groups, int32_t* offsets, int32_t* row_token,
                                                                 int32_t* slot) {
  __shared__ unsigned long long mask[1024];
  __shared__ int tot[1025], before[1024];
  for (int e = threadIdx.x; e < E; e += RT_THREADS) {
    tot[e] = 0;
    before[e] = 0;
  }
  __syncthreads();
  // two experts' counts per load, the threads beyond one row of counts on further rows
  const int pairs = pad / 2, rows = RT_THREADS / pairs;
  if ((int)threadIdx.x < pairs * rows) {
    const int q = threadIdx.x % pairs, r0 = threadIdx.x / pairs;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(counts) + q;
    int all0 = 0, all1 = 0, pre0 = 0, pre1 = 0;
#pragma unroll 8
    for (int b = r0; b < groups; b += rows) {
      const uint32_t v = src[(int64_t)b * pairs];
      const int lo = v & 0xFFFF, hi = v >> 16;
      all0 += lo;
      all1 += hi;
      pre0 += b < (int)blockIdx.x ? lo : 0;
      pre1 += b < (int)blockIdx.x ? hi : 0;
    }
    if (all0) atomicAdd(&tot[2 * q], all0);              // counts past E are 0
    if (all1) atomicAdd(&tot[2 * q + 1], all1);
    if (pre0) atomicAdd(&before[2 * q], pre0);
    if (pre1) atomicAdd(&before[2 * q + 1], pre1);
  }
  __syncthreads();
  if (threadIdx.x < 64) scan_experts(tot, E, threadIdx.x);
  __syncthreads();
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= E; e += RT_THREADS) offsets[e] = tot[e];
  const int64_t first = (int64_t)blockIdx.x * RT_TOK * chunks;
  for (int ch = 0; ch < chunks; ++ch) {
    const int64_t t0 = first + (int64_t)ch * RT_TOK;
    const int nt = (int)std::max<int64_t>(std::min<int64_t>(T - t0, RT_TOK), 0);
    for (int e = threadIdx.x; e < E; e += RT_THREADS) mask[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < nt * k; i += RT_THREADS) {
      const int ex = expert[t0 * k + i];
      if (ex >= 0) atomicOr(&mask[ex], 1ull << (i / k));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nt * k; i += RT_THREADS) {
      const int64_t at = t0 * k + i;
      const int ex = expert[at], tok = i / k;
      int row = -1;
      if (ex >= 0) {
        row = tot[ex] + before[ex] + __popcll(mask[ex] & ((1ull << tok) - 1));
        row_token[row] = (int)(t0 + tok);
      }
      slot[at] = row;
      if (at >= tot[E]) row_token[at] = -1;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += RT_THREADS) before[e] += __popcll(mask[e]);
  }
}

__global__ __launch_bounds__(256) void route_empty_kernel(int32_t* offsets, int E) {
  for (int e = threadIdx.x; e <= E; e += 256) offsets[e] = 0;
}

size_t route_workspace_bytes(int64_t T, int64_t E) {
  return T > RT_TOK ? ((size_t)route_groups(T) * route_pad(E) * 2 + 255) & ~(size_t)255 : 0;
}

template <int NE, int LANES>
static hipError_t run_route(const void* logits, int bf16, int64_t T, int E, int k, int renorm, int32_t* expert,
                            float* weight, int32_t* offsets, int32_t* row_token, int32_t* slot, uint16_t* counts,
                            hipStream_t stream) {
  const int pad = route_pad(E);
  if (T <= RT_TOK) {
    hipLaunchKernelGGL((route_choose_kernel<NE, LANES, true>), dim3(1), dim3(RT_THREADS), 0, stream, logits, bf16, T, E, k,
                       renorm, 1, expert, weight, offsets, row_token, slot, counts, pad);
    return hipGetLastError();
  }
  const int chunks = route_chunks(T), groups = (int)route_groups(T);
  hipLaunchKernelGGL((route_choose_kernel<NE, LANES, false>), dim3(groups), dim3(RT_THREADS), 0, stream, logits, bf16, T, E,
                     k, renorm, chunks, expert, weight, offsets, row_token, slot, counts, pad);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(route_place_kernel, dim3(groups), dim3(RT_THREADS), 0, stream, expert, T, E, k, chunks, counts,
                     pad, groups, offsets, row_token, slot);
  return hipGetLastError();
}

hipError_t launch_route(const void* logits, int logits_bf16, int64_t T, int64_t E, int k, int renorm, int32_t* expert,
                        float* weight, int32_t* offsets, int32_t* row_token, int32_t* slot, void* ws,
                        hipStream_t stream) {
  if (T == 0) {
    hipLaunchKernelGGL(route_empty_kernel, dim3(1), dim3(256), 0, stream, offsets, (int)E);
    return hipGetLastError();
  }
  uint16_t* counts = static_cast<uint16_t*>(ws);
  const int n = (int)E;
#define Q2_ROUTE(NE, LANES)                                                                                          \
  return run_route<NE, LANES>(logits, logits_bf16, T, n, k, renorm, expert, weight, offsets, row_token, slot, counts, \
                              stream)
  if (k <= 16 && n <= 64) Q2_ROUTE(4, 16);
  if (k <= 16 && n <= 128) Q2_ROUTE(8, 16);
  if (k <= 16 && n <= 256) Q2_ROUTE(16, 16);
  if (n <= 64) Q2_ROUTE(1, 64);
  if (n <= 128) Q2_ROUTE(2, 64);
  if (n <= 256) Q2_ROUTE(4, 64);
  if (n <= 512) Q2_ROUTE(8, 64);
  Q2_ROUTE(16, 64);
#undef Q2_ROUTE
}

// ============================================================================
// Combination
// ============================================================================
// Eight columns per thread, a token's chunks over consecutive workgroups.  Bound by
// memory: 8192 tokens, four rows of 2048 in bf16 each, 41 us, 202 MB at 4.9 TB/s (a
// copy of 1 GiB: 5.2).
constexpr int CB_COLS = 8;

__device__ __forceinline__ Eight load8(const void* p, int64_t i, int bf16) {
  return raw_floats(load8raw(p, i, bf16), bf16);
}

__global__ __launch_bounds__(256) void combine_kernel(const void* z, int z_bf16, int64_t R, const int32_t* slot,
                                                      const float* weight, const void* residual, int res_bf16, void* y,
                                                      int out_bf16, int64_t T, int k, int64_t N, int64_t chunks) {
  const int64_t id = (int64_t)workgroup_id() * 256 + threadIdx.x;
  const int64_t t = id / chunks;
  if (t >= T) return;
  const int64_t n0 = (id - t * chunks) * CB_COLS;
  float acc[CB_COLS] = {};
  for (int j = 0; j < k; ++j) {
    const int s = slot[t * k + j];
    if (s < 0 || s >= R) continue;
    const float w = weight[t * k + j];
    const Eight v = load8(z, (int64_t)s * N + n0, z_bf16);
#pragma unroll
    for (int d = 0; d < CB_COLS; ++d) acc[d] = __builtin_fmaf(w, v.v[d], acc[d]);
  }
  const int64_t at = t * N + n0;
  if (residual) {
    const Eight v = load8(residual, at, res_bf16);
#pragma unroll
    for (int d = 0; d < CB_COLS; ++d) acc[d] += v.v[d];
  }
  if (out_bf16) {
    q2_u32x4 r;
#pragma unroll
    for (int d = 0; d < 4; ++d) r[d] = (uint32_t)to_bf16(acc[2 * d]) | ((uint32_t)to_bf16(acc[2 * d + 1]) << 16);
    *reinterpret_cast<q2_u32x4*>(static_cast<uint16_t*>(y) + at) = r;
  } else {
    q2_f32x4* q = reinterpret_cast<q2_f32x4*>(static_cast<float*>(y) + at);
    q[0] = q2_f32x4{acc[0], acc[1], acc[2], acc[3]};
    q[1] = q2_f32x4{acc[4], acc[5], acc[6], acc[7]};
  }
}

// Rows that are not whole 16-byte pieces: a wave per token and 256 W columns, lane
// l holding W neighbours at W l and every 64 W columns on, so that a load's lanes
// read neighbours.  Pairs (W = 2) where the rows allow them: 3081 tokens, six bf16
// rows of 3586 65 us, one by one 89; f32 rows 60 us, 287 MB at 4.8 TB/s.
constexpr int CR_STEPS = 4, CR_WAVES = 4;

template <int W>
struct RaggedCols {
  float v[CR_STEPS * W];
};
template <int W>
__device__ __forceinline__ RaggedCols<W> load_ragged(const void* p, int64_t i, int bf16, int64_t left) {
  typedef uint16_t half_w __attribute__((ext_vector_type(W)));
  typedef float float_w __attribute__((ext_vector_type(W)));
  RaggedCols<W> r = {};
  if (bf16) {
    const uint16_t* q = static_cast<const uint16_t*>(p) + i;
#pragma unroll
    for (int d = 0; d < CR_STEPS; ++d)
      if (64 * W * d < left) {
        const half_w t = *reinterpret_cast<const half_w*>(q + 64 * W * d);
#pragma unroll
        for (int e = 0; e < W; ++e) r.v[W * d + e] = bf16_to_f32(t[e]);
      }
  } else {
    const float* q = static_cast<const float*>(p) + i;
#pragma unroll
    for (int d = 0; d < CR_STEPS; ++d)
      if (64 * W * d < left) {
        const float_w t = *reinterpret_cast<const float_w*>(q + 64 * W * d);
#pragma unroll
        for (int e = 0; e < W; ++e) r.v[W * d + e] = t[e];
      }
  }
  return r;
}

template <int W>
__global__ __launch_bounds__(64 * CR_WAVES) void combine_ragged_kernel(const void* z, int z_bf16, int64_t R,
                                                                       const int32_t* slot, const float* weight,
                                                                       const void* residual, int res_bf16, void* y,
                                                                       int out_bf16, int64_t T, int k, int64_t N,
                                                                       int64_t chunks) {
  typedef uint16_t half_w __attribute__((ext_vector_type(W)));
  typedef float float_w __attribute__((ext_vector_type(W)));
  const int64_t id = (int64_t)workgroup_id() * CR_WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = id / chunks;
  if (t >= T) return;
  const int64_t n = (id - t * chunks) * (64 * W * CR_STEPS) + (threadIdx.x & 63) * W, left = N - n;
  RaggedCols<W> acc = {};
  for (int j = 0; j < k; ++j) {
    const int s = slot[t * k + j];
    if (s < 0 || s >= R) continue;
    const float w = weight[t * k + j];
    const RaggedCols<W> v = load_ragged<W>(z, (int64_t)s * N + n, z_bf16, left);
#pragma unroll
    for (int d = 0; d < CR_STEPS * W; ++d) acc.v[d] = __builtin_fmaf(w, v.v[d], acc.v[d]);
  }
  const int64_t at = t * N + n;
  if (residual) {
    const RaggedCols<W> v = load_ragged<W>(residual, at, res_bf16, left);
#pragma unroll
    for (int d = 0; d < CR_STEPS * W; ++d) acc.v[d] += v.v[d];
  }
#pragma unroll
  for (int d = 0; d < CR_STEPS; ++d) {
    if (64 * W * d >= left) continue;
    half_w h;
    float_w f;
#pragma unroll
    for (int e = 0; e < W; ++e) {
      f[e] = acc.v[W * d + e];
      h[e] = to_bf16(f[e]);
    }
    if (out_bf16) *reinterpret_cast<half_w*>(static_cast<uint16_t*>(y) + at + 64 * W * d) = h;
    else *reinterpret_cast<float_w*>(static_cast<float*>(y) + at + 64 * W * d) = f;
  }
}

hipError_t launch_combine(const void* z, int z_bf16, int64_t R, const int32_t* slot, const float* weight,
                          const void* residual, int res_bf16, void* y, int out_bf16, int64_t T, int k, int64_t N,
                          hipStream_t stream) {
  auto on = [](const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; };
  const bool vec = N % CB_COLS == 0 && on(z, 16) && on(residual, 16) && on(y, 16);
  const bool pairs = N % 2 == 0 && on(z, z_bf16 ? 4 : 8) && on(residual, res_bf16 ? 4 : 8) && on(y, out_bf16 ? 4 : 8);
  const int64_t wide = 64 * CR_STEPS * (pairs ? 2 : 1);
  const int64_t chunks = vec ? N / CB_COLS : (N + wide - 1) / wide;
  const int64_t per = vec ? 256 : CR_WAVES, blocks = (T * chunks + per - 1) / per;
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
#define Q2_COMBINE(KERNEL)                                                                                            \
  hipLaunchKernelGGL(KERNEL, grid_of(blocks), dim3(256), 0, stream, z, z_bf16, R, slot, weight, residual,      \
                     res_bf16, y, out_bf16, T, k, N, chunks)
  if (vec) Q2_COMBINE(combine_kernel);
  else if (pairs) Q2_COMBINE((combine_ragged_kernel<2>));
  else Q2_COMBINE((combine_ragged_kernel<1>));
#undef Q2_COMBINE
  return hipGetLastError();
}

}  // namespace q2dev
