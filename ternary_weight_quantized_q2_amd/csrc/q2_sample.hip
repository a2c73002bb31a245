// q2_sample.hip - a token drawn from each row of logits: temperature, min-p, top-k,
// top-p, and the inverse of the cumulative distribution at a given random number.
//
// Order: logits descending, equal ones by lower token; p_i = exp((l_i - best) / T).
// Every filter leaves the first tokens of that order, and the draw is the first token
// whose cumulative p exceeds u times the sum, so nothing is sorted: each of the three
// borders is the place where a cumulative count or sum reaches a target, found by a
// histogram over the logits' distance from the best one.
//
// A token's p is held as a whole number of 2^-S, S = 62 - ceil(log2 V) (at most 51),
// rounded once from 64-bit floating point.  Sums of whole numbers do not depend on
// their order, so a border that a random number comes close to is the same on every
// run; with 32-bit sums a hundred thousand tokens' borders would be off by as much as
// a per cent of a token's width.  A p below half a unit, 2^-46 at V = 2^17, is never drawn.
#include "q2_token.h"
#include <algorithm>

namespace q2dev {

constexpr int SM_THREADS = 1024, SM_WAVES = SM_THREADS / 64;
constexpr int SM_BUCKETS = 2048, SM_PER = SM_BUCKETS / SM_THREADS;
constexpr int SM_LIST = 256;                             // elements of a bucket that are compared with each other

__device__ __forceinline__ uint32_t logit_key(float v) { // order-preserving, 0 for a masked token
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);              // -0 counts as +0
  return v > -__builtin_inff() ? b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u) : 0u;
}
__device__ __forceinline__ float key_logit(uint32_t o) {
  return __builtin_bit_cast(float, o ^ ((o >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// f(logit, token) for the row's tokens, 16 bytes at a time between the first and the
// last aligned address.
template <class F>
__device__ __forceinline__ void each_logit(const void* row, int bf16, int V, F f) {
  const int size = bf16 ? 2 : 4, per = 16 / size;
  const int head = min(V, (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / size);
  const int body = (V - head) / per;
  auto one = [&](int i) {
    f(bf16 ? bf16_to_f32(static_cast<const uint16_t*>(row)[i]) : static_cast<const float*>(row)[i], i);
  };
  if ((int)threadIdx.x < head) one(threadIdx.x);
  const q2_u32x4* p = reinterpret_cast<const q2_u32x4*>(static_cast<const uint8_t*>(row) + head * size);
  for (int i = threadIdx.x; i < body; i += SM_THREADS) {
    const q2_u32x4 v = p[i];
    const int at = head + i * per;
    if (bf16) {
#pragma unroll
      for (int d = 0; d < 8; ++d)
        f(__builtin_bit_cast(float, (d & 1) ? v[d >> 1] & 0xFFFF0000u : v[d >> 1] << 16), at + d);
    } else {
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const uint32_t b = v[d];                         // a bit cast of the vector's element itself reads element 0
        f(__builtin_bit_cast(float, b), at + d);
      }
    }
  }
  const int tail = head + body * per + threadIdx.x;
  if (tail < V) one(tail);
}

struct SampleShared {
  uint64_t sum[2][SM_BUCKETS];                           // [0] over all tokens, [1] over a range of one bucket
  uint32_t count[2][SM_BUCKETS];
  uint64_t wsum[SM_WAVES];
  uint32_t wcount[SM_WAVES];
  uint64_t best, base_s, list_w[SM_LIST];
  uint32_t list[SM_LIST];
  uint32_t base_n, bucket, n, fill, lo, hi, key;
};

// What a row's tokens are measured by.
struct Measure {
  float best;
  uint32_t best_key;
  double inv_t, unit, min_p;                             // 1 / T, 2^S
  float per_logit;                                       // buckets per unit of the logit

  __device__ __forceinline__ double p(uint32_t key) const {
    if (key == best_key) return 1.0;
    const double d = ((double)best - (double)key_logit(key)) * inv_t;
    return d >= 0.0 ? exp(-d) : 0.0;                     // inf * 0 is NaN: no probability
  }
  // Whole number of units; 0 for a token that is masked, below min-p or too unlikely.
  __device__ __forceinline__ uint64_t weight(uint32_t key) const {
    if (key == 0) return 0;
    const double q = p(key);
    if (!(q >= min_p)) return 0;
    return __builtin_bit_cast(uint64_t, q * unit + 0x1p52) - __builtin_bit_cast(uint64_t, 0x1p52);
  }
  // Does not fall as the logit falls: subtraction and product round monotonically.
  __device__ __forceinline__ int bucket(uint32_t key) const {
    if (key == best_key) return 0;
    const float t = (best - key_logit(key)) * per_logit;
    return t < (float)(SM_BUCKETS - 1) ? (int)t : SM_BUCKETS - 1;
  }
};

// Exclusive sums over the buckets before this thread's (SM_PER each), and the totals.
__device__ __forceinline__ void scan_buckets(SampleShared& s, int h, uint64_t& before_s, uint32_t& before_n,
                                             uint64_t& total_s, uint32_t& total_n) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  uint64_t vs = 0;
  uint32_t vn = 0;
#pragma unroll
  for (int i = 0; i < SM_PER; ++i) vs += s.sum[h][SM_PER * threadIdx.x + i], vn += s.count[h][SM_PER * threadIdx.x + i];
  uint64_t is = vs;
  uint32_t in = vn;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t os = __shfl_up(is, d);
    const uint32_t on = __shfl_up(in, d);
    if (lane >= d) is += os, in += on;
  }
  __syncthreads();                                       // the waves' sums of an earlier scan are read
  if (lane == 63) s.wsum[wv] = is, s.wcount[wv] = in;
  __syncthreads();
  before_s = is - vs;
  before_n = in - vn;
  total_s = 0;
  total_n = 0;
  for (int w = 0; w < SM_WAVES; ++w) {
    if (w < wv) before_s += s.wsum[w], before_n += s.wcount[w];
    total_s += s.wsum[w];
    total_n += s.wcount[w];
  }
}

// The first place of the order where the cumulative count (by_count) or weight reaches
// target, which lies between 1 and the total: the logit's key, what lies before tokens
// of that logit, and how many of these it takes.
struct Place {
  uint32_t key, before_n, ties;
  uint64_t before_s, w;
};

__device__ Place locate(SampleShared& s, const Measure& me, const void* row, int bf16, int V, bool by_count,
                        uint64_t target) {
  Place p;
  uint32_t lo = 1, hi = 0xFFFFFFFFu;                     // keys of the range
  int bucket = -1;
  uint64_t base_s = 0;
  uint32_t base_n = 0;
  for (int h = 0;; h = 1) {
    uint64_t bs, ts;
    uint32_t bn, tn;
    scan_buckets(s, h, bs, bn, ts, tn);
    bs += base_s;
    bn += base_n;
#pragma unroll
    for (int i = 0; i < SM_PER; ++i) {
      const int b = SM_PER * threadIdx.x + i;
      const uint64_t vs = s.sum[h][b];
      const uint32_t vn = s.count[h][b];
      const uint64_t from = by_count ? bn : bs, to = by_count ? bn + vn : bs + vs;
      if (from < target && target <= to) {
        s.bucket = b;
        s.base_s = bs;
        s.base_n = bn;
        s.n = vn;
        s.fill = 0;
      }
      bs += vs;
      bn += vn;
    }
    __syncthreads();
    const int b = s.bucket;
    const uint32_t n = s.n;
    base_s = s.base_s;
    base_n = s.base_n;
    if (h == 0) {
      bucket = b;
    } else {
      const uint64_t span = (uint64_t)hi - lo + 1, per = (span + SM_BUCKETS - 1) / SM_BUCKETS;
      const uint64_t top = hi - (uint64_t)b * per;
      lo = (uint32_t)std::max<int64_t>((int64_t)lo, (int64_t)(top - per + 1));
      hi = (uint32_t)top;
    }
    auto mine = [&](uint32_t key) { return key >= lo && key <= hi && me.bucket(key) == bucket; };
    if (n <= SM_LIST) {
      each_logit(row, bf16, V, [&](float v, int) {
        const uint32_t key = logit_key(v);
        if (key == 0 || !mine(key)) return;
        const uint64_t w = me.weight(key);
        if (w == 0) return;
        const uint32_t at = atomicAdd(&s.fill, 1u);
        s.list[at] = key;
        s.list_w[at] = w;
      });
      __syncthreads();
      if (threadIdx.x < n) {
        const uint32_t key = s.list[threadIdx.x];
        uint64_t gs = base_s;
        uint32_t gn = base_n, eq = 0;
        for (uint32_t j = 0; j < n; ++j) {
          const uint32_t k = s.list[j];
          if (k > key) gs += s.list_w[j], ++gn;
          eq += k == key;
        }
        const uint64_t w = s.list_w[threadIdx.x];
        const uint64_t from = by_count ? gn : gs, step = by_count ? 1 : w;
        if (from < target && target <= from + eq * step) {               // the same from every token of that logit
          s.key = key;
          s.base_s = gs;
          s.base_n = gn;
        }
      }
      __syncthreads();
      p.key = s.key;
      break;
    }
    if (lo == hi) {
      p.key = lo;
      break;
    }
    // too many: the range of their keys, in a histogram of its own
    __syncthreads();
    if (threadIdx.x == 0) s.lo = 0xFFFFFFFFu, s.hi = 0;
    for (int i = threadIdx.x; i < SM_BUCKETS; i += SM_THREADS) s.sum[1][i] = 0, s.count[1][i] = 0;
    __syncthreads();
    uint32_t klo = 0xFFFFFFFFu, khi = 0;
    each_logit(row, bf16, V, [&](float v, int) {
      const uint32_t key = logit_key(v);
      if (key != 0 && mine(key) && me.weight(key) != 0) klo = min(klo, key), khi = max(khi, key);
    });
#pragma unroll
    for (int d = 32; d; d >>= 1) klo = min(klo, __shfl_xor(klo, d)), khi = max(khi, __shfl_xor(khi, d));
    if ((threadIdx.x & 63) == 0) atomicMin(&s.lo, klo), atomicMax(&s.hi, khi);
    __syncthreads();
    lo = s.lo;
    hi = s.hi;
    const uint64_t per = ((uint64_t)hi - lo + SM_BUCKETS) / SM_BUCKETS;
    each_logit(row, bf16, V, [&](float v, int) {
      const uint32_t key = logit_key(v);
      if (key == 0 || !mine(key)) return;
      const uint64_t w = me.weight(key);
      if (w == 0) return;
      const int i = (int)((hi - key) / per);
      atomicAdd(reinterpret_cast<unsigned long long*>(&s.sum[1][i]), (unsigned long long)w);
      atomicAdd(&s.count[1][i], 1u);
    });
    __syncthreads();
  }
  p.w = me.weight(p.key);
  p.before_s = s.base_s;
  p.before_n = s.base_n;
  p.ties = (uint32_t)(by_count ? target - p.before_n : (target - p.before_s + p.w - 1) / p.w);
  __syncthreads();
  return p;
}

// A workgroup per row.
__global__ __launch_bounds__(SM_THREADS) void sample_kernel(SampleArgs a, int shift) {
  __shared__ SampleShared s;
  const int64_t r = blockIdx.x + (int64_t)blockIdx.y * GRID_X;
  if (r >= a.B) return;
  const int V = (int)a.V, lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const void* row = static_cast<const uint8_t*>(a.logits) + r * a.ld * (a.bf16 ? 2 : 4);
  const float temperature = a.temperature ? a.temperature[r] : a.temperature_all;
  const int32_t top_k = a.top_k ? a.top_k[r] : a.top_k_all;
  const float top_p = a.top_p ? a.top_p[r] : a.top_p_all;
  const float min_p = a.min_p ? a.min_p[r] : a.min_p_all;

  uint64_t best = 0;
  each_logit(row, a.bf16, V, [&](float v, int i) {
    const uint32_t key = logit_key(v);
    const uint64_t both = (uint64_t)key << 32 | (uint32_t)~i;
    if (key != 0 && both > best) best = both;
  });
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    const uint64_t o = __shfl_xor(best, d);
    best = o > best ? o : best;
  }
  if (lane == 0) s.wsum[wv] = best;
  for (int i = threadIdx.x; i < SM_BUCKETS; i += SM_THREADS) s.sum[0][i] = 0, s.count[0][i] = 0;
  __syncthreads();
  for (int w = 0; w < SM_WAVES; ++w) best = s.wsum[w] > best ? s.wsum[w] : best;
  // nothing to draw from, or one token left
  if (best == 0 || !(temperature > 0.f) || top_k == 1 || top_p <= 0.f || min_p > 1.f) {
    if (threadIdx.x == 0) {
      a.token[r] = best == 0 ? -1 : (int32_t)~(uint32_t)best;
      a.prob[r] = best == 0 ? 0.f : 1.f;
    }
    return;
  }
  Measure me;
  me.best_key = (uint32_t)(best >> 32);
  me.best = key_logit(me.best_key);
  me.inv_t = 1.0 / (double)temperature;
  me.unit = __builtin_bit_cast(double, (uint64_t)(1023 + shift) << 52);
  me.min_p = min_p > 0.f ? (double)min_p : 0.0;
  me.per_logit = (float)(SM_BUCKETS / ((shift + 1) * 0.6931471805599453) * me.inv_t);

  each_logit(row, a.bf16, V, [&](float v, int) {
    const uint32_t key = logit_key(v);
    const uint64_t w = me.weight(key);
    if (w == 0) return;
    const int b = me.bucket(key);
    atomicAdd(reinterpret_cast<unsigned long long*>(&s.sum[0][b]), (unsigned long long)w);
    atomicAdd(&s.count[0][b], 1u);
  });
  __syncthreads();
  uint64_t bs, total;
  uint32_t bn, count;
  scan_buckets(s, 0, bs, bn, total, count);
  if (top_k > 0 && (uint32_t)top_k < count) {
    const Place p = locate(s, me, row, a.bf16, V, true, (uint64_t)top_k);
    total = p.before_s + p.ties * p.w;
  }
  if (top_p < 1.f) {
    const double x = (double)top_p * (double)total;
    uint64_t target = (uint64_t)x;
    target += (double)target < x;
    target = std::min(std::max<uint64_t>(target, 1), total);
    const Place p = locate(s, me, row, a.bf16, V, false, target);
    total = p.before_s + p.ties * p.w;
  }
  const float u = a.u[r];
  const uint64_t target = u > 0.f ? (uint64_t)std::min((double)u * (double)total, (double)total) : 0;
  const Place p = locate(s, me, row, a.bf16, V, false, std::min(target, total - 1) + 1);

  // the token: the ties-th one that has the logit
  const int per = (V + SM_THREADS - 1) / SM_THREADS, lo = min(V, (int)threadIdx.x * per), hi = min(V, lo + per);
  auto logit = [&](int i) {
    return logit_key(a.bf16 ? bf16_to_f32(static_cast<const uint16_t*>(row)[i]) : static_cast<const float*>(row)[i]);
  };
  uint32_t n = 0;
  for (int i = lo; i < hi; ++i) n += logit(i) == p.key;
  uint32_t in = n;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_up(in, d);
    if (lane >= d) in += o;
  }
  if (lane == 63) s.wcount[wv] = in;
  __syncthreads();
  for (int w = 0; w < wv; ++w) in += s.wcount[w];
  if (in - n < p.ties && p.ties <= in) {
    uint32_t left = p.ties - (in - n);
    int i = lo;
    for (; i < hi; ++i)
      if (logit(i) == p.key && --left == 0) break;
    a.token[r] = i;
    a.prob[r] = (float)(me.p(p.key) * me.unit / (double)total);
  }
}

hipError_t launch_sample(const SampleArgs& a, hipStream_t stream) {
  int bits = 0;
  while (((int64_t)1 << bits) < a.V) ++bits;
  hipLaunchKernelGGL(sample_kernel, grid_of(a.B), dim3(SM_THREADS), 0, stream, a, std::min(62 - bits, 51));
  return hipGetLastError();
}

}  // namespace q2dev
