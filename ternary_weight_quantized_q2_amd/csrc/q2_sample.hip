// q2_sample.hip - a token drawn from each row of logits: temperature, min-p, top-k,
// top-p, and the inverse of the cumulative distribution at a given random number.
//
// Order: logits descending, equal ones by lower token; p_i = exp((l_i - best) / T).
// Every filter leaves the first tokens of that order, and the draw is the first token
// whose cumulative p exceeds u times the sum, so nothing is sorted as a whole: each of
// the three borders is the place where a cumulative count or sum reaches a target.  A
// histogram over the logits' distance from the best one says in which of 4096 parts it
// lies, and only the tokens of those parts are gathered and sorted.
//
// A token's p is held as a whole number of 2^-S, S = 62 - ceil(log2 V) (at most 51),
// rounded once from 64-bit floating point.  Sums of whole numbers do not depend on
// their order, so a border that a random number comes close to is the same on every
// run; with 32-bit sums a hundred thousand tokens' borders would be off by as much as
// a per cent of a token's width.  A p below half a unit, 2^-46 at V = 2^17, is never drawn.
#include "q2_token.h"
#include <algorithm>
#include <cstddef>

namespace q2dev {

constexpr int SM_THREADS = 1024, SM_WAVES = SM_THREADS / 64;
constexpr int SM_BUCKETS = 4096, SM_PER = SM_BUCKETS / SM_THREADS;
constexpr int SM_LIST = 2048;                            // tokens that are sorted
constexpr int SM_PARTS = 64;                             // of a row, at most
constexpr int SM_DRAW = 256;                             // threads that sort a row's list: fewer wait less for each other
constexpr int SM_FEW = 256;                              // tokens that are compared with each other

__device__ __forceinline__ uint32_t logit_key(float v) { // order-preserving, 0 for a masked token
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);              // -0 counts as +0
  return v > -__builtin_inff() ? b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u) : 0u;
}
__device__ __forceinline__ float key_logit(uint32_t o) {
  return __builtin_bit_cast(float, o ^ ((o >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// f(four logits, the first one's token, the step between their tokens) for tokens t0 ..
// t1 - 1 of a row; NaN, which is a masked logit, in places that are none.  16 bytes at a
// time between the first and the last aligned address, four loads of a thread ahead.
// f's code appears once: a launch starts with cold instruction caches and pays about a
// microsecond per KB that it meets for the first time.
template <class F>
__device__ __forceinline__ void each_four(const void* whole, int bf16, int t0, int t1, F f) {
  const int size = bf16 ? 2 : 4, per = 16 / size, V = t1 - t0, threads = blockDim.x;
  const uint8_t* const row = static_cast<const uint8_t*>(whole) + (int64_t)t0 * size;
  const int head = min(V, (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / size);
  const int body = (V - head) / per, rest = V - body * per;              // up to per - 1 tokens in front and behind
  const q2_u32x4* const p = reinterpret_cast<const q2_u32x4*>(row + head * size);
  constexpr int AHEAD = 4;
  q2_u32x4 v[AHEAD], next[AHEAD];
  auto load = [&](int i) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) next[k] = p[min(i + k * threads, body - 1)];
  };
  if (body > 0) load(threadIdx.x);
  const int steps = (body + AHEAD * threads - 1) / (AHEAD * threads);
#pragma unroll 1
  for (int step = 0; step <= steps; ++step) {            // the last one: the rest, a token per thread
    const bool last = step == steps;
    const int i = step * AHEAD * threads + threadIdx.x;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) v[k] = next[k];
    if (step + 1 < steps) load(i + AHEAD * threads);     // past the end: the last piece again
    int one = 0;
    if (last) {
      if ((int)threadIdx.x >= rest) break;
      one = (int)threadIdx.x < head ? (int)threadIdx.x : body * per + (int)threadIdx.x;
      const uint32_t w = bf16 ? (uint32_t)reinterpret_cast<const uint16_t*>(row)[one] << 16 : reinterpret_cast<const uint32_t*>(row)[one];
      v[0] = q2_u32x4{w, 0x7FC00000u, 0x7FC00000u, 0x7FC00000u};
    }
#pragma unroll 1
    for (int k = 0; k < (last ? 1 : AHEAD); ++k) {
      const int piece = i + k * threads;
      if (!last && piece >= body) break;
      const int at = t0 + (last ? one : head + piece * per);
      const int halves = bf16 && !last ? 2 : 1;
#pragma unroll 1
      for (int h = 0; h < halves; ++h) {
        float x[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const uint32_t w = v[0][d];                    // a bit cast of the vector's element itself reads element 0
          x[d] = __builtin_bit_cast(float, halves == 1 ? w : h ? w & 0xFFFF0000u : w << 16);
        }
        f(x, at + h, halves);
      }
#pragma unroll
      for (int q = 1; q < AHEAD; ++q) v[q - 1] = v[q];
    }
  }
}
template <class F>
__device__ __forceinline__ void each_logit(const void* row, int bf16, int t0, int t1, F f) {
  each_four(row, bf16, t0, t1, [&](const float(&x)[4], int at, int by) {
#pragma unroll 1
    for (int d = 0; d < 4; ++d) f(d == 0 ? x[0] : d == 1 ? x[1] : d == 2 ? x[2] : x[3], at + d * by);
  });
}

// A kernel that needs only the beginning of it allocates that.
struct SampleShared {
  uint64_t wsum[SM_WAVES];
  uint32_t wcount[SM_WAVES];
  float wbest[SM_WAVES];
  uint64_t base_s, total, before_s[SM_WAVES];
  uint32_t base_n, bucket, n, fill, lo, hi, key, all;
  uint32_t before_n[SM_WAVES];
  struct {
    int part[2];                                         // where it begins, where it ends
    uint32_t tokens[2];                                  // before the first part, up to the last
  } border[3];
  uint64_t sum[SM_BUCKETS];                              // over all tokens
  uint32_t count[SM_BUCKETS];
  uint64_t list[SM_LIST];
  uint64_t sum2[SM_BUCKETS];                             // over a range of one bucket, or of the list
  uint32_t count2[SM_BUCKETS];
  uint64_t start[SM_BUCKETS];
};

// What a row's tokens are measured by.
struct Measure {
  float best, cut;                                       // no token further than cut from the best has a weight
  double scale, unit, min_p, per_octave;                 // log2(e) / T, 2^S, buckets per halving of p
  double step;                                           // a bucket's width as a distance of logits

  // log2 of 1 / p, at most 1000, where p is 0 in units: also of a masked logit, and of
  // infinity times zero.
  __device__ __forceinline__ double octaves(float v) const {
    return v == best ? 0.0 : __builtin_fmin(((double)best - (double)v) * scale, 1000.0);
  }
  // 2^-y: the power series of 2^r, |r| <= 1/2, to r^11 (off by 7e-15 at most).
  __device__ __forceinline__ static double p_of(double y) {
    const double n = __builtin_rint(y), r = (n - y) * 0.69314718055994530942;
    double q = 1.0 / 39916800;
    q = __builtin_fma(q, r, 1.0 / 3628800);
    q = __builtin_fma(q, r, 1.0 / 362880);
    q = __builtin_fma(q, r, 1.0 / 40320);
    q = __builtin_fma(q, r, 1.0 / 5040);
    q = __builtin_fma(q, r, 1.0 / 720);
    q = __builtin_fma(q, r, 1.0 / 120);
    q = __builtin_fma(q, r, 1.0 / 24);
    q = __builtin_fma(q, r, 1.0 / 6);
    q = __builtin_fma(q, r, 0.5);
    q = __builtin_fma(q, r, 1.0);
    q = __builtin_fma(q, r, 1.0);
    return __builtin_ldexp(q, -(int)n);
  }
  // Whole number of units; 0 for a token that is below min-p or too unlikely.
  __device__ __forceinline__ uint64_t weight(double y) const {
    const double q = p_of(y);
    const uint64_t w = __builtin_bit_cast(uint64_t, q * unit + 0x1p52) - __builtin_bit_cast(uint64_t, 0x1p52);
    return q >= min_p ? w : 0;
  }
  // Does not fall as the logit falls: the difference and the products round monotonically.
  __device__ __forceinline__ int bucket(double y) const {
    const double t = y * per_octave;
    return t < SM_BUCKETS - 1 ? (int)t : SM_BUCKETS - 1;
  }
  // Whether the logit may have a weight; the exact test is weight() != 0.
  __device__ __forceinline__ bool near(float v) const { return !(best - v > cut); }
};

// Inclusive sums over the lanes.
__device__ __forceinline__ void scan_lanes(uint64_t& s, uint32_t& n) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t os = __shfl_up(s, d);
    const uint32_t on = __shfl_up(n, d);
    if (lane >= d) s += os, n += on;
  }
}
// Sums before this thread's SM_PER buckets, and the totals.
__device__ __forceinline__ void scan_buckets(SampleShared& s, const uint64_t (&own_s)[SM_PER], const uint32_t (&own_n)[SM_PER],
                                             uint64_t& before_s, uint32_t& before_n, uint64_t& total_s, uint32_t& total_n) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  uint64_t vs = 0;
  uint32_t vn = 0;
#pragma unroll
  for (int i = 0; i < SM_PER; ++i) vs += own_s[i], vn += own_n[i];
  uint64_t is = vs;
  uint32_t in = vn;
  scan_lanes(is, in);
  __syncthreads();                                       // the waves' sums of an earlier scan are read
  if (lane == 63) s.wsum[wv] = is, s.wcount[wv] = in;
  __syncthreads();
  uint64_t ws = lane < SM_WAVES ? s.wsum[lane] : 0;
  uint32_t wn = lane < SM_WAVES ? s.wcount[lane] : 0;
  scan_lanes(ws, wn);
  total_s = __shfl(ws, 63);
  total_n = __shfl(wn, 63);
  before_s = is - vs;
  before_n = in - vn;
  if (wv > 0) before_s += __shfl(ws, wv - 1), before_n += __shfl(wn, wv - 1);
}

// The first place of the order where the cumulative count (by_count) or weight reaches
// target, which lies between 1 and the total: the logit's key, what lies before tokens
// of that logit, and how many of these it takes.  For parts of the histogram with more
// tokens than the list holds: one pass over the row per step, each with a histogram of
// its own over the range of keys that is left.
struct Place {
  uint32_t key, before_n, ties;
  uint64_t before_s, w;
};

__device__ __noinline__ Place locate(SampleShared& s, const Measure& me, const void* row, int bf16, int V, bool by_count,
                                     uint64_t target) {
  Place p;
  uint32_t lo = 1, hi = 0xFFFFFFFFu;                     // keys of the range
  int bucket = -1;
  uint64_t base_s = 0;
  uint32_t base_n = 0;
  uint64_t* const list_w = s.list + SM_FEW;
  for (int h = 0;; h = 1) {
    uint64_t bs, ts;
    uint32_t bn, tn;
    uint64_t own_s[SM_PER];
    uint32_t own_n[SM_PER];
#pragma unroll
    for (int i = 0; i < SM_PER; ++i) {
      own_s[i] = (h ? s.sum2 : s.sum)[SM_PER * threadIdx.x + i];
      own_n[i] = (h ? s.count2 : s.count)[SM_PER * threadIdx.x + i];
    }
    scan_buckets(s, own_s, own_n, bs, bn, ts, tn);
    bs += base_s;
    bn += base_n;
#pragma unroll
    for (int i = 0; i < SM_PER; ++i) {
      const int b = SM_PER * threadIdx.x + i;
      const uint64_t vs = own_s[i];
      const uint32_t vn = own_n[i];
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
    // tokens of the range that have a weight, with their keys
    auto each = [&](auto f) {
      each_logit(row, bf16, 0, V, [&](float v, int) {
        if (!me.near(v)) return;
        const uint32_t key = logit_key(v);
        const double y = me.octaves(v);
        if (key < lo || key > hi || me.bucket(y) != bucket) return;
        const uint64_t w = me.weight(y);
        if (w != 0) f(key, w);
      });
    };
    if (n <= SM_FEW) {
      each([&](uint32_t key, uint64_t w) {
        const uint32_t at = atomicAdd(&s.fill, 1u);
        s.list[at] = key;
        list_w[at] = w;
      });
      __syncthreads();
      if (threadIdx.x < n) {
        const uint64_t key = s.list[threadIdx.x];
        uint64_t gs = base_s;
        uint32_t gn = base_n, eq = 0;
        for (uint32_t j = 0; j < n; ++j) {
          const uint64_t k = s.list[j];
          if (k > key) gs += list_w[j], ++gn;
          eq += k == key;
        }
        const uint64_t w = list_w[threadIdx.x];
        const uint64_t from = by_count ? gn : gs, step = by_count ? 1 : w;
        if (from < target && target <= from + eq * step) {               // the same from every token of that logit
          s.key = (uint32_t)key;
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
    __syncthreads();
    if (threadIdx.x == 0) s.lo = 0xFFFFFFFFu, s.hi = 0;
    for (int i = threadIdx.x; i < SM_BUCKETS; i += SM_THREADS) s.sum2[i] = 0, s.count2[i] = 0;
    __syncthreads();
    uint32_t klo = 0xFFFFFFFFu, khi = 0;
    each([&](uint32_t key, uint64_t) { klo = min(klo, key), khi = max(khi, key); });
#pragma unroll
    for (int d = 32; d; d >>= 1) klo = min(klo, __shfl_xor(klo, d)), khi = max(khi, __shfl_xor(khi, d));
    if ((threadIdx.x & 63) == 0) atomicMin(&s.lo, klo), atomicMax(&s.hi, khi);
    __syncthreads();
    const uint32_t new_lo = s.lo, new_hi = s.hi;
    const uint64_t per = ((uint64_t)new_hi - new_lo + SM_BUCKETS) / SM_BUCKETS;
    each([&](uint32_t key, uint64_t w) {
      const int i = (int)((new_hi - key) / per);
      atomicAdd(reinterpret_cast<unsigned long long*>(&s.sum2[i]), (unsigned long long)w);
      atomicAdd(&s.count2[i], 1u);
    });
    lo = new_lo;
    hi = new_hi;
    __syncthreads();
  }
  p.w = me.weight(me.octaves(key_logit(p.key)));
  p.before_s = s.base_s;
  p.before_n = s.base_n;
  p.ties = (uint32_t)(by_count ? target - p.before_n : (target - p.before_s + p.w - 1) / p.w);
  __syncthreads();
  return p;
}

// ceil(part * whole) as a target: 1 .. whole.
__device__ __forceinline__ uint64_t part_of(float part, uint64_t whole) {
  const double x = (double)part * (double)whole;
  uint64_t t = (uint64_t)x;
  t += (double)t < x;
  return std::min(std::max<uint64_t>(t, 1), whole);
}
// The cumulative weight that the draw reaches first: more than u of the total.
__device__ __forceinline__ uint64_t draw_target(float u, uint64_t total) {
  const uint64_t t = u > 0.f ? (uint64_t)std::min((double)u * (double)total, (double)total) : 0;
  return std::min(t, total - 1) + 1;
}

// The row's borders by passes over it, whatever the histogram's parts hold: by one
// workgroup, also of a row that several share.  16-bit logits far from zero, whose steps are
// wide, come here: 128009 of them around 16, top-p 0.99 339 us for one row (45 around 10, where
// the list holds the tokens), 444 for 64 rows; 128009 equal ones 680 us.
__device__ __noinline__ void sample_slow(SampleShared& s, const Measure& me, const void* row, int bf16, int V, int top_k,
                                         float top_p, float u, uint64_t total, uint32_t count, int32_t* token, float* prob) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  if (top_k > 0 && (uint32_t)top_k < count) {
    const Place p = locate(s, me, row, bf16, V, true, (uint64_t)top_k);
    total = p.before_s + p.ties * p.w;
  }
  if (top_p < 1.f) {
    const Place p = locate(s, me, row, bf16, V, false, part_of(top_p, total));
    total = p.before_s + p.ties * p.w;
  }
  const Place p = locate(s, me, row, bf16, V, false, draw_target(u, total));
  // the token: the ties-th one that has the logit
  const int per = (V + SM_THREADS - 1) / SM_THREADS, lo = min(V, (int)threadIdx.x * per), hi = min(V, lo + per);
  auto key = [&](int i) {
    return logit_key(bf16 ? bf16_to_f32(static_cast<const uint16_t*>(row)[i]) : static_cast<const float*>(row)[i]);
  };
  uint32_t n = 0;
  for (int i = lo; i < hi; ++i) n += key(i) == p.key;
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
      if (key(i) == p.key && --left == 0) break;
    *token = i;
    *prob = (float)(me.p_of(me.octaves(key_logit(p.key))) * me.unit / (double)total);
  }
}

// ---- a row's steps -----------------------------------------------------------------
// What S, and with it the number of buckets per halving of p, comes to.
struct SampleUnits {
  double unit, per_octave, octaves_per;                  // 2^S; buckets and their inverse
  float reach;                                           // octaves to half a unit
};
struct Settings {
  float temperature, top_p, min_p, u;
  int32_t top_k;
  __device__ __forceinline__ bool greedy() const { // the first token of the order, whatever its p
    return !(temperature > 0.f) || top_k == 1 || top_p <= 0.f || min_p > 1.f;
  }
};
__device__ __forceinline__ Settings settings_of(const SampleArgs& a, int64_t r) {
  return Settings{a.temperature ? a.temperature[r] : a.temperature_all, a.top_p ? a.top_p[r] : a.top_p_all,
                  a.min_p ? a.min_p[r] : a.min_p_all, a.u[r], a.top_k ? a.top_k[r] : a.top_k_all};
}
__device__ __forceinline__ Measure measure_of(const Settings& c, float best, const SampleUnits& of) {
  Measure me;
  const double half = 0.69314718055994530942 * (double)c.temperature;    // the distance that halves p
  me.best = best;
  me.scale = 1.4426950408889634 / (double)c.temperature;
  me.unit = of.unit;
  me.min_p = c.min_p > 0.f ? (double)c.min_p : 0.0;
  me.per_octave = of.per_octave;
  me.step = half * of.octaves_per;
  // Half a unit is 2^-(S + 1); min-p cuts nearer.  A little further out: the exact tests come behind it.
  float reach = of.reach;
  if (c.min_p > 0.f) reach = fminf(reach, 0.01f - __builtin_amdgcn_logf(c.min_p));     // log2
  me.cut = (float)(reach * half * 1.000001);
  return me;
}

__device__ __forceinline__ float max_of_lanes(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}
// The largest of the range's logits, in all threads.
__device__ __forceinline__ float best_of(SampleShared& s, const void* row, int bf16, int t0, int t1) {
  float best = -__builtin_inff();
  each_four(row, bf16, t0, t1, [&](const float(&x)[4], int, int) {                     // a NaN is dropped
    best = fmaxf(best, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
  });
  best = max_of_lanes(best);
  if ((threadIdx.x & 63) == 0) s.wbest[threadIdx.x >> 6] = best;
  __syncthreads();
  return max_of_lanes(s.wbest[threadIdx.x & (SM_WAVES - 1)]);
}
// The range's first token that has the largest logit, ~0 without one, by wave.
__device__ __forceinline__ uint32_t first_of(const void* row, int bf16, int t0, int t1, float best) {
  uint32_t first = 0xFFFFFFFFu;
  each_four(row, bf16, t0, t1, [&](const float(&x)[4], int at, int by) {
#pragma unroll
    for (int d = 0; d < 4; ++d)
      if (x[d] == best) first = min(first, (uint32_t)(at + d * by));
  });
#pragma unroll
  for (int d = 32; d; d >>= 1) first = min(first, __shfl_xor(first, d));
  return first;
}
// The range's tokens into the histogram in s.
__device__ __forceinline__ void fill_histogram(SampleShared& s, const Measure& me, const void* row, int bf16, int t0, int t1) {
  each_four(row, bf16, t0, t1, [&](const float(&x)[4], int, int) {
    if (!(me.near(x[0]) || me.near(x[1]) || me.near(x[2]) || me.near(x[3]))) return;
    uint64_t w[4];
    int b[4];
#pragma unroll
    for (int d = 0; d < 4; ++d) {                        // four chains at once: one waits for every step
      const double y = me.octaves(x[d]);
      w[d] = me.weight(y);
      b[d] = me.bucket(y);
    }
#pragma unroll
    for (int d = 0; d < 4; ++d)
      if (w[d] != 0) {
        atomicAdd(reinterpret_cast<unsigned long long*>(&s.sum[b[d]]), (unsigned long long)w[d]);
        atomicAdd(&s.count[b[d]], 1u);
      }
  });
}

// The parts of the histogram where the borders lie.  Until the tokens of top-k's part
// are looked at, the sum of what it leaves is known to within that part, and so on: a
// range of parts for each border.
struct Borders {
  bool by_k, by_p;
  int lo[3], hi[3];                                      // parts of top-k, top-p, the draw
  uint64_t total;                                        // the sum of all
  uint32_t count;
  uint32_t chosen_count;                                 // tokens in the parts

  __device__ __forceinline__ bool chosen(int b) const {
    return (b >= lo[0] && b <= hi[0]) || (b >= lo[1] && b <= hi[1]) || (b >= lo[2] && b <= hi[2]);
  }
};
// The parts' sums and counts, SM_PER of each thread, are in s.sum and s.count.  start_s,
// start_n, where given: for the chosen parts, what lies before them.  One wave looks for where
// the borders begin and one for where they end, while the others wait: sixteen that find
// the same take four turns of each SIMD for it (5 us in place of 3).
__device__ __forceinline__ Borders borders_of(SampleShared& s, const Settings& c, const uint64_t (&vs)[SM_PER], const uint32_t (&vn)[SM_PER],
                                              uint64_t* start_s, uint32_t* start_n) {
  static_assert(SM_WAVES <= 64 && SM_PER <= 64 && SM_LIST >= SM_THREADS + SM_THREADS / 2, "one lane each, room in the list");
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  uint64_t* const upto_s = s.list;                       // a thread's parts and those before them in its wave
  uint32_t* const upto_n = reinterpret_cast<uint32_t*>(s.list + SM_THREADS);
  uint64_t is = 0;
  uint32_t in = 0;
#pragma unroll
  for (int i = 0; i < SM_PER; ++i) is += vs[i], in += vn[i];
  const uint64_t own_s = is;
  const uint32_t own_n = in;
  scan_lanes(is, in);
  upto_s[threadIdx.x] = is;
  upto_n[threadIdx.x] = in;
  if (lane == 63) s.wsum[wv] = is, s.wcount[wv] = in;
  __syncthreads();
  if (wv < 2) {
    const uint64_t wave_s = lane < SM_WAVES ? s.wsum[lane] : 0;
    const uint32_t wave_n = lane < SM_WAVES ? s.wcount[lane] : 0;
    uint64_t ws = wave_s;
    uint32_t wn = wave_n;
    scan_lanes(ws, wn);
    uint64_t left = __shfl(ws, 63);                      // the least or the most that the borders so far leave
    const uint32_t all = __shfl(wn, 63);
    if (wv == 0) {
      if (lane < SM_WAVES) s.before_s[lane] = ws - wave_s, s.before_n[lane] = wn - wave_n;
      if (lane == 0) s.total = left, s.all = all;
    }
    const bool by_k = c.top_k > 0 && (uint32_t)c.top_k < all, by_p = c.top_p < 1.f;
#pragma unroll 1
    for (int border = by_k ? 0 : by_p ? 1 : 2; border < 3; border = border == 0 && !by_p ? 2 : border + 1) {
      const uint64_t target = border == 0 ? (uint64_t)c.top_k : border == 1 ? part_of(c.top_p, left) : draw_target(c.u, left);
      // the part that reaches the target: its wave, its thread there, its place
      const int at = __builtin_ctzll(__builtin_amdgcn_ballot_w64(lane < SM_WAVES && (border ? ws : (uint64_t)wn) >= target));
      const uint64_t base_s = __shfl(ws - wave_s, at);
      const uint32_t base_n = __shfl(wn - wave_n, at);
      const uint64_t ts = base_s + upto_s[64 * at + lane];
      const uint32_t tn = base_n + upto_n[64 * at + lane];
      const int th = __builtin_ctzll(__builtin_amdgcn_ballot_w64((border ? ts : (uint64_t)tn) >= target));
      uint64_t before = th ? __shfl(ts, th - 1) : base_s, own;
      uint32_t before_n = th ? __shfl(tn, th - 1) : base_n, own_n;
      int part = SM_PER * (64 * at + th);
      const int last = part + SM_PER - 1;
#pragma unroll 1
      for (;; ++part) {
        own = s.sum[part];
        own_n = s.count[part];
        if (part == last || (border ? before + own : (uint64_t)before_n + own_n) >= target) break;
        before += own;
        before_n += own_n;
      }
      left = wv ? before + own : before + 1;
      if (lane == 0) s.border[border].part[wv] = part, s.border[border].tokens[wv] = wv ? before_n + own_n : before_n;
    }
  }
  __syncthreads();
  Borders o;
  o.total = s.total;
  o.count = s.all;
  o.by_k = c.top_k > 0 && (uint32_t)c.top_k < o.count;
  o.by_p = c.top_p < 1.f;
  // A later border's parts lie at or before an earlier one's; what both hold counts once.
  uint32_t counted = o.count;
  o.chosen_count = 0;
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    const bool is = j == 0 ? o.by_k : j == 1 ? o.by_p : true;
    o.lo[j] = is ? s.border[j].part[0] : 0;
    o.hi[j] = is ? s.border[j].part[1] : -1;
    const uint32_t from = is ? s.border[j].tokens[0] : counted, to = is ? s.border[j].tokens[1] : counted;
    o.chosen_count += min(to, counted) - min(from, counted);
    counted = min(from, counted);
  }
  if (start_s) {
    uint64_t before_s = s.before_s[wv] + is - own_s;
    uint32_t before_n = s.before_n[wv] + in - own_n;
#pragma unroll
    for (int i = 0; i < SM_PER; ++i) {
      const int b = SM_PER * threadIdx.x + i;
      if (o.chosen(b)) start_s[b] = before_s, start_n[b] = before_n;
      before_s += vs[i];
      before_n += vn[i];
    }
  }
  return o;
}

// The range's tokens of the parts, key above the complement of the token.  The logits of
// a border's parts lie in a range of distances from the best one, and rounding does not
// turn an order round, so distances in 32 bits drop nearly all others: first by the
// draw's range and one that holds top-k's and top-p's.  Distances are not negative and are
// compared by their bits.
template <class F>
__device__ __forceinline__ void each_chosen(const Measure& me, const Borders& o, const void* row, int bf16, int t0, int t1, F f) {
  uint32_t from[3], over[3], lo = 0xFFFFFFFFu, hi = 0;   // lo, hi: of top-k and top-p
#pragma unroll
  for (int j = 0; j < 3; ++j) {                          // a little wider: the exact test comes behind it
    const bool none = o.lo[j] > o.hi[j], all = !(me.best < __builtin_inff());          // its own distance is no number
    const uint32_t first = all || o.lo[j] == 0 ? 0u : __builtin_bit_cast(uint32_t, (float)(o.lo[j] * me.step * (1 - 1e-6)));
    const uint32_t last = all || o.hi[j] == SM_BUCKETS - 1 ? 0xFFFFFFFFu : __builtin_bit_cast(uint32_t, (float)((o.hi[j] + 1) * me.step * (1 + 1e-6)));
    from[j] = none ? 0xFFFFFFFFu : first;
    over[j] = none ? 0u : last - first;
    if (!none && j < 2) lo = min(lo, first), hi = max(hi, last);
  }
  each_four(row, bf16, t0, t1, [&](const float(&x)[4], int at, int by) {
    uint32_t away[4];
#pragma unroll
    for (int d = 0; d < 4; ++d) away[d] = __builtin_bit_cast(uint32_t, me.best - x[d]);
    auto least = [&](uint32_t n) { return min(min(away[0] - n, away[1] - n), min(away[2] - n, away[3] - n)); };
    bool in = least(from[2]) <= over[2];
    if (o.by_k || o.by_p) in |= least(lo) <= hi - lo;    // the same for all lanes
    if (!in) return;
#pragma unroll 1
    for (int d = 0; d < 4; ++d) {
      const uint32_t w = d == 0 ? away[0] : d == 1 ? away[1] : d == 2 ? away[2] : away[3];
      if (w - from[0] > over[0] && w - from[1] > over[1] && w - from[2] > over[2]) continue;
      const float v = d == 0 ? x[0] : d == 1 ? x[1] : d == 2 ? x[2] : x[3];
      const double y = me.octaves(v);
      if (o.chosen(me.bucket(y)) && me.weight(y) != 0) f((uint64_t)logit_key(v) << 32 | (uint32_t)~(at + d * by));
    }
  });
}

// The draw from the n tokens of the parts, in s.list in any order (n <= SM_LIST);
// start_s, start_n: what lies before the parts.  By the first SM_DRAW threads alone (one row of
// 4099: 15.3 us in place of 16.5 by all).  One row of 8192 with 100 equal logits at the border 19 us,
// 300 26, 1000 37, 2000 62.
__device__ __forceinline__ void draw(SampleShared& s, const Settings& c, const Measure& me, bool by_k, bool by_p, uint64_t total,
                                     const uint64_t* start_s, const uint32_t* start_n, uint32_t n, int32_t* token, float* prob) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  int size = 64;
  while (size < (int)n) size <<= 1;
  if (size <= SM_DRAW) {
    // Largest first: an entry's place is the number of larger ones.  All are different.
    __syncthreads();
    const uint64_t mine = threadIdx.x < n ? s.list[threadIdx.x] : 0;
    int place = 0;
    if ((int)threadIdx.x < (int)((n + 63) & ~63u)) {     // whole waves
#pragma unroll 4
      for (int j = 0; j < (int)n; ++j) place += s.list[j] > mine;
    }
    __syncthreads();
    if (threadIdx.x < n) s.list[place] = mine;
    __syncthreads();
  } else {
    for (int i = (int)n + threadIdx.x; i < size; i += SM_DRAW) s.list[i] = 0;
    __syncthreads();
#pragma unroll 1
    for (int span = 2; span <= size; span <<= 1)
#pragma unroll 1
      for (int step = span >> 1; step; step >>= 1) {
#pragma unroll 1
        for (int i = threadIdx.x; i < size / 2; i += SM_DRAW) {
          const int lo = ((i & ~(step - 1)) << 1) | (i & (step - 1)), hi = lo | step;
          const uint64_t x = s.list[lo], z = s.list[hi];
          if ((x < z) == ((lo & span) == 0)) s.list[lo] = z, s.list[hi] = x;
        }
        __syncthreads();
      }
  }
  // What lies before each entry: the sum over the list, less where its part begins, and
  // what lies before the part.  A thread takes `own` entries, one after the other; their
  // weights and parts lie where the histogram was.
  const int own = (size + SM_DRAW - 1) / SM_DRAW, i0 = own * threadIdx.x, i1 = min(i0 + own, (int)n);
  auto octaves = [&](int i) { return me.octaves(key_logit((uint32_t)(s.list[i] >> 32))); };
  uint64_t vs = 0;
#pragma unroll 1
  for (int i = i0; i < i1; ++i) {
    const double y = octaves(i);
    const uint64_t w = me.weight(y);
    s.sum[i] = w;
    s.count[i] = (uint32_t)me.bucket(y);
    vs += w;
  }
  __syncthreads();
  uint32_t vf = 0;                                       // the last entry that begins a part
#pragma unroll 1
  for (int i = max(i0, 1); i < i1; ++i)
    if (s.count[i - 1] != s.count[i]) vf = i;
  uint64_t is = vs;
  uint32_t mf = vf;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t os = __shfl_up(is, d);
    const uint32_t of = __shfl_up(mf, d);
    if (lane >= d) is += os, mf = max(mf, of);
  }
  if (lane == 63) s.wsum[wv] = is, s.wcount[wv] = mf;
  __syncthreads();
  uint64_t run = is - vs;
  uint32_t first = __shfl_up(mf, 1);
  if (lane == 0) first = 0;
#pragma unroll 1
  for (int k = 0; k < wv; ++k) run += s.wsum[k], first = max(first, s.wcount[k]);
  const uint64_t run0 = run;
#pragma unroll 1
  for (int i = i0; i < i1; ++i) s.sum2[i] = run, run += s.sum[i];
  __syncthreads();
  // f(entry, the number and weight of what lies before it, its own weight)
  auto each = [&](auto f) {
    uint64_t at = run0;
    uint32_t from = first;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
      const uint32_t part = s.count[i];
      const uint64_t w = s.sum[i];
      if (i > 0 && s.count[i - 1] != part) from = i;
      f(i, start_n[part] + (i - from), start_s[part] + at - s.sum2[from], w);
      at += w;
    }
  };
#pragma unroll 1
  for (int step = by_k ? 0 : by_p ? 1 : 2; step < 3; step = step == 0 && !by_p ? 2 : step + 1) {
    const uint64_t target = step == 0 ? 0 : step == 1 ? part_of(c.top_p, total) : draw_target(c.u, total);
    each([&](int i, uint32_t before_n, uint64_t before, uint64_t w) {
      if (step == 0 ? before_n + 1 != (uint32_t)c.top_k : before >= target || target > before + w) return;
      if (step < 2) {
        s.total = before + w;
      } else {
        *token = (int32_t)~(uint32_t)s.list[i];
        *prob = (float)(me.p_of(octaves(i)) * me.unit / (double)total);
      }
    });
    __syncthreads();
    if (step < 2) total = s.total;
    __syncthreads();
  }
}

__device__ __forceinline__ const void* row_of(const SampleArgs& a, int64_t r) {
  return static_cast<const uint8_t*>(a.logits) + r * a.ld * (a.bf16 ? 2 : 4);
}

// ---- a workgroup per row ------------------------------------------------------------
// One row of 4099, top-k: 15.3 us, dependent steps of one workgroup (best 2.4, histogram 3.4,
// borders 3.0, gathering 2.5, draw 2.6).  256 rows of 128009, min-p: 91 us for 131 MB;
// the best logit 24 (5.4 TB/s), a pass of exponentials and LDS additions 24, the one that gathers 16, the slowest
// row 20 behind the median; vector instructions issue in 38 % of the cycles.  Greedy, 256
// rows of 128009 48 us: the row is read once for its largest logit and once for its place.
__global__ __launch_bounds__(SM_THREADS) void sample_kernel(SampleArgs a, SampleUnits of) {
  extern __shared__ __align__(16) uint8_t smem[];
  SampleShared& s = *reinterpret_cast<SampleShared*>(smem);
  const int64_t r = blockIdx.x + (int64_t)blockIdx.y * GRID_X;
  if (r >= a.B) return;
  const int V = (int)a.V;
  const void* const row = row_of(a, r);
  const Settings c = settings_of(a, r);
  for (int i = threadIdx.x; i < SM_BUCKETS; i += SM_THREADS) s.sum[i] = 0, s.count[i] = 0;
  if (threadIdx.x == 0) s.lo = 0xFFFFFFFFu;
  const float best = best_of(s, row, a.bf16, 0, V);
  if (!(best > -__builtin_inff())) {                     // nothing to draw from
    if (threadIdx.x == 0) a.token[r] = -1, a.prob[r] = 0.f;
    return;
  }
  if (c.greedy()) {
    const uint32_t at = first_of(row, a.bf16, 0, V, best);
    if ((threadIdx.x & 63) == 0) atomicMin(&s.lo, at);
    __syncthreads();
    if (threadIdx.x == 0) a.token[r] = (int32_t)s.lo, a.prob[r] = 1.f;
    return;
  }
  const Measure me = measure_of(c, best, of);
  fill_histogram(s, me, row, a.bf16, 0, V);
  __syncthreads();
  uint64_t vs[SM_PER];
  uint32_t vn[SM_PER];
#pragma unroll
  for (int i = 0; i < SM_PER; ++i) vs[i] = s.sum[SM_PER * threadIdx.x + i], vn[i] = s.count[SM_PER * threadIdx.x + i];
  const Borders o = borders_of(s, c, vs, vn, s.start, s.count2);
  if (o.chosen_count > SM_LIST) {
    sample_slow(s, me, row, a.bf16, V, c.top_k, c.top_p, c.u, o.total, o.count, a.token + r, a.prob + r);
    return;
  }
  if (threadIdx.x == 0) s.fill = 0;
  __syncthreads();
  each_chosen(me, o, row, a.bf16, 0, V, [&](uint64_t e) { s.list[atomicAdd(&s.fill, 1u)] = e; });
  __syncthreads();
  if (threadIdx.x >= SM_DRAW) return;                    // whole waves
  draw(s, c, me, o.by_k, o.by_p, o.total, s.start, s.count2, o.chosen_count, a.token + r, a.prob + r);
}

// ---- several workgroups per row -------------------------------------------------------
// Few rows leave most CUs idle: one row of 128009 takes one workgroup 87 us.  Here a row's
// tokens are cut into parts, and what the workgroups of a row tell each other goes through
// the workspace from one launch to the next: each part's best logit, the histogram, the
// list of the tokens to sort.  One row of 128009 25 us, 32 rows 42, 64 rows bf16 61 to 64: the four
// launches' dependent steps, then the 64-bit exponentials (8 and 13 us of the last two).
struct RowSpace {
  uint64_t sum[SM_BUCKETS];
  uint64_t list[SM_LIST];
  uint64_t start_s[SM_BUCKETS];
  uint32_t count[SM_BUCKETS];
  uint32_t start_n[SM_BUCKETS];
  float best[SM_PARTS];
  uint64_t total;
  uint32_t fill, first, all, chosen, by_k, by_p;
};

struct Part {
  int64_t r;
  int t0, t1;
  const void* row;
};
__device__ __forceinline__ Part part_of_row(const SampleArgs& a, int per) {
  Part p;
  p.r = blockIdx.y;
  p.t0 = blockIdx.x * per;
  p.t1 = min(p.t0 + per, (int)a.V);
  p.row = row_of(a, p.r);
  return p;
}
__device__ __forceinline__ float row_best(const RowSpace& sp, int parts) {
  static_assert(SM_PARTS == 64, "a lane for each part");
  return max_of_lanes(sp.best[min((int)threadIdx.x & 63, parts - 1)]);
}

__global__ __launch_bounds__(SM_THREADS) void sample_best_kernel(SampleArgs a, int per, RowSpace* ws) {
  extern __shared__ __align__(16) uint8_t smem[];
  const Part p = part_of_row(a, per);
  RowSpace& sp = ws[p.r];
  for (int i = blockIdx.x * SM_THREADS + threadIdx.x; i < SM_BUCKETS; i += gridDim.x * SM_THREADS) sp.sum[i] = 0, sp.count[i] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) sp.fill = 0, sp.first = 0xFFFFFFFFu;
  const float best = best_of(*reinterpret_cast<SampleShared*>(smem), p.row, a.bf16, p.t0, p.t1);
  if (threadIdx.x == 0) sp.best[blockIdx.x] = best;
}

__global__ __launch_bounds__(SM_THREADS) void sample_histogram_kernel(SampleArgs a, int per, SampleUnits of, RowSpace* ws) {
  extern __shared__ __align__(16) uint8_t smem[];
  SampleShared& s = *reinterpret_cast<SampleShared*>(smem);
  const Part p = part_of_row(a, per);
  RowSpace& sp = ws[p.r];
  const Settings c = settings_of(a, p.r);
  const float best = row_best(sp, gridDim.x);
  if (!(best > -__builtin_inff())) return;
  if (c.greedy()) {
    const uint32_t at = first_of(p.row, a.bf16, p.t0, p.t1, best);
    if ((threadIdx.x & 63) == 0 && at != 0xFFFFFFFFu) atomicMin(&sp.first, at);
    return;
  }
  for (int i = threadIdx.x; i < SM_BUCKETS; i += SM_THREADS) s.sum[i] = 0, s.count[i] = 0;
  __syncthreads();
  fill_histogram(s, measure_of(c, best, of), p.row, a.bf16, p.t0, p.t1);
  __syncthreads();
  for (int i = threadIdx.x; i < SM_BUCKETS; i += SM_THREADS) {
    if (s.count[i] == 0) continue;
    atomicAdd(reinterpret_cast<unsigned long long*>(&sp.sum[i]), (unsigned long long)s.sum[i]);
    atomicAdd(&sp.count[i], s.count[i]);
  }
}

__global__ __launch_bounds__(SM_THREADS) void sample_gather_kernel(SampleArgs a, int per, SampleUnits of, RowSpace* ws) {
  extern __shared__ __align__(16) uint8_t smem[];
  SampleShared& s = *reinterpret_cast<SampleShared*>(smem);
  const Part p = part_of_row(a, per);
  RowSpace& sp = ws[p.r];
  const Settings c = settings_of(a, p.r);
  const float best = row_best(sp, gridDim.x);
  if (!(best > -__builtin_inff()) || c.greedy()) return;
  const bool lead = blockIdx.x == 0;                     // tells the draw what it found
  if (threadIdx.x == 0) s.fill = 0;
  uint64_t vs[SM_PER];
  uint32_t vn[SM_PER];
#pragma unroll
  for (int i = 0; i < SM_PER; ++i) {
    const int b = SM_PER * threadIdx.x + i;
    s.sum[b] = vs[i] = sp.sum[b];
    s.count[b] = vn[i] = sp.count[b];
  }
  const Borders o = borders_of(s, c, vs, vn, lead ? sp.start_s : nullptr, lead ? sp.start_n : nullptr);
  if (lead && threadIdx.x == 0) sp.total = o.total, sp.all = o.count, sp.chosen = o.chosen_count, sp.by_k = o.by_k, sp.by_p = o.by_p;
  if (o.chosen_count > SM_LIST) return;
  each_chosen(measure_of(c, best, of), o, p.row, a.bf16, p.t0, p.t1, [&](uint64_t e) { s.list[atomicAdd(&s.fill, 1u)] = e; });
  __syncthreads();
  const uint32_t n = s.fill;                             // a wait for memory for all of them, not for each
  if (threadIdx.x == 0 && n > 0) s.n = atomicAdd(&sp.fill, n);
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < n; i += SM_THREADS)
    if (s.n + i < SM_LIST) sp.list[s.n + i] = s.list[i];
}

__global__ __launch_bounds__(SM_THREADS) void sample_draw_kernel(SampleArgs a, int parts, SampleUnits of, RowSpace* ws) {
  extern __shared__ __align__(16) uint8_t smem[];
  SampleShared& s = *reinterpret_cast<SampleShared*>(smem);
  const int64_t r = blockIdx.x;
  const RowSpace& sp = ws[r];
  const Settings c = settings_of(a, r);
  const float best = row_best(sp, parts);
  const bool none = !(best > -__builtin_inff());
  if (none || c.greedy()) {
    if (threadIdx.x == 0) a.token[r] = none ? -1 : (int32_t)sp.first, a.prob[r] = none ? 0.f : 1.f;
    return;
  }
  const Measure me = measure_of(c, best, of);
  const uint32_t n = sp.chosen;
  if (n > SM_LIST) {
    for (int i = threadIdx.x; i < SM_BUCKETS; i += SM_THREADS) s.sum[i] = sp.sum[i], s.count[i] = sp.count[i];
    __syncthreads();
    sample_slow(s, me, row_of(a, r), a.bf16, (int)a.V, c.top_k, c.top_p, c.u, sp.total, sp.all, a.token + r, a.prob + r);
    return;
  }
  if (threadIdx.x >= SM_DRAW) return;                    // whole waves
  for (int i = threadIdx.x; i < (int)n; i += SM_DRAW) s.list[i] = sp.list[i];
  draw(s, c, me, sp.by_k != 0, sp.by_p != 0, sp.total, sp.start_s, sp.start_n, n, a.token + r, a.prob + r);
}

// Tokens of a part; 0 where a workgroup takes whole rows.  As many parts as keep the
// workgroups of all rows on the CUs at once, where what the parts spare, about half a
// microsecond per 1024 tokens, is more than three launches and the ways through memory
// cost, which grows with the rows, quickly up to 32.  By one workgroup and by parts, f32 from the
// whole distribution: 1 row of 16384 19.4 / 21.7 us, of 20000 22.5 / 21.6; 8 of 18000 22.4 / 23.5,
// of 24000 25.7 / 24.0; 16 of 20000 24.2 / 25.1, of 24000 26.1 / 25.6; 32 of 24000 26.7 / 29.5, of 32768
// 31.2 / 31.9, of 40000 36.8 / 32.7; 64 of 32768 32.0 / 36.3, of 40000 37.5 / 37.5, of 50021 43.6 / 38.0; 96
// of 40000 38.3 / 41.7, of 50021 45.0 / 44.8, of 64000 51.6 / 48.6; 128 of 50021 45.5 / 48.8, of 64000 53.6 / 55.5,
// of 128009 95.8 / 84.8.  With top-k and top-p, or bf16, the two meet up to a tenth of the tokens apart.
static int part_tokens(int64_t B, int64_t V) {
  const int64_t parts = std::min<int64_t>({256 / std::max<int64_t>(B, 1), (V + 4095) / 4096, SM_PARTS});
  const int64_t least = std::max(std::min<int64_t>(14000 + 350 * B, 25000), 14000 + 100 * B);
  if (parts <= 1 || V - V / parts < least) return 0;
  return (int)(((V + parts - 1) / parts + 1023) / 1024 * 1024);
}

size_t sample_workspace_bytes(int64_t B, int64_t V) {
  return part_tokens(B, V) ? (size_t)B * sizeof(RowSpace) : 0;
}

hipError_t launch_sample(const SampleArgs& a, void* workspace, hipStream_t stream) {
  int bits = 0;
  while (((int64_t)1 << bits) < a.V) ++bits;
  const int shift = std::min(62 - bits, 51), per = part_tokens(a.B, a.V);
  const SampleUnits of = {(double)(1ull << shift), (double)SM_BUCKETS / (shift + 1), (shift + 1) / (double)SM_BUCKETS, shift + 1.01f};
  constexpr size_t LDS = sizeof(SampleShared), SMALL = offsetof(SampleShared, sum), HIST = offsetof(SampleShared, list), LIST = offsetof(SampleShared, sum2);
  if (per == 0) {
    hipLaunchKernelGGL(sample_kernel, grid_of(a.B), dim3(SM_THREADS), LDS, stream, a, of);
    return hipGetLastError();
  }
  RowSpace* const ws = static_cast<RowSpace*>(workspace);
  const dim3 grid((unsigned)((a.V + per - 1) / per), (unsigned)a.B);
  hipLaunchKernelGGL(sample_best_kernel, grid, dim3(SM_THREADS), SMALL, stream, a, per, ws);
  hipLaunchKernelGGL(sample_histogram_kernel, grid, dim3(SM_THREADS), HIST, stream, a, per, of, ws);
  hipLaunchKernelGGL(sample_gather_kernel, grid, dim3(SM_THREADS), LIST, stream, a, per, of, ws);
  hipLaunchKernelGGL(sample_draw_kernel, dim3((unsigned)a.B), dim3(SM_THREADS), LDS, stream, a, (int)grid.x, of, ws);
  return hipGetLastError();
}

}  // namespace q2dev
