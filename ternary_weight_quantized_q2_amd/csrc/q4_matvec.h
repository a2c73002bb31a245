// q4_matvec.h - the kernel of the 4-bit products with scales per group, instantiated
// by q4_matvec*.hip for one kind of group each.
//
// y = epilogue(x W^T), w = (q - z) s with one s and z per group of 32, 64 or a
// multiple of 128 inputs.  A code decodes to bf16 1 + q / 16 (q2_device.h); per group
// sum x (1 + q / 16) - (1 + z / 16) sum x = sum x (q - z) / 16 on the matrix cores,
// exact products and fp32 sums, and one FMA per output applies the group's scale.  Of an
// f16 zero point below 2^-9 the sum 1 + z / 16 would lose bits: sum x goes off first,
// then (z / 16) sum x (over 17 to 64 rows up to 7 % slower than the one FMA with 1 + z / 16;
// both forms with a branch by what the unit's zero points need spill, up to 35 % slower).
// A group whose codes all equal a whole zero point takes a scale of 0, so it adds exactly
// nothing; where the sums with 1.5, which stands for 8 without zero points, run through
// the same instructions as the products they cancel bit for bit by themselves.
#pragma once
#include "q2_token.h"
#include <algorithm>

namespace q2dev {

constexpr int MV_LDS = 160 * 1024;
constexpr int MV_ROWS = 64;                              // of a workgroup, at most
enum { GROUP_32 = 0, GROUP_64 = 1, GROUP_128 = 2 };      // 128: and its multiples

// Sizes that the host works out: a division takes a wave tens of scalar instructions,
// and the waves of a CU share one scalar unit.
struct MatvecShape {
  int units;                  // of a weight row
  int chunk_units;            // units whose x is in LDS at a time, a multiple of the waves of a strip
  int tile_groups, tiles;     // tiles of 16 output columns per workgroup
  int segments, row_stride;   // of x in LDS: pieces of 512 inputs per row, bytes between rows
  int segment_magic, row_step, segment_step;             // 2^16 / segments; the workgroup's waves by segments: quotient, rest
  int keep, sums;             // whether all of x stays in LDS; where the partial sums go behind it
  int last_piece, last_group, zero_bytes, per;           // per: blocks per group (groups of 128 and more)
  uint32_t weight_row;                                   // bytes
};

// The workgroup's waves are (kg, ns): ns strips of 16 weight columns, each by kg waves
// that take its units in turn; a unit is two 128-input blocks of a strip, their scales
// and zero points.  With a gated epilogue two strips hold the factors of one tile.  Up
// to four rows (E == 1) or RT tiles of sixteen share each decoded weight.
//
// x goes to LDS by direct copies, whole where it fits, else in parts, one ahead; a unit's
// codes, scales and zero points to registers, one unit ahead.  A launch starts with
// cold instruction caches, and code that runs once costs a wave about a microsecond per
// KB: the loop's body appears once, and sizes come from the host.  Captured launches
// back to back, weights from memory: one row, K = 2560, N = 2 x 9728 in groups of 64
// 11.5 us (28 MB, 2.4 TB/s; at 4.9 TB/s between the first load and the last, the rest
// is the launch, the first instructions and the last workgroups), N = 128009 44 us (184
// MB, 4.2 TB/s); 13 rows, N = 6144 7.4 us; 61 rows, K = 2560, N = 9728 in groups of 128
// 18.6 us, waits for x and for LDS with one workgroup per CU; 32 rows, K = 4096, N = 128009
// in groups of 32 120 us (320 MB), bound by vector instructions: decode, and an FMA per
// output and group.
template <int GM, int ZM, int E, int RT>
__global__ __launch_bounds__(RT > 2 ? 512 : 1024) void matvec_kernel(MatvecArgs m, MatvecShape sh) {
  constexpr int GPB = GM == GROUP_32 ? 4 : GM == GROUP_64 ? 2 : 1;        // groups per block
  constexpr int STEPS = 4 / GPB;                         // matrix steps per group
  constexpr int ROWS = E == 1 ? 4 : 16 * RT;             // of x, of a workgroup
  constexpr int NS = 2 * GPB;                            // scales of a unit and column
  constexpr int SW = GM == GROUP_128 ? 2 : NS / 2;       // dwords of scales and of f16 zero points
  constexpr int ZW = ZM == ZERO_F16 || GM == GROUP_128 ? SW : 1;
  // Where 1 + z / 16 is a bf16 and a lane has several outputs, each step adds
  // minus its products with x first, which leaves one FMA per output and group.
  constexpr bool CHAIN = E > 1 && ZM != ZERO_F16;
  const FusedArgs& a = m.f;
  extern __shared__ __align__(16) uint8_t xs[];
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int kg = blockDim.x >> 6, waves = kg * blockDim.y;
  const int ki = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), si = __builtin_amdgcn_readfirstlane(threadIdx.y);
  const int wv = si * kg + ki;
  const int64_t m0 = (int64_t)blockIdx.y * ROWS;
  const int rows = (int)std::min<int64_t>(a.M - m0, ROWS), K = (int)a.K;
  const uint32_t n_out = (uint32_t)a.N >> a.gated;
  const int half = a.gated & si, tile = si >> a.gated;
  float* const red = reinterpret_cast<float*>(xs + sh.sums);
  const NatConsts kc = q4_nat_consts();

  // Rows of x from unit u0 on, 512 inputs per copy.  Piece q of a row lies at
  // q ^ x_swizzle(row) of its 16: the 16 lanes that a pass of a fragment read serves
  // then touch 16 different bank groups, whichever the order of the groups.
  auto x_swizzle = [](int row) { return (-(row >> 2) & 3) | (row & 3) << 2; };
  const uint8_t* const x0 = reinterpret_cast<const uint8_t*>(a.x + m0 * K);
  const int wave_row = wv * sh.segment_magic >> 16;      // wv / segments
  auto each_segment = [&](auto f) {
    int row = wave_row, seg = wv - wave_row * sh.segments;
#pragma unroll 1
    while (row < rows) {
      f(row, seg);
      row += sh.row_step;
      seg += sh.segment_step;
      if (seg >= sh.segments) {
        seg -= sh.segments;
        ++row;
      }
    }
  };
  auto copy_x = [&](int u0, uint8_t* to) {
    each_segment([&](int row, int seg) {
      const int k = u0 * 256 + seg * 512 + 8 * (lane ^ x_swizzle(row & 15));
      const uint8_t* const from = x0 + ((uint32_t)row * (uint32_t)K + (uint32_t)min(k, K - 8)) * 2u;
      __builtin_amdgcn_global_load_lds(from, (lds_void*)(to + row * sh.row_stride + seg * 1024), 16, 0, 0);
    });
  };
  // Zeros where the copies ran past the end of a row.
  auto clear_x = [&](int u0, uint8_t* to) {
    if (K - u0 * 256 >= sh.segments * 512) return;
    each_segment([&](int row, int seg) {
      if (u0 * 256 + seg * 512 + 8 * (lane ^ x_swizzle(row & 15)) >= K)
        *reinterpret_cast<q2_u32x4*>(to + row * sh.row_stride + seg * 1024 + 16 * lane) = q2_u32x4{0u, 0u, 0u, 0u};
    });
  };

  struct Unit {
    uint32_t w[2][4], s[SW], z[ZW];
  };
  // Scales are one load that stays in its row, moved to their places where it began
  // before the unit; of groups of 128 and more, a half-word per block.
  auto first_scale = [&](int u) { return min(NS * u, sh.last_group + 1 - NS); };
  auto first_code = [&](int u) { return min(GPB * u, sh.zero_bytes - GPB); };
  // The next unit to load: tile group, unit, the lane's weight row.
  int tg_l = blockIdx.x, u_l = ki;
  const uint8_t *wp, *cp;
  const uint16_t *sp, *zp;
  auto aim = [&]() {
    const uint32_t n = min(((uint32_t)tg_l * sh.tiles + tile) * 16 + c, n_out - 1) + (half ? n_out : 0);
    wp = a.w + (uint64_t)n * sh.weight_row;
    sp = a.s + (uint64_t)n * (uint32_t)(sh.last_group + 1);
    if constexpr (ZM == ZERO_F16) zp = a.z + (uint64_t)n * (uint32_t)(sh.last_group + 1);
    if constexpr (ZM == ZERO_CODES) cp = m.zero_codes + (uint64_t)n * (uint32_t)sh.zero_bytes;
  };
  auto group_of = [&](int block) { return min(sh.per > 1 ? block / sh.per : block, sh.last_group); };
  auto load = [&](Unit& v) {
    if (tg_l >= sh.tile_groups) return;
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      // past the row: its last piece, x is zero there
      const q2_u32x4 t = *reinterpret_cast<const q2_u32x4*>(wp + 16u * (uint32_t)min(8 * u_l + 4 * d + g, sh.last_piece));
#pragma unroll
      for (int q = 0; q < 4; ++q) v.w[d][q] = t[q];
    }
    if constexpr (GM == GROUP_128) {
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const int gr = group_of(2 * u_l + d);
        v.s[d] = sp[gr];
        if constexpr (ZM == ZERO_F16) v.z[d] = zp[gr];
        if constexpr (ZM == ZERO_CODES) v.z[d] = cp[gr / 2];
      }
    } else {
      __builtin_memcpy(v.s, sp + first_scale(u_l), 2 * NS);
      if constexpr (ZM == ZERO_F16) __builtin_memcpy(v.z, zp + first_scale(u_l), 2 * NS);
      if constexpr (ZM == ZERO_CODES) __builtin_memcpy(v.z, cp + first_code(u_l), GPB);
    }
    u_l += kg;
    if (u_l >= sh.units) {
      u_l = ki;
      tg_l += gridDim.x;
      aim();
    }
  };
  // The halves of w moved down by n places.
  auto shift_halves = [](uint32_t(&w)[SW], int n) {
#pragma unroll
    for (int bit = NS / 2; bit > 0; bit /= 2)
      if (n & bit) {
#pragma unroll
        for (int i = 0; i < SW; ++i) {
          auto at = [&](int k) { return k < SW ? w[k] : 0u; };
          w[i] = bit > 1 ? at(i + bit / 2) : __builtin_amdgcn_alignbit(at(i + 1), w[i], 16);
        }
      }
  };

  const uint32_t sone = ZM == ZERO_8 ? 0x3FC03FC0u : 0x3F803F80u;         // bf16 1.5 / 1 pairs
  const q2_u32x4 sones = q2_u32x4{sone, sone, sone, sone};
  // Tile row 4 r holds row r where there are up to four: one of a lane's four results counts.
  int xrow[RT], swz[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int row = min(E == 1 ? c >> 2 : 16 * i + c, rows - 1);
    xrow[i] = row * sh.row_stride;
    swz[i] = x_swizzle(row & 15);
  }
  float acc[RT][E];

  Unit cur, next;
  uint8_t *xb = xs, *xnext = xs;                         // the inputs in use and the ones on their way
  copy_x(0, xs);
  if (ki < sh.units) {
    aim();
    load(next);
  }
  bool staged = false;
  for (int tg = blockIdx.x; tg < sh.tile_groups; tg += gridDim.x) {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) acc[i][e] = 0.f;
#pragma unroll 1
    for (int u0 = 0, end; u0 < sh.units; u0 = end) {     // the same for all waves of the workgroup
      end = min(u0 + sh.chunk_units, sh.units);
      if (!staged) {
        xb = xnext;
        __builtin_amdgcn_s_waitcnt(0);
        asm volatile("" ::: "memory");
        clear_x(u0, xb);
        stage_barrier<63>();                             // these are there, and the ones before are read
        if (sh.keep) {
          staged = true;
        } else {
          xnext = xs + (xb == xs ? sh.sums / 2 : 0);
          if (end < sh.units) copy_x(end, xnext);
          else if (tg + (int)gridDim.x < sh.tile_groups) copy_x(0, xnext);
        }
      }
#pragma unroll 1
      for (int u = u0 + ki; u < end; u += kg) {
        cur = next;
        load(next);
        const int at = (u - u0) * 512;
        if constexpr (GM == GROUP_128) {
          if constexpr (ZM == ZERO_CODES) {
#pragma unroll
            for (int d = 0; d < 2; ++d) cur.z[d] >>= 4 * (group_of(2 * u + d) & 1);
          }
        } else if (NS * (u + 1) > sh.last_group + 1) {     // the unit that the row ends in
          const int n = NS * u - first_scale(u);
          shift_halves(cur.s, n);
          if constexpr (ZM == ZERO_F16) shift_halves(cur.z, n);
          if constexpr (ZM == ZERO_CODES) cur.z[0] >>= 8 * (GPB * u - first_code(u));
        }
        auto scale_of = [&](int i) {
          return f16_to_f32((uint16_t)(GM == GROUP_128 ? cur.s[i] : cur.s[i / 2] >> (16 * (i & 1))));
        };
        auto zero_of = [&](int i) -> float {
          if constexpr (ZM == ZERO_F16) return f16_to_f32((uint16_t)(GM == GROUP_128 ? cur.z[i] : cur.z[i / 2] >> (16 * (i & 1))));
          else if constexpr (ZM == ZERO_8) return 8.f;
          else return (float)((GM == GROUP_128 ? cur.z[i] : cur.z[0] >> (4 * i)) & 15u);
        };
        // 16 bytes of a lane are 32 inputs of its column, piece g of the block.  Lane
        // swaps bring the dwords of a group of 32 or 64 inputs into the same registers.
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          uint32_t(&w)[4] = cur.w[d];
          auto swap32 = [&](int p, int q) {
            auto r = __builtin_amdgcn_permlane32_swap(w[p], w[q], false, false);
            w[p] = r[0];
            w[q] = r[1];
          };
          auto swap16 = [&](int p, int q) {
            auto r = __builtin_amdgcn_permlane16_swap(w[p], w[q], false, false);
            w[p] = r[0];
            w[q] = r[1];
          };
          if constexpr (GM == GROUP_32) {
            swap32(0, 2);
            swap32(1, 3);
            swap16(0, 1);
            swap16(2, 3);
          } else if constexpr (GM == GROUP_64) {
            swap32(0, 1);
            swap32(2, 3);
          }
        }
        auto reg = [](int gr, int t) { return GM == GROUP_32 ? gr : GM == GROUP_64 ? 2 * t + gr : t; };
        if constexpr (ZM != ZERO_8 || CHAIN) {
          // A group whose codes all equal its zero point is rare: look closer only where
          // the eight codes of some lane's dword are equal.
          uint64_t any = 0;
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            const uint32_t w0 = cur.w[i / GPB][reg(i % GPB, 0)];
            any |= __builtin_amdgcn_ballot_w64(w0 == __builtin_amdgcn_alignbit(w0, w0, 4));
          }
          if (any != 0) {
#pragma unroll
            for (int i = 0; i < NS; ++i) {
              uint32_t part[STEPS];
#pragma unroll
              for (int t = 0; t < STEPS; ++t) part[t] = cur.w[i / GPB][reg(i % GPB, t)];
              const uint64_t dead = column_all(q4_part_zero(part, zero_of(i)));
              if constexpr (GM == GROUP_128) cur.s[i] = zero_where(cur.s[i], dead);
              else cur.s[i / 2] &= zero_where(0xFFFFu << (16 * (i & 1)), dead) | 0xFFFFu << (16 * (~i & 1));
            }
          }
        }
        // Step j: its x was read a step before, and the sums of the group before are added
        // up behind its first products: waits for LDS and for the matrix cores overlap.
        // Left alone the compiler reads and multiplies all groups before it adds any up, which
        // takes more registers than there are: with several row tiles the reads stay in order.
        auto read = [&](int j, q2_u32x4(&v)[RT]) {
          const int d = j / 4, gr = j % 4 / STEPS, t = j % STEPS;
          const int q = GM == GROUP_32 ? 4 * gr + g : GM == GROUP_64 ? 8 * gr + 4 * (g & 1) + 2 * t + (g >> 1) : 4 * g + t;
#pragma unroll
          for (int i = 0; i < RT; ++i) v[i] = *reinterpret_cast<const q2_u32x4*>(xb + xrow[i] + at + 256 * d + 16 * (q ^ swz[i]));
        };
        q2_f32x4 sum[2][RT], tmp[2][RT];
        auto add_up = [&](int k) {
          const float s = scale_of(k), z16 = zero_of(k) * 0.0625f;
#pragma unroll
          for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int e = 0; e < E; ++e) {
              const float su = sum[k & 1][i][e];
              float t = tmp[k & 1][i][e];
              if constexpr (!CHAIN) {
                if constexpr (ZM == ZERO_8) t -= su;
                else if constexpr (ZM == ZERO_CODES) t = __builtin_fmaf(-(1.f + z16), su, t);
                else t = __builtin_fmaf(-z16, su, t - su);
              }
              float v = __builtin_fmaf(s, t, acc[i][e]);
              if constexpr (RT > 1) asm volatile("" : "+v"(v));
              acc[i][e] = v;
            }
        };
        q2_u32x4 av[2][RT];
        read(0, av[0]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int k = j / STEPS, t = j % STEPS, d = j / 4, gr = k % GPB;
          if constexpr (RT > 1) asm volatile("" ::: "memory");
          if (j + 1 < 8) read(j + 1, av[(j + 1) & 1]);
          q2_u32x4 ones = sones;
          if constexpr (CHAIN) {                           // - (1 + z / 16) in every place
            uint32_t z = 0xBFC0BFC0u;
            if constexpr (ZM == ZERO_CODES)
              z = ((GM == GROUP_128 ? cur.z[k] : cur.z[0] >> (4 * k)) & 15u) * 0x00080008u | 0xBF80BF80u;
            ones = q2_u32x4{z, z, z, z};
          }
          if constexpr (RT > 1) asm volatile("" : "+v"(cur.w[d][reg(gr, t)]));
          const q2_u32x4 bf = q4_frag(cur.w[d][reg(gr, t)], kc);
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const q2_f32x4 none = q2_f32x4{0.f, 0.f, 0.f, 0.f};
            q2_f32x4 &su = sum[k & 1][i], &tm = tmp[k & 1][i];
            su = mfma(av[j & 1][i], ones, t == 0 ? none : CHAIN ? tm : su);
            tm = mfma(av[j & 1][i], bf, CHAIN ? su : t == 0 ? none : tm);
          }
          if (t == 0 && k > 0) add_up(k - 1);
        }
        add_up(NS - 1);
      }
    }
    // Partial sums through LDS, added in the waves' order, a row tile at a time: room that
    // they take is x's.  Lane (c, g) holds rows 4 g .. (E == 1: row g).
#pragma unroll 1
    for (int rt = 0; rt < RT; ++rt) {
      if (rt > 0) stage_barrier<63>();                   // the last ones are read
#pragma unroll
      for (int e = 0; e < E; ++e) {
        red[(wv * E + e) * 64 + lane] = acc[0][e];
#pragma unroll
        for (int i = 1; i < RT; ++i) acc[i - 1][e] = acc[i][e];
      }
      stage_barrier<63>();
#pragma unroll 1
      for (int i = wv; i < sh.tiles * E; i += waves) {
        const int t = i / E, e = i % E, row = E == 1 ? g : 16 * rt + 4 * g + e;
        const uint32_t n = ((uint32_t)tg * sh.tiles + t) * 16 + c;
        const float* p = red + ((t << a.gated) * kg * E + e) * 64 + lane;
        float v = 0.f, u = 0.f;
#pragma unroll 4
        for (int q = 0; q < kg; ++q) v += p[q * 64 * E];
        if (a.gated) {
          p += kg * 64 * E;
#pragma unroll 4
          for (int q = 0; q < kg; ++q) u += p[q * 64 * E];
        }
        if (row < rows && n < n_out) store_out(a, a.bias, n_out, m0 + row, n, v * 16.f, u * 16.f);
      }
    }
    if (sh.keep && tg + (int)gridDim.x < sh.tile_groups) stage_barrier<63>();        // before the sums of the next tiles
  }
}

template <int GM, int ZM, int E, int RT>
static hipError_t run_matvec(const MatvecArgs& m, hipStream_t stream) {
  const FusedArgs& a = m.f;
  constexpr int ROWS = E == 1 ? 4 : 16 * RT;
  const int rows = (int)std::min<int64_t>(a.M, ROWS);
  MatvecShape sh = {};
  sh.units = (int)((a.K + 255) / 256);
  const int64_t out_tiles = (fused_n_out(a) + 15) / 16, strips = a.gated ? 2 * out_tiles : out_tiles;
  const int64_t row_blocks = (a.M + ROWS - 1) / ROWS;
  // Waves.  One to four rows: about ten for each CU, where the strips are fewer by
  // sharing them; where they are more, two strips by two waves each per workgroup.  More
  // waves pay more for their start, fewer leave memory idle.  A CU holds that many while
  // the rows take up to 64 KB of LDS; beyond that x goes in two parts of up to 79 KB, one
  // workgroup per CU (K = 11008, N = 16384: one row 28 us, two 47, three 81).  Workgroups of up to
  // sixteen for more rows, one per CU, whose x goes to its LDS once: as many tiles for each
  // as fill the fewest turns of the CUs.
  // One row, K = 2560: 1216 strips 11.1 us with two waves, 12.9 with one, 16.8 with five;
  // 8001 strips 45 in pairs of two waves, 48 in pairs of one or singly, 81 with five.  160
  // strips, K = 9728: 8.5 with thirteen waves, 9.4 with six.  13 rows, 384 strips: 7.2 two
  // strips by five waves each, 8.1 one by ten, 9.4 four by four.
  constexpr int WAVES = RT > 2 ? 8 : 16;                 // of a workgroup, at most
  int kg, tiles, lds;
  int64_t most = 1 << 20;
  if constexpr (E == 1) {
    tiles = strips > 1250 ? 2 : 1;
    kg = strips > 1250 ? 2 : (int)std::clamp<int64_t>(2500 / strips, 1, a.gated ? WAVES / 2 : WAVES);
    lds = 64;
  } else {
    const int widest = (RT > 1 ? WAVES : 8) / (a.gated ? 2 : 1);
    most = std::max<int64_t>(1, 256 / row_blocks);
    const int64_t turns = (out_tiles + most * widest - 1) / (most * widest);
    tiles = (int)((out_tiles + most * turns - 1) / (most * turns));
    kg = WAVES / (a.gated ? 2 * tiles : tiles);
    lds = 140;
  }
  kg = std::min(kg, sh.units);
  kg = (sh.units + (sh.units + kg - 1) / kg - 1) / ((sh.units + kg - 1) / kg);          // the same number of units for all
  const int ns = a.gated ? 2 * tiles : tiles;
  auto stride = [&](int units) { return (units * 256 + 511) / 512 * 1024; };
  // All of x in LDS where it fits, else two parts of it in turn.
  const int sum_bytes = kg * ns * 256 * E, part = (MV_LDS - sum_bytes) / 2;
  const int64_t whole = (int64_t)rows * stride(sh.units);
  sh.keep = whole <= lds * 1024 && whole + sum_bytes <= MV_LDS;
  if (!sh.keep) {
    while (kg > 1 && rows * stride(kg) > part) --kg;
    int per = 1;                                         // units of a wave in a part
    while (per * kg < sh.units && rows * stride((per + 1) * kg) <= part) ++per;
    sh.chunk_units = per * kg;
  } else {
    sh.chunk_units = sh.units;
  }
  sh.segments = (std::min(sh.chunk_units, sh.units) * 256 + 511) / 512;
  sh.row_stride = sh.segments * 1024;
  sh.segment_magic = (65536 + sh.segments - 1) / sh.segments;              // exact for 16 waves and up to 4095 segments
  sh.row_step = kg * ns / sh.segments;
  sh.segment_step = kg * ns % sh.segments;
  sh.sums = rows * sh.row_stride * (sh.keep ? 1 : 2);
  const int64_t groups = (out_tiles + tiles - 1) / tiles;
  sh.tile_groups = (int)groups;
  sh.tiles = tiles;
  sh.last_piece = (int)(a.K / 32) - 1;
  sh.last_group = (int)(a.K / m.group) - 1;
  sh.zero_bytes = (sh.last_group + 2) / 2;
  sh.per = (int)(m.group / BLOCK_K);
  sh.weight_row = (uint32_t)(a.K / 2);
  const int bytes = sh.sums + sum_bytes;
  if (bytes > MV_LDS || kg * ns > WAVES || row_blocks > 65535) return hipErrorInvalidValue;
  hipLaunchKernelGGL((matvec_kernel<GM, ZM, E, RT>), dim3((unsigned)std::min<int64_t>(groups, most), (unsigned)row_blocks), dim3(64 * kg, ns),
                     bytes, stream, m, sh);
  return hipGetLastError();
}

template <int GM, int ZM>
static hipError_t pick_matvec(const MatvecArgs& m, hipStream_t stream) {
  if (m.f.M <= 4) return run_matvec<GM, ZM, 1, 1>(m, stream);
  // More rows share a decoded weight as there is work for all CUs.  By tiles of 16 x 16
  // outputs, groups of 64 with 4-bit zero points, 16 and 32 rows per decoded weight: K = 2560,
  // 32 rows, 768 tiles 8.5 / 11.1 us, 1216 12.2 / 13.2, 2048 14.7 / 15.3, but 20 rows, 1216 tiles 11.8 /
  // 11.2, and K = 4096, 32 rows, 1216 tiles 16.7 / 16.2, 1792 20.1 / 18.8; groups of 32 with f16 zero
  // points, K = 2560, 32 rows, 1216 tiles 15.2 / 17.3; 61 rows, K = 2560, groups of 128, 2432 tiles 19.4 /
  // 17.9.  The border lies where the first of these cross.  32 and 64 rows, 64 rows of K = 2560:
  // 12288 tiles 51 / 61, 20480 87 / 89, 24576 91 / 90, 32004 120 / 117.
  const int64_t work = ((fused_n_out(m.f) + 15) / 16 << m.f.gated) * ((m.f.M + 15) / 16);
  if (m.f.M <= 16 || work <= 1200) return run_matvec<GM, ZM, 4, 1>(m, stream);
  if (m.f.M > 32 && work >= 24000) return run_matvec<GM, ZM, 4, 4>(m, stream);
  return run_matvec<GM, ZM, 4, 2>(m, stream);
}

template <int GM>
hipError_t launch_matvec(const MatvecArgs& m, hipStream_t stream) {
  if (m.zero == ZERO_CODES) return pick_matvec<GM, ZERO_CODES>(m, stream);
  if (m.zero == ZERO_F16) return pick_matvec<GM, ZERO_F16>(m, stream);
  return pick_matvec<GM, ZERO_8>(m, stream);
}
extern template hipError_t launch_matvec<GROUP_32>(const MatvecArgs&, hipStream_t);
extern template hipError_t launch_matvec<GROUP_64>(const MatvecArgs&, hipStream_t);
extern template hipError_t launch_matvec<GROUP_128>(const MatvecArgs&, hipStream_t);

}  // namespace q2dev
