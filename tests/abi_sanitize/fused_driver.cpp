// Host-side driver for the argument validation of the fused and grouped
// linears, the router and the combination, built like driver.cpp with
// AddressSanitizer and UndefinedBehaviorSanitizer on the host code.  Every call
// is rejected or empty before any HIP call.
#include <cstdint>
#include <cstdio>

#include "q2.h"

static int failures = 0;

static void expect(int got, int want, const char* what) {
  if (got != want) {
    std::fprintf(stderr, "FAIL %s: got %d (%s), want %d\n", what, got, q2_strerror(got), want);
    ++failures;
  }
}
static void expect_bytes(size_t got, size_t want, const char* what) {
  if (got != want) {
    std::fprintf(stderr, "FAIL %s: got %zu bytes, want %zu\n", what, got, want);
    ++failures;
  }
}

int main() {
  alignas(256) static unsigned char arena[1024];         // never dereferenced
  void* const F = arena;
  void* const F1 = arena + 1;
  const int64_t big = INT64_MAX, small = INT64_MIN, lim = (int64_t)1 << 46;
  auto u16 = [](void* p) { return static_cast<const uint16_t*>(p); };
  auto u8 = [](void* p) { return static_cast<const uint8_t*>(p); };
  auto i32 = [](void* p) { return static_cast<int32_t*>(p); };

  // workspace sizes: every extreme of every argument
  const int64_t edge[] = {small, -1, 0, 1, 127, 128, 511, 512, 65535, 65536, (int64_t)1 << 24, (int64_t)1 << 31, lim, lim + 1, big};
  for (int64_t m : edge)
    for (int64_t n : edge)
      for (int64_t k : edge) {
        q2_route_workspace_bytes(m, n, k);
        for (int64_t e : edge) {
          const size_t f = q2_linear_fused_workspace_bytes(m, n, k, e);
          if (e > 0 && e <= 65535 && m > 0 && n > 0 && f < q2_lowrank_workspace_bytes(m, e)) ++failures;
          q2_linear_grouped_workspace_bytes(m, e, n, k);
        }
      }
  expect_bytes(q2_linear_fused_workspace_bytes(1, 8, 128, 0), 0, "no workspace");
  expect_bytes(q2_linear_fused_workspace_bytes(lim, 8, 128, 65535), SIZE_MAX, "limbs beyond size_t");
  expect_bytes(q2_linear_grouped_workspace_bytes(8, 65537, 8, 128), 0, "too many groups");
  expect_bytes(q2_route_workspace_bytes(64, 8, 2), 0, "one workgroup");

  auto fused = [&](void* x, void* y, int64_t M, int64_t N, int64_t K, int64_t r, const q2_epilogue* e, void* ws, size_t wb) {
    return q2_linear_fused(u16(x), u8(F), u16(F), u16(F), u16(F), r, e, y, M, N, K, ws, wb, nullptr);
  };
  expect(fused(F, F, small, 8, 128, 0, nullptr, F, 0), Q2_ERR_ARG, "fused M smallest");
  expect(fused(F, F, big, 8, 128, 0, nullptr, F, 0), Q2_ERR_ARG, "fused M largest");
  expect(fused(F, F, 4, big, 128, 0, nullptr, F, 0), Q2_ERR_ARG, "fused N largest");
  expect(fused(F, F, 4, 8, big, 0, nullptr, F, 0), Q2_ERR_SHAPE, "fused K largest");
  expect(fused(F, F, 4, 8, 128, big, nullptr, F, 0), Q2_ERR_ARG, "fused r largest");
  expect(fused(F, F, 4, 8, 128, small, nullptr, F, 0), Q2_ERR_ARG, "fused r smallest");
  expect(fused(F1, F, 4, 8, 128, 0, nullptr, F, 0), Q2_ERR_ALIGN, "fused x align");
  expect(fused(F, nullptr, 4, 8, 128, 0, nullptr, F, 0), Q2_ERR_ARG, "fused y null");
  expect(fused(F, F, 4, 8, 128, 3, nullptr, F, 1), Q2_ERR_WORKSPACE, "fused workspace small");
  expect(fused(F, F, 4, 8, 128, 3, nullptr, nullptr, SIZE_MAX), Q2_ERR_ARG, "fused workspace null");
  expect(fused(F, F, 4096, 8192, 4096, 0, nullptr, F, 1024), Q2_ERR_WORKSPACE, "fused conversion workspace small");
  expect(fused(nullptr, nullptr, 0, 8, 128, 0, nullptr, nullptr, 0), Q2_OK, "fused no rows");
  q2_epilogue e = {~0u, 0u, nullptr, nullptr, nullptr};
  expect(fused(F, F, 4, 8, 128, 0, &e, F, 0), Q2_ERR_ARG, "fused activation");
  e = {Q2_ACT_NONE, ~0u, nullptr, nullptr, nullptr};
  expect(fused(F, F, 4, 8, 128, 0, &e, F, 0), Q2_ERR_ARG, "fused flags");
  e = {Q2_ACT_SILU, Q2_EPI_GATED, nullptr, nullptr, nullptr};
  expect(fused(F, F, 4, 7, 128, 0, &e, F, 0), Q2_ERR_SHAPE, "fused odd gated N");
  expect(q4_linear_fused(u16(F), u8(F), u16(F), u16(F1), nullptr, F, 4, 8, 128, nullptr), Q2_ERR_ALIGN, "q4 zero align");
  expect(q4_linear_fused(u16(F), u8(F), u16(F), u16(F), nullptr, F, big, big, 128, nullptr), Q2_ERR_ARG, "q4 sizes");

  auto grouped = [&](int64_t x_rows, void* index, int64_t R, int64_t E, int64_t N, int64_t K, const q2_epilogue* ep) {
    return q2_linear_grouped(u16(F), x_rows, i32(index), i32(F), u8(F), u16(F), ep, F, R, E, N, K, F, 0, nullptr);
  };
  expect(grouped(4, nullptr, 4, small, 8, 128, nullptr), Q2_ERR_ARG, "grouped E smallest");
  expect(grouped(4, nullptr, 4, big, 8, 128, nullptr), Q2_ERR_SHAPE, "grouped E largest");
  expect(grouped(big, F, 4, 2, 8, 128, nullptr), Q2_ERR_SHAPE, "grouped x_rows largest");
  expect(grouped(4, F, big, 2, 8, 128, nullptr), Q2_ERR_ARG, "grouped R largest");
  expect(grouped(4, F, 4, 65536, lim, 128, nullptr), Q2_ERR_ARG, "grouped E * N");
  expect(grouped(5, nullptr, 4, 2, 8, 128, nullptr), Q2_ERR_ARG, "grouped x_rows without an index");
  expect(grouped(4, F1, 4, 2, 8, 128, nullptr), Q2_ERR_ALIGN, "grouped index align");
  expect(grouped(0, nullptr, 0, 2, 8, 128, nullptr), Q2_OK, "grouped no rows");
  expect(grouped(4, nullptr, 4, 0, 8, 128, nullptr), Q2_OK, "grouped no groups");
  e = {Q2_ACT_NONE, 0u, nullptr, static_cast<float*>(F), nullptr};
  expect(grouped(4, nullptr, 4, 2, 8, 128, &e), Q2_ERR_ARG, "grouped gate");
  expect(q4_linear_grouped(u16(F), 4, nullptr, nullptr, u8(F), u16(F), u16(F), nullptr, F, 4, 2, 8, 128, nullptr),
         Q2_ERR_ARG, "q4 grouped offsets null");

  auto route = [&](int64_t T, int64_t E, int64_t k, uint32_t flags, size_t wb) {
    return q2_route(F, T, E, k, flags, i32(F), static_cast<float*>(F), i32(F), i32(F), i32(F), F, wb, nullptr);
  };
  expect(route(small, 8, 2, 0, 0), Q2_ERR_ARG, "route T smallest");
  expect(route(big, 8, 2, 0, 0), Q2_ERR_SHAPE, "route T largest");
  expect(route(4, big, 2, 0, 0), Q2_ERR_SHAPE, "route E largest");
  expect(route(4, 8, big, 0, 0), Q2_ERR_SHAPE, "route k largest");
  expect(route(4, 8, 0, 0, 0), Q2_ERR_SHAPE, "route no choice");
  expect(route(4, 8, 2, ~0u, 0), Q2_ERR_ARG, "route flags");
  expect(route(65, 8, 2, 0, 0), Q2_ERR_WORKSPACE, "route workspace");

  auto combine = [&](int64_t R, int64_t T, int64_t k, int64_t N, void* y) {
    return q2_combine(F, R, i32(F), static_cast<float*>(F), nullptr, y, T, k, N, 0, nullptr);
  };
  expect(combine(small, 4, 2, 8, F), Q2_ERR_ARG, "combine R smallest");
  expect(combine(big, 4, 2, 8, F), Q2_ERR_SHAPE, "combine R largest");
  expect(combine(4, big, 2, big, F), Q2_ERR_SHAPE, "combine T largest");
  expect(combine(4, 4, big, 8, F), Q2_ERR_SHAPE, "combine k largest");
  expect(combine(4, 4, 2, 8, F1), Q2_ERR_ALIGN, "combine y align");
  expect(combine(4, 0, 2, 8, nullptr), Q2_OK, "combine no tokens");
  if (failures == 0) std::printf("fused abi driver ok\n");
  return failures != 0;
}
