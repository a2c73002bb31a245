// Host-side driver for the argument validation of the 4-bit products with scales
// per group and of the sampler, built like driver.cpp with AddressSanitizer and
// UndefinedBehaviorSanitizer on the host code.  Every call is rejected or empty
// before any HIP call.
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

int main() {
  alignas(256) static unsigned char arena[1024];         // never dereferenced
  unsigned char* const F = arena;
  const int64_t big = INT64_MAX, small = INT64_MIN, lim = (int64_t)1 << 46;

  // workspace sizes and refused sizes: every extreme of every argument
  const int64_t edge[] = {small, -1, 0, 1, 32, 64, 127, 128, 4096, 8193, 65535, (int64_t)1 << 24, ((int64_t)1 << 24) + 1, (int64_t)1 << 30,
                          (int64_t)1 << 31, lim, lim + 1, big - 127, big};
  auto matvec = [&](void* x, void* z, int64_t group, uint32_t flags, const q2_epilogue* e, void* y, int64_t M, int64_t N, int64_t K) {
    return q4_matvec(reinterpret_cast<uint16_t*>(x), F, reinterpret_cast<uint16_t*>(F), z, group, flags, e, y, M, N, K, nullptr);
  };
  auto sample = [&](void* logits, int64_t B, int64_t V, int64_t ld, uint32_t flags, const q2_sampling* s, void* ws, size_t bytes) {
    return q2_sample(logits, B, V, ld, flags, s, reinterpret_cast<float*>(F), reinterpret_cast<int32_t*>(F),
                     reinterpret_cast<float*>(F), ws, bytes, nullptr);
  };
  for (int64_t a : edge)
    for (int64_t b : edge) {
      const size_t bytes = q2_sample_workspace_bytes(a, b);
      if (bytes > 0 && (a > 128 || b <= 8192)) expect((int)a, 0, "workspace bytes");
      for (int64_t c : edge) {
        // a null y, or null logits, is refused where the sizes are not
        if (a != 0 && b != 0 && matvec(F, F, 64, 0, nullptr, nullptr, a, b, c) == Q2_OK) expect(0, 1, "null y");
        if (matvec(F, F, c, 0, nullptr, nullptr, 4, 8, a) == Q2_OK) ++failures;
        if (a != 0 && sample(nullptr, a, b, c, 0, nullptr, F, 0) == Q2_OK) expect(0, 1, "null logits");
      }
    }
  expect(matvec(F, F, 64, 0, nullptr, F, small, 8, 128), Q2_ERR_ARG, "M smallest");
  expect(matvec(F, F, 64, 0, nullptr, F, big, 8, 128), Q2_ERR_ARG, "M largest");
  expect(matvec(F, F, 64, 0, nullptr, F, 4, big, 128), Q2_ERR_ARG, "N largest");
  expect(matvec(F, F, 128, 0, nullptr, F, 4, 8, big - 127), Q2_ERR_ARG, "K largest");
  expect(matvec(F, F, big, 0, nullptr, F, 4, 8, 128), Q2_ERR_SHAPE, "group largest");
  expect(matvec(F, F, small, 0, nullptr, F, 4, 8, 128), Q2_ERR_SHAPE, "group smallest");
  expect(matvec(F, F, 64, ~0u, nullptr, F, 4, 8, 128), Q2_ERR_ARG, "flags");
  expect(matvec(F + 1, F, 64, 0, nullptr, F, 4, 8, 128), Q2_ERR_ALIGN, "x align");
  expect(matvec(F, F + 1, 64, 0, nullptr, F, 4, 8, 128), Q2_ERR_ALIGN, "zero align");
  expect(matvec(F, nullptr, 64, Q4_ZERO_CODES, nullptr, F, 4, 8, 128), Q2_ERR_ARG, "no zero points");
  q2_epilogue e = {~0u, 0u, nullptr, nullptr, nullptr};
  expect(matvec(F, F, 64, 0, &e, F, 4, 8, 128), Q2_ERR_ARG, "activation");
  e = {Q2_ACT_SILU, Q2_EPI_GATED, nullptr, nullptr, nullptr};
  expect(matvec(F, F, 64, 0, &e, F, 4, 7, 128), Q2_ERR_SHAPE, "odd gated N");
  expect(matvec(F, F, 64, 0, nullptr, F, 4, 8, 128), Q2_ERR_ARG, "y is x");
  expect(matvec(nullptr, nullptr, 64, 0, nullptr, nullptr, 0, 8, 128), Q2_OK, "no rows");

  q2_sampling s = {1.f, 0, 1.f, 0.f, nullptr, nullptr, nullptr, nullptr};
  expect(sample(F, small, 8, 8, 0, &s, F, 0), Q2_ERR_ARG, "B smallest");
  expect(sample(F, big, 8, 8, 0, &s, F, 0), Q2_ERR_SHAPE, "B largest");
  expect(sample(F, 4, big, big, 0, &s, F, 0), Q2_ERR_SHAPE, "V largest");
  expect(sample(F, 4, 8, small, 0, &s, F, 0), Q2_ERR_ARG, "ld smallest");
  expect(sample(F, 4, 8, big, 0, &s, F, 0), Q2_ERR_ARG, "ld largest");
  expect(sample(F, 4, 8, 8, ~0u, &s, F, 0), Q2_ERR_ARG, "sample flags");
  expect(sample(F + 2, 4, 8, 8, 0, &s, F, 0), Q2_ERR_ALIGN, "logits align");
  expect(sample(F, 4, 100000, 100000, 0, &s, F, 255), Q2_ERR_WORKSPACE, "workspace small");
  expect(sample(F, 4, 100000, 100000, 0, &s, nullptr, SIZE_MAX), Q2_ERR_ARG, "workspace null");
  expect(sample(F, 4, 100000, 100000, 0, &s, F + 128, SIZE_MAX), Q2_ERR_ALIGN, "workspace align");
  s.top_k_rows = reinterpret_cast<int32_t*>(F + 2);
  expect(sample(F, 4, 8, 8, 0, &s, F, 0), Q2_ERR_ALIGN, "top_k align");
  expect(sample(nullptr, 0, 8, 8, 0, nullptr, nullptr, 0), Q2_OK, "no logits");
  if (failures == 0) std::printf("token abi driver ok\n");
  return failures != 0;
}
