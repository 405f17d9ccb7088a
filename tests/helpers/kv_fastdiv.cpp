// Quotients of the K/V cache's launch-time divisors (csrc/kv/host.hpp,
// FastDiv), computed by its own code on the host (test code).  Prints the
// number of quotients compared; exit status 1 where one differs.
#include <cinttypes>
#include <cstdio>

#include "kv/host.hpp"

using nvfp4rq::FastDiv;

static uint64_t compared = 0, wrong = 0;

static void check(uint32_t d, const FastDiv& f, int64_t n) {
  if (n < 0 || n > INT32_MAX) return;
  ++compared;
  if (f.div(static_cast<uint32_t>(n)) != static_cast<uint32_t>(n) / d) {
    if (++wrong <= 10) std::fprintf(stderr, "%" PRId64 " / %u gives %u\n", n, d, f.div(static_cast<uint32_t>(n)));
  }
}

static void divisor(uint32_t d) {
  const FastDiv f = FastDiv::make(d);
  if (f.d != d || f.m >> 33) ++wrong;
  const int64_t top = INT32_MAX, k = top / d;
  // around the first, the last and a spread of multiples: where quotients change
  const int64_t step = k / 64 + 1;
  for (int64_t q = 0; q <= k; q += step)
    for (int64_t n = q * d - 2; n <= q * d + 2; ++n) check(d, f, n);
  for (int64_t q : {int64_t{1}, k - 1, k})
    for (int64_t n = q * d - 2; n <= q * d + 2; ++n) check(d, f, n);
  for (int64_t n = top - 3; n <= top; ++n) check(d, f, n);
}

int main() {
  for (uint32_t d = 1; d <= 70000; ++d) divisor(d);
  for (int s = 1; s < 31; ++s)
    for (int i = -3; i <= 3; ++i) {
      const int64_t d = (int64_t{1} << s) + i;
      if (d >= 1) divisor(static_cast<uint32_t>(d));
    }
  uint32_t x = 1;
  for (int i = 0; i < 200000; ++i) {  // a full-period sequence's upper bits
    x = x * 1664525u + 1013904223u;
    divisor((x >> 1) ? x >> 1 : 1);
    divisor((x >> (1 + i % 31)) ? x >> (1 + i % 31) : 1);
  }
  for (uint32_t d : {2147483647u, 2147483646u, 2147483645u, 1073741825u, 1431655766u}) divisor(d);
  std::printf("%" PRIu64 " quotients, %" PRIu64 " wrong\n", compared, wrong);
  return wrong != 0;
}
