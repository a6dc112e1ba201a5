// Host run of the attention's index arithmetic against brute force: which key units a tile of rows reads, how they are
// shared out, and how a sequence's numbers are clamped whatever the device arrays hold. No GPU is used.
#include <stdio.h>

#include <algorithm>
#include <random>
#include <vector>

#include "../../activation_sparse_ffn_predictor_amd/csrc/attn.h"

using namespace sffn;

#define CHECK(c, ...)                                  \
  do {                                                 \
    if (!(c)) {                                        \
      printf("line %d: %s: ", __LINE__, #c);           \
      printf(__VA_ARGS__);                             \
      printf("\n");                                    \
      return 1;                                        \
    }                                                  \
  } while (0)

int main() {
  std::mt19937 g(1);
  auto pick = [&](int lo, int hi) { return (int)(lo + (long)(g() % (unsigned)(hi - lo + 1))); };
  for (int it = 0; it < 200000; ++it) {
    const int ush = pick(5, 6), len = pick(0, it % 3 ? 300 : 3000), n = pick(1, 130);
    const int p0 = len - n, r0 = pick(0, n - 1), p_lo = p0 + r0, p_hi = p0 + pick(r0, n - 1);
    const int window = it % 2 ? 0 : pick(1, 1 << pick(0, 11)), sinks = pick(0, 1 << pick(0, 9));
    const Units un = key_units(p_lo, p_hi, len, window, sinks, ush);
    std::vector<int> hit((len >> ush) + 2, 0);
    for (int u = 0; u < un.tot; ++u) {
      const int k = un.key0(u, ush);
      CHECK(k >= 0 && k < len && !(k & ((1 << ush) - 1)), "unit %d at key %d of %d", u, k, len);
      ++hit[k >> ush];
    }
    for (int x : hit) CHECK(x <= 1, "a unit twice: len %d p %d..%d window %d sinks %d", len, p_lo, p_hi, window, sinks);
    for (int p = p_lo; p <= p_hi; ++p)
      for (int j = 0; j <= p && j < len; ++j)
        if (window <= 0 || j > p - window || j < sinks)
          CHECK(hit[j >> ush], "key %d of position %d is in no unit: len %d p %d..%d window %d sinks %d", j, p, len, p_lo, p_hi,
                window, sinks);
    const int ns = pick(1, MAX_SHARES), least = pick(1, 20), step = pick(1, 2) * pick(1, 4);
    const int per = share_units(un.tot, ns, least, step), used = std::max(1, (un.tot + per - 1) / per);
    CHECK(per >= least && per % step == 0 && used <= ns, "tot %d ns %d: %d shares of %d", un.tot, ns, used, per);
    CHECK((long)used * per >= un.tot, "tot %d ns %d: %d shares of %d", un.tot, ns, used, per);
  }
  const int odd[] = {0, 1, -1, 5, 100, 2147483647, -2147483647 - 1, 1 << 30, -(1 << 30), 77};
  for (int a : odd)
    for (int b : odd)
      for (int l : odd)
        for (int T : {0, 1, 60, 1 << 24})
          for (int cols : {1, 7, 1 << 20}) {
            const int cu[2] = {a, b};
            const Seqs q{cu, &l, nullptr, 1, T, cols, cols};
            const Seq s = load_seq(q, 0, 10);
            CHECK(s.q0 >= 0 && s.n >= 0 && (long)s.q0 + s.n <= T && s.len >= 0 && s.len <= (long)cols << 10, "cu %d %d len %d T %d", a, b, l, T);
            const Units un = key_units(s.len - s.n, s.len - 1, s.len, 1 << 30, 1 << 30, 5);
            CHECK(un.tot == (s.len + 31) / 32, "len %d: %d units", s.len, un.tot);
          }
  printf("index arithmetic ok\n");
  return 0;
}
