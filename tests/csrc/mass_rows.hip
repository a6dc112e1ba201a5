// Host run of the tile kernel's row arithmetic for attention mass: which new tokens see some of a tile's keys, against brute force;
// and, whatever the device arrays hold, always tokens that there are. No GPU is used.
#include <stdio.h>

#include <algorithm>
#include <random>

#include "../../activation_sparse_ffn_predictor_amd/csrc/mass.h"

using namespace sffn;

int main() {
  std::mt19937 g(5);
  auto pick = [&](int lo, int hi) { return (int)(lo + (long)(g() % (unsigned)(hi - lo + 1))); };
  for (int it = 0; it < 200000; ++it) {
    const int n = pick(0, 60), p0 = pick(-40, 80), k0 = pick(0, 100), k1 = k0 + pick(0, 40), window = it % 2 ? 0 : pick(1, 50),
              sinks = pick(0, it % 3 ? 5 : 120);
    const Tokens t = tokens_of_keys(p0, n, k0, k1, window, sinks);
    if (!(0 <= t.first && t.first <= n && 0 <= t.end && t.end <= n)) { printf("n %d: %d .. %d\n", n, t.first, t.end); return 1; }
    for (int i = 0; i < n; ++i) {
      bool some = false;
      for (int j = k0; j <= k1; ++j) some |= j <= p0 + i && (window <= 0 || j > p0 + i - window || j < sinks);
      if (some && !(t.first <= i && i < t.end)) { printf("p0 %d n %d keys %d .. %d window %d sinks %d: token %d\n", p0, n, k0, k1, window, sinks, i); return 1; }
    }
  }
  // positions as mass_seq has them, keys, windows and sinks to their limits, heads that share one up to T * G < 2^31
  const int ps[] = {-(1 << 25), -(1 << 25) + 1, -(1 << 24), -1, 0, 1, 1 << 20, 1 << 30, (1 << 30) + (1 << 24)};
  const int ks[] = {0, 128, 256, 1 << 20, (1 << 28) + 256, (1 << 30) - 256};
  for (int p0 : ps)
    for (int k0 : ks)
      for (int n : {0, 1, 100, 1 << 24})
        for (int window : {0, 1, 1 << 20, MOST_LEN})
          for (int sinks : {0, 4, 1 << 30})
            for (int G : {1, 8, 64, 127, 65535}) {
              if ((long)n * G >= 1l << 31) continue;
              const Tokens t = tokens_of_keys(p0, n, k0, k0 + 255, window, sinks);
              const long r0 = (long)t.first * G, r1 = (long)t.end * G;
              if (t.first < 0 || t.first > n || t.end < 0 || t.end > n || r0 >= 1l << 31 || r1 >= 1l << 31) {
                printf("p0 %d k0 %d n %d window %d G %d: %d .. %d\n", p0, k0, n, window, G, t.first, t.end);
                return 1;
              }
            }
  printf("ok\n");
  return 0;
}
