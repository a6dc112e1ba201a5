// Host run of where tokens stand: the positions that the attention and the write compute from a sequence's numbers, for any
// values in them, against 64-bit arithmetic. No GPU is used.
#include <stdio.h>

#include <algorithm>
#include <random>

#include "../../activation_sparse_ffn_predictor_amd/csrc/attn.h"

using namespace sffn;

int main() {
  const long MOST = (1l << 30) + (1l << 24);
  std::mt19937 g(2);
  const int odd[] = {0, 1, -1, 5, 63, 64, 65, 100, 2147483647, -2147483647 - 1, 1 << 30, -(1 << 30), 77, 1 << 24, (1 << 30) + (1 << 24)};
  long seen = 0;
  auto one = [&](int a, int b, int l, int T, int cols, int psh) {
    const int cu[2] = {a, b};
    const Seq s = load_seq(Seqs{cu, &l, nullptr, 1, T, cols, cols}, 0, psh);
    const long held = std::max(0l, std::min<long>(l, (long)cols << psh));
    if (s.len != held) { printf("len %d: %d held of %ld\n", l, s.len, held); return false; }
    for (int k = 0; k < 3 && s.n > 0; ++k) {
      const int i = k == 0 ? 0 : k == 1 ? s.n - 1 : (int)(g() % (unsigned)s.n), t = s.q0 + i;
      const long want = std::min<long>(l, MOST) - b + t;           // kv_len - n + (t - a)
      const long got = (long)s.p0 + i, other = token_pos(l, b, t);
      if (got != want && !(want < -(1l << 24) && got < 0)) { printf("cu %d %d len %d T %d row %d: %ld for %ld\n", a, b, l, T, t, got, want); return false; }
      if (other != want && !(want < -(1l << 24) && other < 0)) { printf("write: cu %d %d len %d row %d: %ld for %ld\n", a, b, l, t, other, want); return false; }
      ++seen;
    }
    return true;
  };
  for (int a : odd)
    for (int b : odd)
      for (int l : odd)
        for (int T : {1, 60, 1 << 24})
          for (int cols : {1, 4, 1 << 20})
            if (!one(a, b, l, T, cols, 10) || !one(a, b, l, T, cols, 4)) return 1;
  for (int it = 0; it < 300000; ++it) {
    const int a = (int)(g() % 200), n = (int)(g() % 100), T = 1 + (int)(g() % 300), l = (int)(g() % 300) - 20;
    if (!one(a, a + n, l, T, 1 + (int)(g() % 8), 4)) return 1;
  }
  printf("positions ok: %ld\n", seen);
  return 0;
}
