// Host run of where the block-scaled product's lanes read: every direct load of a tile, and every factor, stays inside its matrix
// whether or not the range check counts a load's scalar offset, which never exceeds the descriptor's bytes; what exists is read,
// once, to its place. No GPU is used.
#include <stdio.h>

#include <algorithm>
#include <random>
#include <vector>

#include "../../activation_sparse_ffn_predictor_amd/csrc/mm.h"

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

static const char* const BASE = (const char*)0x100000000l;

// one operand of a tile of n rows from r0 on, loaded by W waves: blocks 0 .. KB - 1, and what is asked for behind them
int operand(long rows, long ld, int K, int n, int W, long r0) {
  const Span s = rows_of(BASE, ld, r0, rows, n, K);
  const int KB = (K + 127) >> 7;
  for (int kb = 0; kb < KB + 3; ++kb) {
    std::vector<int> seen(n * 8, 0);
    for (int i = 0; i < n / 8 / W; ++i)
      for (int w = 0; w < W; ++w)
        for (int l = 0; l < 64; ++l) {
          const int row = lane_row(w, l), col = lane_col(row, l);
          const Span t = turn_of(s, i, W, ld);
          const Cols c = cols_of(kb, KB, K, col, kb < KB);
          const uint64_t off = c.in ? (uint32_t)row * (uint32_t)ld + (uint32_t)col : OOB, at = off + c.at;
          CHECK(c.at < t.bytes, "scalar offset %u of %u bytes", c.at, t.bytes);
          const long r = r0 + i * W * 8 + row, k = kb * 128l + col, byte = t.p - BASE + (long)at;
          const bool exists = r < rows && k < K;
          // whether the range check counts the scalar offset or not
          const bool a = off < t.bytes, b = at < t.bytes;
          for (const bool read : {a, b}) {
            CHECK(!exists || read, "row %ld of %ld, column %ld of %d is not read", r, rows, k, K);
            if (!read) continue;
            const long br = byte / ld, bc = byte % ld;
            CHECK(br < rows && bc + 16 <= K, "row %ld, column %ld: reads row %ld of %ld, column %ld of %d", r, k, br, rows, bc, K);
            CHECK(off + 16 <= t.bytes && (!b || at + 16 <= t.bytes), "row %ld, column %ld: partly", r, k);
            if (exists) CHECK(br == r && bc == k, "row %ld, column %ld: %ld, %ld", r, k, br, bc);
            CHECK(exists || r >= rows, "row %ld, column %ld of %d: read, and not to be", r, k, K);
          }
          // the place in LDS: 64 lanes of 16 bytes behind (i * W + w) * 1024
          const int to = (i * W + w) * 1024 + l * 16, lr = to / 128, slot = to % 128 / 16;
          CHECK(lr == i * W * 8 + row && (slot ^ ((lr >> 1) & 7)) == col / 16, "row %d slot %d", lr, slot);
          ++seen[lr * 8 + col / 16];
        }
    for (int x : seen) CHECK(x == 1, "a chunk %d times", x);
  }
  return 0;
}

// factors of a tile of BT tokens, blocks k0 .. k0 + nk - 1
int factors(int T, int KB, int BT, int t0, int k0, int nk) {
  const Span s{BASE + (long)t0 * KB * 4, (uint32_t)std::min(T - t0, BT) * (uint32_t)KB * 4};
  const int SL = BT / 8;
  const long all = (long)T * KB * 4;
  std::vector<long> ring(3 * BT * 8, -1);
  auto fetch = [&](int p) -> bool {
    for (int id = 0; id < BT; ++id) {
      const int ft = id >> 3, fk = id & 7;
      const uint32_t off = factor_at(p, SL, KB, k0, ft, fk);
      const long addr = off < s.bytes ? s.p + off - BASE : -1;
      if (addr >= 0 && (addr + 4 > all || off + 4 > s.bytes)) return false;
      ring[((((p >> 3) + 1) % 3) * BT + (p & 7) * SL + ft) * 8 + fk] = addr;
    }
    return true;
  };
  for (int p = -8; p < 2; ++p) CHECK(fetch(p), "p %d", p);
  for (int kb = 0; kb < nk; ++kb) {
    CHECK(fetch(kb + 2), "block %d of %d", kb, nk);
    for (int t = 0; t < BT && t0 + t < T; ++t) {
      const long got = ring[((kb >> 3) % 3 * BT + t) * 8 + (kb & 7)];
      CHECK(got == ((long)(t0 + t) * KB + k0 + kb) * 4, "token %d of %d, block %d + %d of %d: %ld", t0 + t, T, k0, kb, KB, got);
    }
  }
  CHECK(fetch(nk + 2), "behind %d", nk);
  return 0;
}

int main() {
  std::mt19937 g(3);
  auto pick = [&](int lo, int hi) { return (int)(lo + (long)(g() % (unsigned)(hi - lo + 1))); };
  for (int it = 0; it < 1500; ++it) {
    const int shapes[][2] = {{32, 4}, {64, 4}, {64, 8}, {128, 4}, {128, 8}, {256, 8}};
    const int *sh = shapes[it % 6], n = sh[0], W = sh[1];
    const long rows = it % 3 ? pick(1, 3 * n) : pick(1, 20), tiles = (rows + n - 1) / n;
    const int K = 16 * pick(1, it % 2 ? 30 : 9);
    const long lds[] = {K, K + 16, K + 16l * pick(1, 40), 1 << 22};
    for (long ld : lds)
      if (operand(rows, ld, K, n, W, n * (long)pick(0, (int)tiles - 1))) return 1;
  }
  if (operand(65, 1 << 22, 65536, 128, 4, 0) || operand(257, 1 << 22, 272, 256, 8, 256)) return 1;
  for (int it = 0; it < 3000; ++it) {
    const int BT = it % 2 ? 128 : 256, T = it % 3 ? pick(1, 2 * BT + 5) : pick(1, 9), KB = pick(1, it % 5 ? 40 : 3), ks = pick(1, 8);
    const int per = (KB + ks - 1) / ks, share = pick(0, ks - 1), k0 = std::min(KB, share * per), nk = std::min(KB, k0 + per) - k0;
    if (factors(T, KB, BT, BT * pick(0, (T - 1) / BT), k0, nk)) return 1;
  }
  printf("ok\n");
  return 0;
}
