// Compiled and run by tests/test_host_dense_steps.py: the closed form by which the
// dense attention kernels count a request's steps, against a plain sum over
// its row tiles, for every number of heads and every size of row tile.
#include <cstdio>
#include <cstdlib>

#include "dense_steps.h"

using namespace dsa::dense;

static uint64_t state = 1;
static int64_t upto(int64_t n) {  // a whole number below n
  state = state * 6364136223846793005ull + 1442695040888963407ull;
  return static_cast<int64_t>((state >> 33) % static_cast<uint64_t>(n));
}

static int check(int H, int rows, int64_t new_tokens, int64_t keys, int64_t cap) {
  const int tpt = rows / H;
  const Request r = make_request(0, static_cast<int32_t>(new_tokens), keys, cap, tpt);
  int64_t sum = 0;
  for (int n = 0; n <= r.n_tiles; ++n) {
    const int64_t got = steps_before(r, tpt, r.n_tiles, n);
    if (got != sum) {
      std::printf("%d heads, %d rows, %lld new tokens, %lld keys: %lld steps before row tile %d, counted %lld\n", H,
                  rows, static_cast<long long>(new_tokens), static_cast<long long>(keys), static_cast<long long>(sum),
                  n, static_cast<long long>(got));
      return 1;
    }
    if (n == r.n_tiles) break;
    // the tile's steps, counted from the definition
    const int64_t last = (n + 1) * static_cast<int64_t>(tpt) < new_tokens ? (n + 1) * static_cast<int64_t>(tpt) : new_tokens;
    int64_t seen = keys - new_tokens + last;
    if (keys < new_tokens || keys > cap) seen = keys < cap ? keys : cap;
    const int64_t steps = seen > 128 ? (seen + 127) / 128 : 1;
    if (steps != steps_of(r, tpt, n)) {
      std::printf("%d heads, %d rows: steps of row tile %d\n", H, rows, n);
      return 1;
    }
    sum += steps;
  }
  return 0;
}

int main() {
  const int tiles[4] = {16, 32, 128, 256};
  int bad = 0;
  for (int H = 1; H <= 128; ++H)
    for (int rows : tiles) {
      if (H > rows) continue;
      int wrong = 0;
      for (int i = 0; i < 60 && !wrong; ++i) {
        const int64_t n = i < 10 ? i : 1 + upto(3000), more = i % 3 ? upto(20000) : upto(300);
        wrong |= check(H, rows, n, n + more, int64_t(1) << 40);
        if (n > 1 && i % 5 == 0) wrong |= check(H, rows, n, upto(n), int64_t(1) << 40);         // fewer keys than tokens
        if (i % 7 == 0) wrong |= check(H, rows, n, n + more, 64 * upto((n + more) / 64 + 1));  // a table too small
      }
      bad += wrong;
    }
  // contexts up to the last position that 31 bits hold
  for (int H = 1; H <= 128; ++H)
    for (int rows : tiles)
      if (H <= rows) bad += check(H, rows, 400, 0x7FFFFF00 - upto(1000), int64_t(1) << 40);
  if (bad) return 1;
  std::printf("steps ok\n");
  return 0;
}
