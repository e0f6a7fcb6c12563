// A dense attention batch as row tiles and steps of 128 keys: whole numbers
// only, for the kernels and, compiled by a host compiler, for the tests.
#pragma once
#include <algorithm>
#include <cstdint>

#ifdef __CUDACC__
#define DSA_STEPS_FN __device__ __forceinline__
#else
#define DSA_STEPS_FN inline
#endif

namespace dsa {
namespace dense {

#ifndef __CUDACC__
using std::max;
using std::min;
#endif

constexpr int kTile = 128;  // keys of a step

// A request's rows as work: row tile i has steps(i) = max(1, ceil(keys its
// last token sees / 128)).
struct Request {
  int32_t q0, q_len, n_tiles, kv_len;  // kv_len: its cached keys that the table can hold
  int32_t c;     // position of its first new token (a length below 0 counts as 0)
  bool uneven;   // lengths that contradict each other: every tile is charged kv_len
};

// Query tokens [q0, q1), sl cached keys (the new tokens' among them), room for
// `cap` in the block table, tpt tokens a row tile.
DSA_STEPS_FN Request make_request(int32_t q0, int32_t q1, int64_t sl, int64_t cap, int tpt) {
  Request r;
  r.q0 = q0;
  r.q_len = max(q1 - q0, 0);
  r.n_tiles = (r.q_len + tpt - 1) / tpt;
  // at most 2^31 - 256, so that sums of a few steps stay within 31 bits
  r.kv_len = static_cast<int32_t>(max(int64_t(0), min(min(sl, cap), int64_t(0x7FFFFF00))));
  r.c = static_cast<int32_t>(max(sl, int64_t(0))) - r.q_len;
  r.uneven = r.c < 0 || r.kv_len != sl;
  return r;
}
// keys visible to the token i (from 0) of the request
DSA_STEPS_FN int visible(const Request& r, int i) {
  return max(0, min(r.c + i + 1, r.kv_len));
}
DSA_STEPS_FN int steps_of(const Request& r, int tpt, int tile) {
  const int keys = r.uneven ? r.kv_len : visible(r, min(r.q_len, (tile + 1) * tpt) - 1);
  return max(1, (keys + kTile - 1) / kTile);
}
// sum over i < n of floor((a i + b) / 128)
DSA_STEPS_FN int64_t floor_sum(int64_t n, int64_t a, int64_t b) {
  if (a <= kTile && (a & (a - 1)) == 0) {  // a divides 128: floor((i + b / a) / (128 / a)), a whole run of each quotient
#ifdef __CUDA_ARCH__
    const int sh = 7 - (31 - __clz(static_cast<int>(a)));
#else
    const int sh = 7 - (31 - __builtin_clz(static_cast<unsigned>(a)));
#endif
    const auto upto = [&](int64_t x) {  // sum over j < x of floor(j / 2^sh)
      const int64_t k = x >> sh;
      return ((k * (k - 1) / 2) << sh) + k * (x & ((int64_t(1) << sh) - 1));
    };
    const int64_t b0 = b / a;
    return upto(n + b0) - upto(b0);
  }
  // the well-known count of the lattice points under a line by the steps of
  // Euclid's algorithm, here for (a, 128): whole multiples are taken out of a and
  // b, then the axes change places
  int64_t sum = 0, m = 128;
  while (true) {
    sum += (n - 1) * n / 2 * (a / m) + n * (b / m);
    a %= m;
    b %= m;
    const int64_t top = a * n + b;
    if (top < m) return sum;
    n = top / m;
    b = top % m;
    const int64_t t = m;
    m = a;
    a = t;
  }
}
// steps of the request's first n row tiles (of n_tiles) of tpt tokens
DSA_STEPS_FN int64_t steps_before(const Request& r, int tpt, int n_tiles, int n) {
  if (r.uneven) return static_cast<int64_t>(n) * steps_of(r, tpt, 0);
  if (n == 0) return 0;
  const int64_t b = static_cast<int64_t>(r.c) + tpt + kTile - 1;
  return n < n_tiles ? floor_sum(n, tpt, b) : floor_sum(n - 1, tpt, b) + steps_of(r, tpt, n - 1);
}

}  // namespace dense
}  // namespace dsa
