// The list of steps that the attention of many rows (paged_attn.cu) cuts into equal shares: what its
// kernels, and the join of a common beginning with the sequences' tails (decode.cu), agree on.
//
// A unit is 128 query rows: tokens * heads.  A segment is a pair of units of one sequence (or group
// of sequences) and KV head, or its last odd unit; a step is one tile of 128 keys.  Each segment has steps + kPagedAttnSegCost positions; segments
// stand in the order (sequence, KV head and chunk of its query heads, pair).
#pragma once

#include "internal.h"

namespace mcs {

constexpr int kPagedAttnRows = 128;
constexpr int kPagedAttnKeys = 128;
constexpr int kPagedAttnSegCost = 2;  // what changing the segment costs, in steps

// Parts of segments that cross shares: slot 2 c of share c for a segment that ends there, 2 c + 1
// for one that goes on.  (log2 maximum, sum of weights) of the 256 rows, then the rows' D sums.
constexpr int kPagedAttnPartRows = 2 * kPagedAttnRows;
__host__ __device__ constexpr size_t paged_attn_part_floats(int D) { return static_cast<size_t>(kPagedAttnPartRows) * (2 + D); }

#ifdef __CUDACC__

// x / y, in 32 bits where that is enough (a fifth of the time).
__device__ __forceinline__ long long quotient(long long x, long long y) {
  return ((x | y) >> 32) == 0 ? static_cast<uint32_t>(x) / static_cast<uint32_t>(y) : x / y;
}

// sum of floor((a i + b) / m) over i < n: Euclid's algorithm on (m, a), both below 2^16; b below 2^32.
__device__ __forceinline__ long long floor_sum(long long n, uint32_t m, uint32_t a, long long b) {
  long long sum = 0;
  while (n > 0) {
    const uint32_t qa = a / m;
    const long long qb = quotient(b, m);
    sum += (n - 1) * n / 2 * qa + n * qb;
    a -= qa * m;
    b -= qb * m;
    const long long y = a * n + b;
    if (y < m) break;
    n = quotient(y, m);
    b = y - n * m;
    const uint32_t t = m;
    m = a;
    a = t;
  }
  return sum;
}

// A sequence of the list (shared beginnings: a group): n tokens, rows cu .. cu + n of q, keys
// [0, keys), of which token t sees keys - n + t + 1 (causal) or all.
struct Seq {
  int cu, n, keys;
};
__device__ __forceinline__ int tiles_until(const PagedAttnArgs& a, const Seq& s, int e) {
  return static_cast<int>((static_cast<long long>(a.causal ? s.keys - s.n + e : s.keys) + kPagedAttnKeys - 1) / kPagedAttnKeys);
}
__device__ __forceinline__ bool load_seq(const PagedAttnArgs& a, int g, Seq& s, bool report) {
  const int lo = a.cu[g], hi = a.cu[g + 1];
  s.keys = a.keys[g];
  s.cu = lo;
  s.n = 0;
  if (s.keys < 0 || static_cast<long long>(s.keys) > static_cast<long long>(a.max_pages) * a.page ||
      (hi != lo && (lo < 0 || hi < lo || hi > a.T || (a.causal && hi - lo > s.keys)))) {
    if (report) atomicOr(a.status, DEV_BOUNDS);
    return false;
  }
  s.n = s.keys > 0 ? hi - lo : 0;
  return s.n > 0;
}
__device__ __forceinline__ int units_of(const PagedAttnArgs& a, const Seq& s) {
  return (s.n + a.tokens - 1) / a.tokens;
}
// Positions of the first k pairs of a sequence's KV head.
__device__ __forceinline__ long long pairs_upto(const PagedAttnArgs& a, const Seq& s, int k) {
  if (k <= 0) return 0;
  if (!a.causal) return static_cast<long long>(k) * (tiles_until(a, s, s.n) + kPagedAttnSegCost);
  const int w = 2 * a.tokens;
  // the last pair may end with the sequence, inside its second unit
  const bool cut = static_cast<long long>(k) * w > s.n;
  const int whole = cut ? k - 1 : k;
  return floor_sum(whole, kPagedAttnKeys, w, static_cast<long long>(s.keys) - s.n + w + kPagedAttnKeys - 1) +
         (cut ? tiles_until(a, s, s.n) : 0) + static_cast<long long>(k) * kPagedAttnSegCost;
}
__device__ __forceinline__ long long positions_of(const PagedAttnArgs& a, const Seq& s) {
  const int units = units_of(a, s);
  return pairs_upto(a, s, units / 2) + ((units & 1) ? tiles_until(a, s, s.n) + kPagedAttnSegCost : 0);
}

// The shares of a list of `all` positions: share c begins at floor(all * c / shares).
__device__ __forceinline__ long long share_begin(int c, long long all, int shares) {
  const long long q = quotient(all, shares);
  return c * q + static_cast<uint32_t>(c) * static_cast<uint32_t>(all - q * shares) / static_cast<uint32_t>(shares);
}
// The share that holds position x: an estimate that is off by one at most, then exact products.
__device__ __forceinline__ int share_of(long long x, long long all, int shares) {
  const long long y = (x + 1) * shares;
  int c = static_cast<int>(static_cast<float>(x) * (static_cast<float>(shares) / static_cast<float>(all)));
  while (c > 0 && c * all >= y) --c;
  while ((c + 1) * all < y) ++c;
  return c;
}

// Where the row of sequence b's query head hh of KV head h lies in a common beginning's result: parts
// of shares c0 to c1, at `row` of each, or (c0 == c1) whole.
struct PagedAttnPlace {
  int c0, c1, row;
};
__device__ __forceinline__ PagedAttnPlace paged_attn_place(const SharedArgs& p, int b, int h, int hh) {
  const int g = p.group_of[b], n = p.cu[g + 1] - p.cu[g], t = b - p.cu[g];
  const int units = (n + p.tokens - 1) / p.tokens, pairs = units / 2, u = t / p.tokens;
  const int segs = p.segs, i = u / 2, steps = (p.keys[g] + kPagedAttnKeys - 1) / kPagedAttnKeys;
  const long long pair_size = steps + kPagedAttnSegCost, size = (pairs + (units & 1)) * pair_size;
  const long long all = p.places[p.G] * segs;
  const long long at = p.places[g] * segs + (h * p.chunks + hh / p.heads) * size + i * pair_size;
  const int shares = static_cast<int>(min(all, static_cast<long long>(p.grid)));
  return {share_of(at, all, shares), share_of(at + steps - 1, all, shares),
          (i < pairs ? (u & 1) * kPagedAttnRows : 0) + (t - u * p.tokens) * p.heads + hh % p.heads};
}

#endif

}  // namespace mcs
