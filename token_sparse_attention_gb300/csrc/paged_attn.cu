// Attention of many query rows over a paged cache on tcgen05 tensor cores: the new tokens
// of a step, several per sequence (causal), and the common beginning of sequences that
// decode together.
//
// o_i = sum_j exp(s_ij - m_i) v_j / l_i with s_ij = scale q_i . k_j over the keys j that row
// i sees: the query heads of a KV head and the tokens of a sequence (or the sequences of a
// group) are rows of one product with the same keys.  4 D flops per visible (row, key) pair
// against 4 D bytes (bf16) per key: from about 290 rows on the tensor cores bound it,
// below that HBM does, as long as each key is read once for all rows.
//
// A unit is 128 rows (MMA M): tokens * heads, a token's heads next to each other, as they lie
// in q.  A segment is a pair of units (a, b) of one sequence and KV head, which share every
// K and V tile of 128 keys, or its last odd unit, whose tiles the two softmax chains take in
// turn (a the even, b the odd ones) and join in the CTA.  All segments in a row form one list
// of steps (a step: one tile for two units, or two tiles for one), and each of the SMs' CTAs
// takes an equal share of it, whatever the lengths are: few long sequences are so split along
// their keys, many short ones along the list.  What a share holds whole it writes at once;
// parts of segments that cross shares go to the workspace and are joined in the order of
// their keys by a second, programmatically dependent launch.
//
// One CTA per SM, 16 warps, as in the dense kernel:
//   warps 0-3   softmax and epilogue of chain a; thread t owns row t (TMEM lane t)
//   warps 4-7   the same for chain b
//   warp 8      loads: TMA boxes of a page's rows
//   warps 9-14  bf16: look through the V tiles in which some row's mask leaves something out
//               (below).  E4M3: convert every tile to f16
//   warp 15     TMEM and MMA issue (one elected lane)
// TMEM: S_a, S_b (P is written over S), O_a, O_b.  Shared memory: Q_a, Q_b and a ring of K
// and V tiles that runs on from segment to segment; the next segment's queries are loaded
// once its last scores are there, while softmax, products and epilogue are still at work.
//
// A weight of zero does not hide an infinite or NaN value from a matrix product: 0 * inf =
// NaN.  So V tiles that hold keys behind a row's last one are looked through before the
// product: rows that hold no token become zeros, and values of tokens that are not finite
// become zeros, too, with the first such key of each column kept; a row that sees that key
// gets NaN in the column.  One or two tiles per segment are concerned.
#include <cuda_fp16.h>

#include <algorithm>

#include "internal.h"
#include "launch.cuh"
#include "paged_list.cuh"
#include "ptx.cuh"

namespace mcs {
namespace {

constexpr int BM = kPagedAttnRows;  // rows per unit
constexpr int BN = kPagedAttnKeys;  // keys per tile
constexpr int kSegCost = kPagedAttnSegCost;
constexpr int kLoaders = 7;
constexpr int kFirstLoader = 8;
constexpr int kMmaWarp = kFirstLoader + kLoaders;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr int kMaxSms = 160;
constexpr int kSlab = 16;    // keys that surely lie in one page
constexpr int kSlabs = BN / kSlab;
constexpr int kWindow = 32 / kSlabs;  // tiles whose pages a warp looks up at once
constexpr int kBadSlots = 16;         // steps ahead of the softmax that loads may be: ring depth

// Rescaled only when a row's maximum grows by more than 2^16 (f16 weights: 2^15 < 65504).
template <bool E4M3>
constexpr float kThreshold = E4M3 ? 15.f : 16.f;

template <int D, bool E4M3>
struct Layout {
  static constexpr int kSub = D / 64;                 // 128-byte column sub-tiles of a row
  static constexpr int kSubBytes = BN * 128;
  static constexpr int kTileBytes = kSub * kSubBytes;
  // E4M3 bytes on their way to f16: in the tile's second half, whose lines they are converted to
  // (D = 128), or behind the tile (D = 64: a row's bytes are not as long as a line)
  static constexpr int kRaw = D == 128 ? kSubBytes : kTileBytes;
  static constexpr int kStageBytes = kTileBytes + (E4M3 && D == 64 ? BN * D : 0);
  static constexpr int kStages = D == 128 ? 5 : E4M3 ? 8 : 12;
  static constexpr int kRing = 2 * kTileBytes;
  static constexpr int kBars = kRing + kStages * kStageBytes;
  // MMA batches done, round robin.  A waiter reads the phase of batch n's barrier, which is
  // unambiguous as long as batch n + kDone cannot be done yet.  Loads lag furthest: they wait for the
  // last reader of the item kStages back, and what the kStages - 1 items behind it feed is at most
  // three batches for every two (segments of one step), and three more.
  static constexpr int kDone = D == 128 ? 16 : 32;
  static_assert(kDone >= (kStages - 1) / 2 * 3 + 5, "batch barriers must outnumber the lag");
  static constexpr int kNumBars = 3 * kStages + kDone + 10;
  static constexpr int kBadKey = kBars + kNumBars * 8;           // [2][D] words
  static constexpr int kMl = kBadKey + 2 * D * 4;                // [3][128] floats
  static constexpr int kMisc = kMl + 3 * BM * 4;                 // Misc
  static constexpr int kSmem = kMisc + 80;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kStages <= kBadSlots, "bad slots");
};

// ------------------------------------------------------------------ the list

// A walk over a CTA's share, segment by segment; every role makes it by itself.
struct Walk {
  Seq s;
  int g, head, i;  // sequence, KV head and its chunk of query heads, pair (the last odd unit behind them)
  bool single;     // an odd unit, whose tiles the chains take in turn
  int tiles, tiles_a;  // of the segment; of a pair's first unit
  int steps;       // of the segment
  int t0, count;   // the share's steps of it: [t0, t0 + count)
  long long left;  // positions from t0 to the share's end
  int index;       // segments of the share in front of this one
};
__device__ __forceinline__ void set_segment(const PagedAttnArgs& a, Walk& w) {
  const int pairs = units_of(a, w.s) / 2;
  w.single = w.i >= pairs;
  if (w.single) {
    w.tiles = w.tiles_a = tiles_until(a, w.s, w.s.n);
    w.steps = (w.tiles + 1) / 2;
  } else {
    const long long e = (2LL * w.i + 2) * a.tokens;
    w.tiles = tiles_until(a, w.s, static_cast<int>(min(e, static_cast<long long>(w.s.n))));
    w.tiles_a = tiles_until(a, w.s, static_cast<int>(e - a.tokens));
    w.steps = w.tiles;
  }
}
__device__ __forceinline__ bool next_segment(const PagedAttnArgs& a, Walk& w) {
  w.left -= w.steps + kSegCost - w.t0;
  if (w.left <= 0) return false;
  const int units = units_of(a, w.s);
  if (++w.i >= units / 2 + (units & 1)) {
    w.i = 0;
    if (++w.head >= a.Hkv * a.chunks) {
      w.head = 0;
      do {  // (there is one, unless the lengths change under the kernel)
        if (++w.g >= a.G) return false;
      } while (!load_seq(a, w.g, w.s, false));
    }
  }
  set_segment(a, w);
  w.t0 = 0;
  w.count = static_cast<int>(min(static_cast<long long>(w.steps), w.left));
  ++w.index;
  return true;
}
// Whether chain x has a tile in step j of the share's part of the segment, and which.
__device__ __forceinline__ int tile_of(const Walk& w, int x, int j) {
  return w.single ? 2 * (w.t0 + j) + x : w.t0 + j;
}
__device__ __forceinline__ bool has_tile(const Walk& w, int x, int j) {
  return tile_of(w, x, j) < (!w.single && x == 0 ? w.tiles_a : w.tiles);
}
// Keys that every row of the segment sees: tiles behind it are looked through.
__device__ __forceinline__ int seen_by_all(const PagedAttnArgs& a, const Walk& w) {
  return a.causal ? w.s.keys - w.s.n + 2 * w.i * a.tokens + 1 : w.s.keys;
}
// A walk in one register of a warp's lanes, while the softmax needs the registers.
__device__ __forceinline__ int fold(const Walk& w, int lane) {
  const int f[14] = {w.s.cu, w.s.n, w.s.keys, w.g, w.head, w.i, w.single, w.tiles, w.tiles_a, w.steps, w.t0, w.index,
                     static_cast<int>(w.left), static_cast<int>(w.left >> 32)};
  int x = w.count;
#pragma unroll
  for (int k = 0; k < 14; ++k)
    if (lane == k) x = f[k];
  return x;
}
__device__ __forceinline__ Walk unfold(int x) {
  int f[15];
#pragma unroll
  for (int k = 0; k < 15; ++k) f[k] = __shfl_sync(0xffffffffu, x, k);
  return {{f[0], f[1], f[2]}, f[3], f[4], f[5], f[6] != 0, f[7], f[8], f[9], f[10], f[14],
          static_cast<long long>(static_cast<uint32_t>(f[12])) | (static_cast<long long>(f[13]) << 32), f[11]};
}

// In how many steps of the share's part chain x has a tile (the first ones).
__device__ __forceinline__ int steps_of(const Walk& w, int x) {
  const int all = w.single ? (w.tiles - x + 1) / 2 : x == 0 ? w.tiles_a : w.tiles;
  return max(0, min(w.count, all - w.t0));
}
__device__ __forceinline__ int last_tile(const Walk& w) { return min(tile_of(w, w.single ? 1 : 0, w.count - 1), w.tiles - 1); }

// ------------------------------------------------------------------ small pieces

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status));
}
// Used only while tearing down: bounded by time alone.
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - t0 > kWaitLimitCycles) return;
  }
}
__device__ __forceinline__ float sum8(const uint64_t* acc) {
  float a0, a1, a2, a3, a4, a5, a6, a7;
  f2_unpack(acc[0], a0, a1);
  f2_unpack(acc[1], a2, a3);
  f2_unpack(acc[2], a4, a5);
  f2_unpack(acc[3], a6, a7);
  return ((a0 + a1) + (a2 + a3)) + ((a4 + a5) + (a6 + a7));
}
__device__ __forceinline__ float max64(const float* s) {
  float m0 = s[0], m1 = s[1], m2 = s[2], m3 = s[3];
#pragma unroll
  for (int c = 4; c < 60; c += 8) {
    m0 = fmax3(m0, s[c + 0], s[c + 1]);
    m1 = fmax3(m1, s[c + 2], s[c + 3]);
    m2 = fmax3(m2, s[c + 4], s[c + 5]);
    m3 = fmax3(m3, s[c + 6], s[c + 7]);
  }
  m0 = fmax3(m0, s[60], s[61]);
  m1 = fmax3(m1, s[62], s[63]);
  return fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
}
// Byte offset of 16-byte chunk `seg` of row r in a 128-row tile of 128-byte-swizzled sub-tiles.
__device__ __forceinline__ int swz_offset(int r, int seg) {
  return (seg >> 3) * (BN * 128) + r * 128 + (((seg & 7) ^ (r & 7)) << 4);
}
// Scores that the row does not see become -inf where they stand (TMEM): keys from `valid` on and
// slabs of pages outside the cache.  Few tiles have any; the others' path holds no mask.
__device__ __noinline__ void mask_scores(uint32_t tS, int valid, uint32_t bad) {
#pragma unroll 1
  for (int c0 = 0; c0 < BN; c0 += 32) {
    uint32_t s[32];
    tmem_ld32(tS + c0, s);
    tmem_ld_wait();
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (c0 + c >= valid || ((bad >> ((c0 + c) / kSlab)) & 1u)) s[c] = 0xFF800000u;
    tmem_st32(tS + c0, s);
  }
  tmem_st_wait();
}

// Values that are not finite in tiles that are looked through: per column the first key, as
// segment (its number in the share, plus one) << 10 | 1023 - (key - first such tile's first key), so
// that a later segment's entries are larger than what is left of an earlier one's.  Two
// segments' records stand side by side; a third waits until the first one's rows are written.
// The tiles of a segment that are looked through hold fewer than 128 + 256 + 128 keys.
__device__ __forceinline__ uint32_t bad_mark(int index) { return (static_cast<uint32_t>(index + 1) & 0x3FFFFFu) << 10; }
// Notes the bf16 (or E4M3) values of 16 bytes that are not finite, of key `rel` from the first such
// tile's first on, and makes them zero.
template <bool E4M3>
__device__ __noinline__ uint4 note_bad(uint4 v, uint32_t* record, volatile uint32_t* any, uint32_t mark, int rel) {
  constexpr int kPerWord = E4M3 ? 4 : 2, kBits = 32 / kPerWord;
  constexpr uint32_t kValue = E4M3 ? 0xFFu : 0xFFFFu, kNot = E4M3 ? 0x7Fu : 0x7F80u;
  uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
#pragma unroll 1
    for (int k = 0; k < kPerWord; ++k) {
      if (((u[e] >> (k * kBits)) & kNot) != kNot) continue;
      u[e] &= ~(kValue << (k * kBits));
      atomicMax(record + e * kPerWord + k, mark | (1023u - static_cast<uint32_t>(rel)));
      *any = mark;
    }
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}
template <bool E4M3>
__device__ __forceinline__ bool has_bad(uint4 v) {
  constexpr uint32_t kNot = E4M3 ? 0x7F7F7F7Fu : 0x7F807F80u, kOne = E4M3 ? 0x01010101u : 0x00800080u;
  constexpr uint32_t kTop = E4M3 ? 0x80808080u : 0x80008000u;
  return ((((v.x & kNot) + kOne) | ((v.y & kNot) + kOne) | ((v.z & kNot) + kOne) | ((v.w & kNot) + kOne)) & kTop) != 0;
}
// The first key of the column that is not finite (none: beyond every key).
__device__ __forceinline__ int first_bad(const uint32_t* record, const Walk& w, int seen, int col) {
  const uint32_t x = record[col];
  return (x & ~1023u) == bad_mark(w.index) ? seen / BN * BN + static_cast<int>(1023u - (x & 1023u)) : 0x7fffffff;
}

struct Misc {
  uint8_t bad[kBadSlots][2];  // slabs of each step's tiles whose pages lie outside the cache
  uint32_t tmem;
  int abort;
  uint32_t any_bad[2];
  struct {
    long long offset;
    int g, head, i;
  } start;
};
static_assert(sizeof(Misc) <= 80, "misc");

constexpr int kPartRows = kPagedAttnPartRows;
__host__ __device__ constexpr size_t part_floats(int D) { return paged_attn_part_floats(D); }

// ------------------------------------------------------------------ the kernel

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                      const __grid_constant__ CUtensorMap tv, const PagedAttnArgs a) {
  using L = Layout<D, E4M3>;
  constexpr int NS = L::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];  // (swizzled tiles; there is no other shared memory)
  uint8_t* qs = smem;
  uint8_t* ring = smem + L::kRing;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBars);  // [NS] stage loaded
  uint64_t* raw = full + NS;                                     // [NS] loaded, to be looked through (bf16) or converted (E4M3)
  uint64_t* looked = raw + NS;                                   // [NS] and looked through
  uint64_t* q_full = looked + NS;                                // queries loaded
  uint64_t* p_full = q_full + 1;                                 // [2] P_x written
  uint64_t* joined = p_full + 2;                                 // [4] chain b's maxima and sums there
  uint64_t* written = joined + 4;                                // [2] epilogue of segment i done: written[i & 1]
  uint64_t* fin = written + 2;                                   // every MMA done
  uint64_t* done = fin + 1;                                      // [kDone] MMA batch n done: done[n % kDone]
  uint32_t* records = reinterpret_cast<uint32_t*>(smem + L::kBadKey);  // [2][D]
  float* s_ml = reinterpret_cast<float*>(smem + L::kMl);         // chain b's maxima and sums
  Misc& misc = *reinterpret_cast<Misc*>(smem + L::kMisc);
  volatile int* abort_flag = &misc.abort;

  const int warp = warp_id(), lane = lane_id(), tid = threadIdx.x;
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(full + s, E4M3 ? kLoaders - 1 : 1);
      mbar_init(raw + s, 1);
      mbar_init(looked + s, kLoaders - 1);
    }
    mbar_init(q_full, E4M3 ? kLoaders - 1 : 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(p_full + x, 4);
      mbar_init(written + x, 8);
      misc.any_bad[x] = 0;
    }
    for (int x = 0; x < 4; ++x) mbar_init(joined + x, 1);
    mbar_init(fin, 1);
    for (int n = 0; n < L::kDone; ++n) mbar_init(done + n, 1);
    *abort_flag = 0;
    misc.start.g = -1;
    fence_mbar_init();
  }
  if (tid < 2 * D) records[tid] = 0;
  if (tid < 2 * kBadSlots) (&misc.bad[0][0])[tid] = 0;
  if (!E4M3 && a.heads * a.tokens < BM) {  // rows of the query tiles that no load fills
    for (int i = tid; i < 2 * L::kTileBytes / 16; i += kThreads) st_shared16(qs + 16 * i, make_uint4(0u, 0u, 0u, 0u));
    fence_proxy_async_smem();
  }
  pdl_begin();

  // ---- this CTA's share: thread t sums sequences [t * per, (t + 1) * per)
  const int per = (a.G + kThreads - 1) / kThreads, segs = a.Hkv * a.chunks;
  long long own = 0;
  for (int k = 0; k < per; ++k) {
    Seq s;
    const int g = tid * per + k;
    if (g < a.G && load_seq(a, g, s, blockIdx.x == 0)) own += positions_of(a, s);
  }
  long long upto = own;
  long long* sums = reinterpret_cast<long long*>(s_ml);  // (not in use yet)
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += y;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  long long all = 0;
#pragma unroll
  for (int k = 0; k < kThreads / 32; ++k) {
    if (k < warp) upto += sums[k];
    all += sums[k];
  }
  if (blockIdx.x == 0 && a.places != nullptr) {  // where each sequence begins, for the join
    long long at = upto - own;
    for (int k = 0; k < per; ++k) {
      Seq s;
      const int g = tid * per + k;
      if (g >= a.G) break;
      a.places[g] = at;
      if (load_seq(a, g, s, false)) at += positions_of(a, s);
    }
    if (tid == 0) a.places[a.G] = all;
  }
  all *= segs;
  const int shares = static_cast<int>(min(all, static_cast<long long>(gridDim.x)));
  const bool busy = static_cast<int>(blockIdx.x) < shares;
  const long long lo = busy ? all * blockIdx.x / shares : 0, hi = busy ? all * (blockIdx.x + 1) / shares : 0;
  if (busy && lo >= (upto - own) * segs && lo < upto * segs) {
    long long base = (upto - own) * segs;
    for (int k = 0; k < per; ++k) {
      Seq s;
      const int g = tid * per + k;
      if (g >= a.G || !load_seq(a, g, s, false)) continue;
      const long long size = positions_of(a, s);
      if (lo < base + size * segs) {
        const long long in = lo - base;
        misc.start.g = g;
        misc.start.head = static_cast<int>(in / size);
        misc.start.offset = in - misc.start.head * size;
        break;
      }
      base += size * segs;
    }
  }
  if (warp == kMmaWarp && busy) {
    tmem_alloc(&misc.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  Walk w = {};
  bool more = busy && misc.start.g >= 0;
  if (more && warp == 0) {  // the pair, 32 places at a time
    Seq s;
    load_seq(a, misc.start.g, s, false);
    const int pairs = units_of(a, s) / 2;
    int first = 0, n = pairs + 1;  // the last k in [first, first + n) with pairs_upto(k) <= offset
    while (n > 1) {
      const int step = (n + 31) / 32, k = first + lane * step;
      const bool in = lane * step < n && pairs_upto(a, s, k) <= misc.start.offset;
      const int at = 31 - __clz(__ballot_sync(0xffffffffu, in));  // (lane 0 is in)
      n = min(step, n - at * step);
      first += at * step;
    }
    if (lane == 0) {
      misc.start.i = first;
      misc.start.offset -= pairs_upto(a, s, first);
    }
  }
  __syncthreads();
  int part_from = -1;  // the share in which the first segment begins, if that is not this one
  if (more) {
    w.g = misc.start.g;
    w.head = misc.start.head;
    w.i = misc.start.i;
    load_seq(a, w.g, w.s, false);
    const int units = units_of(a, w.s);
    w.i = min(w.i, units / 2 + (units & 1) - 1);
    set_segment(a, w);
    w.t0 = static_cast<int>(misc.start.offset);
    w.left = hi - lo;
    w.count = static_cast<int>(min(static_cast<long long>(w.steps - w.t0), w.left));
    if (w.t0 > 0 && w.count > 0 && w.t0 + w.count == w.steps) {
      part_from = share_of(lo - w.t0, all, shares);
    }
    if (tid == 0) {
      a.ends[blockIdx.x] = make_int4(part_from >= 0 ? w.g : -1, w.head, w.i, part_from);
    }
    if (w.count <= 0) more = next_segment(a, w);
    w.index = 0;
  } else if (tid == 0) {
    a.ends[blockIdx.x] = make_int4(-1, 0, 0, 0);
  }
  if (!busy) return;
  const uint32_t tmem = misc.tmem;  // S_a +0, S_b +128, O_a +256, O_b +256+D
  const int group = a.Hq / a.Hkv;
  // MMA batches of a segment, from number `base` on: base QK_a(0) QK_b(0); base + 2 j + x + 1
  // PV_x(j) QK_x(j + 1).  Each ends in one commit, which signals every earlier MMA, too: it tells
  // the softmax that S_x is there, the epilogue that O_x is final, the loads that tiles are read.
  int base = 0;
  auto wait_batch = [&](int n) { return warp_wait(done + n % L::kDone, (n / L::kDone) & 1, abort_flag, a.status); };

  if (warp >= kFirstLoader && warp < kMmaWarp) {
    // ------------------------------------------------------------ loads
    // pages of a window's tiles: lane i has the row in the caches of the i-th slab, -1 where
    // there is nothing; the window behind it is asked for when one is begun
    const int slabs_per_page = a.page / kSlab, shift = 31 - __clz(slabs_per_page);
    int found[3] = {-1, -1, -1}, window = -1;
    uint32_t outside[3] = {0, 0, 0};  // slabs inside the sequence whose page is none
    auto look_up = [&](int win, int& row, bool& out) {
      const long long slab = static_cast<long long>(win) * 32 + lane;
      row = -1;
      out = false;
      if (slab * kSlab >= w.s.keys) return;
      const int j = static_cast<int>(slab >> shift);
      const int at = a.row_of != nullptr ? a.row_of[w.g] : w.g;
      const int pid = a.table[static_cast<size_t>(at) * a.max_pages + j];
      if (pid < 0 || pid >= a.num_pages) {
        out = true;
        return;
      }
      row = (pid * a.Hkv + w.head / a.chunks) * a.page + (static_cast<int>(slab) & (slabs_per_page - 1)) * kSlab;
    };
    auto begin_windows = [&](int tile) {
      window = tile / kWindow;
      bool out;
      found[0] = -1;
      outside[0] = 0;
      look_up(window, found[1], out);
      outside[1] = __ballot_sync(0xffffffffu, out);
      look_up(window + 1, found[2], out);
      outside[2] = __ballot_sync(0xffffffffu, out);
    };
    // (tiles come in order; a V tile is at most two behind the last K tile)
    auto to_window = [&](int tile) {
      if (tile / kWindow > window) {
        ++window;
        found[0] = found[1], found[1] = found[2];
        outside[0] = outside[1], outside[1] = outside[2];
        bool out;
        look_up(window + 1, found[2], out);
        outside[2] = __ballot_sync(0xffffffffu, out);
      }
    };
    // Ring items of a segment, in the order in which the MMA warp asks for them: the chains' first K,
    // then for every step and chain its V and its next K (a pair's tiles come with chain a).
    int it = 0;  // items so far
    if (warp == kFirstLoader) {
      // ---------------------------------------------------------- TMA
      if (elect_one()) {
        if (!E4M3) tma_prefetch_desc(&tq);
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
      }
      __syncwarp();
      // Two items at a time, as the MMA warp takes them: lanes 0-15 load the first one's boxes (a
      // page's rows, 128 bytes wide), lanes 16-31 the second's.
      constexpr int kBoxSubs = E4M3 ? 1 : L::kSub, kBoxBytes = E4M3 ? D : 128;
      const int half = lane >> 4, box = (lane & 15) / kBoxSubs, sub = (lane & 15) % kBoxSubs, boxes = BN / a.page;
      const uint32_t to = smem_u32(ring) + (E4M3 ? L::kRaw : sub * L::kSubBytes) + box * a.page * kBoxBytes;
      int reader = 0, q_reader = 0;  // lane i: the last batch that reads stage i; the last that reads the queries
      int next_st = 0, step = 0;
      uint32_t raw_used = 0, raw_parity = 0;  // bf16, of each stage: a tile went to `raw`; the last one's parity
      uint32_t dirty = 0;                     // steps (and chains) whose `bad` is not zero
      auto issue = [&](bool first, bool first_k, int first_tile, int first_read, bool look, bool second, int second_tile,
                       int second_read) -> bool {
        const int st0 = next_st, st1 = first ? (st0 + 1 == NS ? 0 : st0 + 1) : st0;
        const int st = half ? st1 : st0;
        const bool mine = half ? second : first;
        const int n = __shfl_sync(0xffffffffu, reader, st);
        const bool used = it + (half && first ? 1 : 0) >= NS;
        bool ok = !mine || !used || mbar_try_wait(done + n % L::kDone, (n / L::kDone) & 1);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = !mine || !used || mbar_wait(done + n % L::kDone, (n / L::kDone) & 1, abort_flag, a.status);
          if (!__all_sync(0xffffffffu, ok)) return false;
        }
        if (second) to_window(second_tile);
        const int tile = half ? second_tile : first_tile;
        const bool behind = tile / kWindow != window;
        const int from = (tile % kWindow) * kSlabs + (box < boxes ? box : 0) * slabs_per_page;
        const int r0 = __shfl_sync(0xffffffffu, found[0], from), r1 = __shfl_sync(0xffffffffu, found[1], from);
        const int row = behind ? r0 : r1;
        const bool to_raw = E4M3 || (look && half == 0);
        uint64_t* bar = (to_raw ? raw : full) + st;
        if (mine && (lane & 15) == 0) {
          mbar_expect_tx(bar, E4M3 ? BN * D : L::kTileBytes);
          if (!E4M3 && to_raw) mbar_arrive(full + st);  // `full` keeps its turn: such tiles complete it empty
        }
        __syncwarp();
        if (mine && box < boxes) {  // (a row past the tensor's end reads zeros)
          const bool is_k = half || first_k;
          tma_load_2d_at(to + st * L::kStageBytes, is_k ? &tk : &tv, sub * 64, row < 0 ? a.rows : row, bar);
        }
        __syncwarp();
        if (!E4M3 && look) {
          raw_parity ^= ((raw_used >> st0) & 1u) << st0;
          raw_used |= 1u << st0;
        }
        if (first && lane == st0) reader = first_read;
        if (second && lane == st1) reader = second_read;
        it += (first ? 1 : 0) + (second ? 1 : 0);
        next_st = second ? (st1 + 1 == NS ? 0 : st1 + 1) : st1;
        return true;
      };
      // slabs of the tile whose pages are none, for the softmax; in front of the load that it goes with
      auto tell = [&](int tile, int at, int x) {
        to_window(tile);
        const uint32_t out = ((tile / kWindow != window ? outside[0] : outside[1]) >> ((tile % kWindow) * kSlabs)) & 0xffu;
        const int slot = (at % kBadSlots) * 2 + x;
        if (out == 0 && ((dirty >> slot) & 1u) == 0) return;
        dirty = (dirty & ~(1u << slot)) | (out ? 1u << slot : 0u);
        if (lane == 0) {
          (&misc.bad[0][0])[slot] = static_cast<uint8_t>(out);
          if (out) atomicOr(a.status, DEV_BOUNDS);
        }
        __syncwarp();
      };
      bool ok = true;
      for (; ok && more; more = next_segment(a, w)) {
        const bool single = w.single;
        const int count = w.count, n0 = steps_of(w, 0), n1 = steps_of(w, 1), tile0 = tile_of(w, 0, 0);
        const int kn0 = single ? n0 : count, first_look = seen_by_all(a, w) / BN;
        begin_windows(tile0);
        if (w.index > 0) ok = wait_batch(q_reader);
        if (!ok) break;
        if (!E4M3 && elect_one()) {
          // a box is tokens x heads rows; tokens behind the sequence's are other ones' or zeros
          const int units = single ? 1 : 2;
          mbar_expect_tx(q_full, units * L::kSub * 128 * a.heads * a.tokens);
          const int head = w.head / a.chunks * group + w.head % a.chunks * a.heads;
          for (int u = 0; u < units; ++u)
            for (int s = 0; s < L::kSub; ++s)
              tma_load_3d(qs + u * L::kTileBytes + s * L::kSubBytes, &tq, s * 64, head, w.s.cu + (2 * w.i + u) * a.tokens, q_full);
        }
        __syncwarp();
        tell(tile0, step, 0);
        if (!single) tell(tile0, step, 1);
        if (single && n1 > 0) tell(tile0 + 1, step, 1);
        ok = issue(true, true, tile0, base, false, single && n1 > 0, tile0 + 1, base);
        // (one call of `issue` in the loop: its code is long)
        const int turns = single ? 2 * count : count;
#pragma unroll 1
        for (int i = 0; ok && i < turns; ++i) {
          const int j = single ? i >> 1 : i, x = single ? i & 1 : 0;
          if (a.fault && j >= 1) ok = false;  // test only: starve the MMA warp
          const bool v = !single || j < (x ? n1 : n0), k = j + 1 < (x ? n1 : kn0);
          const int v_tile = tile0 + i, k_tile = v_tile + (single ? 2 : 1);
          if (k) {
            tell(k_tile, step + j + 1, x);
            if (!single) tell(k_tile, step + j + 1, 1);
          }
          // V_x(j) is read by batch base + 2 j + x + 1, K_x(j + 1) too (a pair's by chain b's)
          const int read = base + 2 * j + (single ? x + 1 : 2);
          if (ok && v) ok = issue(true, false, v_tile, read, v_tile >= first_look, k, k_tile, read);
        }
        step += count;
        q_reader = base + 2 * (count - 1);
        base += 2 * count + 1;
      }
      if (*abort_flag)
        for (int i = max(it - NS, 0); i < it; ++i) {
          if (!E4M3) drain_wait(full + i % NS, (i / NS) & 1);
          if (E4M3) drain_wait(raw + i % NS, (i / NS) & 1);
          if (!E4M3 && ((raw_used >> (i % NS)) & 1u)) drain_wait(raw + i % NS, (raw_parity >> (i % NS)) & 1u);
        }
    } else {
      // ---------------------------------------------------------- tiles on their way to the MMA
      // bf16: V tiles that masks cut are looked through.  E4M3: every tile is converted to f16
      // (exact: every E4M3 value is an f16 value), looked through where that is asked for, and
      // the queries, too.
      constexpr int kHelp = 32 * (kLoaders - 1), kSegsRow = D / 8;
      const int hw = warp - kFirstLoader - 1, me = 32 * hw + lane;
      uint32_t raw_parity = 0;  // of each stage
      int q_reader = 0;
      bool ok = true;
      for (; ok && more; more = next_segment(a, w)) {
        const bool single = w.single;
        const int count = w.count, n0 = steps_of(w, 0), n1 = steps_of(w, 1), tile0 = tile_of(w, 0, 0);
        const int first_look = seen_by_all(a, w) / BN, mark = w.index & 1, keys = w.s.keys;
        // a record's last segment, two back, has been read when this one's is begun
        const bool looks = first_look <= last_tile(w);
        if (looks && w.index >= 2) ok = warp_wait(written + mark, ((w.index - 2) / 2) & 1, abort_flag, a.status);
        if (!ok) break;
        if constexpr (!E4M3) {
          // items in front of step j
          auto items_until = [&](int j) {
            return single ? 2 * j + 1 + (n1 > 0 ? 1 + min(j, n1) + min(j, n1 - 1) : 0) : 2 * j + 1;
          };
          const int jl = looks ? max(0, single ? (first_look - tile0) >> 1 : first_look - tile0) : count;
          int i = it + items_until(jl);
          for (int j = jl; ok && j < count; ++j) {
            for (int x = 0; x < (single ? 2 : 1); ++x) {
              const int tile = tile0 + (single ? 2 * j + x : j), st = i % NS;
              if (single && j >= (x ? n1 : n0)) continue;
              i += j + 1 < (single ? (x ? n1 : n0) : count) ? 2 : 1;
              if (tile < first_look) continue;
              ok = warp_wait(raw + st, (raw_parity >> st) & 1u, abort_flag, a.status);
              if (!ok) break;
              raw_parity ^= 1u << st;
              uint8_t* v = ring + st * L::kStageBytes;
              for (int c = me; c < BN * kSegsRow; c += kHelp) {
                const int r = c / kSegsRow, sg = c % kSegsRow;
                uint8_t* at = v + swz_offset(r, sg);
                if (r >= keys - tile * BN) {
                  st_shared16(at, make_uint4(0u, 0u, 0u, 0u));
                  continue;
                }
                const uint4 q = ld_shared16(at);
                if (has_bad<false>(q))
                  st_shared16(at, note_bad<false>(q, records + mark * D + sg * 8, misc.any_bad + mark, bad_mark(w.index),
                                                  (tile - first_look) * BN + r));
              }
              fence_proxy_async_smem();  // generic writes -> tensor-core operand reads
              __syncwarp();
              if (lane == 0) mbar_arrive(looked + st);
            }
          }
          it += single ? 2 * n0 + (n1 > 0 ? 2 * n1 : 0) : 2 * count;
        } else {
          if (w.index > 0) ok = wait_batch(q_reader);
          if (!ok) break;
          // queries: bf16 to f16 through registers, kAtOnce chunks side by side
          constexpr int kChunks = BM * kSegsRow, kAtOnce = 6;
          const int chunk0 = w.head % a.chunks * a.heads, head = w.head / a.chunks * group + chunk0;
#pragma unroll 1
          for (int c0 = me; c0 < (single ? 1 : 2) * kChunks; c0 += kAtOnce * kHelp) {
            uint4 qw[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
              const int c = c0 + kHelp * k, r = c % kChunks / kSegsRow, sg = c % kSegsRow;
              const int t = r / a.heads, h = r - t * a.heads, tok = (2 * w.i + c / kChunks) * a.tokens + t;
              qw[k] = make_uint4(0u, 0u, 0u, 0u);
              if (c < 2 * kChunks && t < a.tokens && tok < w.s.n && chunk0 + h < group)
                qw[k] = ld_global16(a.q + static_cast<size_t>(w.s.cu + tok) * a.q_stride + static_cast<size_t>(head + h) * D + sg * 8);
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
              const int c = c0 + kHelp * k;
              if (c < 2 * kChunks)
                st_shared16(qs + c / kChunks * L::kTileBytes + swz_offset(c % kChunks / kSegsRow, c % kSegsRow),
                            make_uint4(bf16x2_to_f16x2(qw[k].x), bf16x2_to_f16x2(qw[k].y), bf16x2_to_f16x2(qw[k].z),
                                       bf16x2_to_f16x2(qw[k].w)));
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(q_full);
          // One row of 16-byte chunks per kSegs lanes.  Only these lanes touch a row's bytes and its f16
          // line; where both share memory (D = 128) a __syncwarp between reads and writes orders them.
          constexpr int kSegs = D / 16, kRows = 32 / kSegs, kGroups = BN / kRows, kTurns = (kGroups + kLoaders - 2) / (kLoaders - 1);
          const int sub = lane / kSegs, seg = lane % kSegs;
          const int heads_of = single ? 1 + (n1 > 0 ? 1 : 0) : 1;
          const int turns = heads_of + (single ? 4 : 2) * count;
#pragma unroll 1
          for (int i = 0; ok && i < turns; ++i) {
            // item i: the first K, then (V, next K) of each step and chain
            const int m = i - heads_of, u = m >> 1, j = single ? u >> 1 : u, x = single ? u & 1 : 0;
            const bool is_k = m < 0 || (m & 1);
            if (m >= 0 && j + (is_k ? 1 : 0) >= (single ? (x ? n1 : n0) : count)) continue;
            const int tile = tile0 + u, st = it % NS;  // (of a V tile)
            const bool look = !is_k && tile >= first_look;
            ok = warp_wait(raw + st, (it / NS) & 1, abort_flag, a.status);
            if (!ok) break;
            ++it;
            uint8_t* stage = ring + st * L::kStageBytes;
            uint8_t* from = stage + L::kRaw;
            if (look) {
#pragma unroll 1
              for (int k = 0; k < kTurns; ++k) {
                const int r = (hw + (kLoaders - 1) * k) * kRows + sub;
                if (r >= BN) continue;
                uint4 q = ld_shared16(from + r * D + seg * 16);
                if (r >= keys - tile * BN)
                  q = make_uint4(0u, 0u, 0u, 0u);
                else if (has_bad<true>(q))  // NaN codes (there are no infinities)
                  q = note_bad<true>(q, records + mark * D + seg * 16, misc.any_bad + mark, bad_mark(w.index),
                                     (tile - first_look) * BN + r);
                st_shared16(from + r * D + seg * 16, q);
              }
              __syncwarp();
            }
            uint4 v[kTurns];
#pragma unroll
            for (int k = 0; k < kTurns; ++k)
              if (hw + (kLoaders - 1) * k < kGroups) v[k] = ld_shared16(from + ((hw + (kLoaders - 1) * k) * kRows + sub) * D + seg * 16);
            __syncwarp();
#pragma unroll
            for (int k = 0; k < kTurns; ++k) {
              if (hw + (kLoaders - 1) * k < kGroups) {
                const int r = (hw + (kLoaders - 1) * k) * kRows + sub;
                uint4 p, q;
                e4m3x4_to_f16x4(v[k].x, p.x, p.y);
                e4m3x4_to_f16x4(v[k].y, p.z, p.w);
                e4m3x4_to_f16x4(v[k].z, q.x, q.y);
                e4m3x4_to_f16x4(v[k].w, q.z, q.w);
                st_shared16(stage + swz_offset(r, 2 * seg), p);
                st_shared16(stage + swz_offset(r, 2 * seg + 1), q);
              }
            }
            fence_proxy_async_smem();  // generic writes -> tensor-core operand reads
            __syncwarp();
            if (lane == 0) mbar_arrive(full + st);
          }
          q_reader = base + 2 * (count - 1);
          base += 2 * count + 1;
        }
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issue
    constexpr uint32_t idesc_qk = E4M3 ? idesc_f16(BM, BN, false, false) : idesc_bf16(BM, BN, false, false);
    constexpr uint32_t idesc_pv = E4M3 ? idesc_f16(BM, D, false, true) : idesc_bf16(BM, D, false, true);
    // The tensor core holds one or two MMAs ahead and the issue of a batch ends as its last ones
    // begin: whatever stands between that and the next batch's issue leaves it idle.  So stages,
    // parities and barriers of the next batch are worked out in front of the present one's issue.
    const uint32_t ring_addr = smem_u32(ring), q_addr = smem_u32(qs);
    uint32_t look_parity = 0;       // of each stage's `looked`
    int next_st = 0, dn = 0;        // the next ring item's stage; the next batch's barrier
    uint32_t next_ph = 0, step = 0;
    struct Item {
      int st;
      uint32_t ph;
      bool look;  // a V tile that is looked through
    };
    auto take = [&](bool look) {
      const Item i = {next_st, next_ph, look};
      if (++next_st == NS) next_st = 0, next_ph ^= 1;
      return i;
    };
    auto try_item = [&](const Item& i) {
      return i.look ? mbar_try_wait(looked + i.st, (look_parity >> i.st) & 1) : mbar_try_wait(full + i.st, i.ph);
    };
    auto wait_item = [&](const Item& i) {
      return i.look ? warp_wait(looked + i.st, (look_parity >> i.st) & 1, abort_flag, a.status)
                    : warp_wait(full + i.st, i.ph, abort_flag, a.status);
    };
    auto issue_qk = [&](int x, int st) {
      const uint32_t kb = ring_addr + st * L::kStageBytes, qb = q_addr + (w.single ? 0 : x) * L::kTileBytes;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk >> 2) * L::kSubBytes + (kk & 3) * 32;
        umma_ss(tmem + x * 128, sdesc_sw128(qb + off, 16, 1024), sdesc_sw128(kb + off, 16, 1024), idesc_qk, kk > 0);
      }
    };
    auto issue_pv = [&](int x, int st, bool first) {
      const uint32_t vb = ring_addr + st * L::kStageBytes;
#pragma unroll
      for (int kk = 0; kk < BN / 16; ++kk)
        umma_ts(tmem + 256 + x * D, tmem + x * 128 + kk * 8, sdesc_sw128(vb + kk * 16 * 128, L::kSubBytes, 1024), idesc_pv,
                (!first || kk > 0) ? 1u : 0u);
    };
    bool ok = true;
    for (; ok && more; more = next_segment(a, w)) {
      const bool single = w.single;
      const int count = w.count, n0 = steps_of(w, 0), n1 = steps_of(w, 1);
      // steps from look[x] on have a V tile that is looked through
      const int seen = seen_by_all(a, w), first = seen / BN - tile_of(w, 0, 0);
      const int look0 = E4M3 ? count : single ? (first + 1) >> 1 : first, look1 = E4M3 ? count : first >> 1;
      Item k0 = take(false), k1 = single && n1 > 0 ? take(false) : k0;
      ok = warp_wait(q_full, w.index & 1, abort_flag, a.status) && wait_item(k0) && wait_item(k1);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        if (n0 > 0) issue_qk(0, k0.st);
        if (n1 > 0) issue_qk(1, k1.st);
        umma_commit(done + dn);
      }
      __syncwarp();
      dn = dn + 1 == L::kDone ? 0 : dn + 1;
      Item v0 = k0, v1 = k0;
      // the chains' items of step j: chain a's V, next K, and (an odd unit's) chain b's
      auto take0 = [&](int j) {
        if (!single || j < n0) v0 = take(j >= look0);
        if (j + 1 < (single ? n0 : count)) k0 = take(false);
      };
      auto take1 = [&](int j) {
        if (single) {
          if (j < n1) v1 = take(j >= look1);
          if (j + 1 < n1) k1 = take(false);
        } else {
          v1 = v0, k1 = k0;
        }
      };
      take0(0);
#pragma unroll 1
      for (int j = 0; ok && j < count; ++j, ++step) {
        {
          const bool mine = j < n0, next = j + 1 < n0, loads_v = !single || mine, loads_k = j + 1 < (single ? n0 : count);
          bool ready = mbar_try_wait(p_full, step & 1);
          if (loads_v) ready &= try_item(v0);
          if (loads_k) ready &= mbar_try_wait(full + k0.st, k0.ph);
          if (!__all_sync(0xffffffffu, ready))
            ok = (!loads_v || wait_item(v0)) && (!loads_k || wait_item(k0)) && warp_wait(p_full, step & 1, abort_flag, a.status);
          if (!ok) break;
          if (loads_v && v0.look) look_parity ^= 1u << v0.st;
          uint64_t* bar = done + dn;
          dn = dn + 1 == L::kDone ? 0 : dn + 1;
          take1(j);
          const int vs = v0.st, ks = k0.st;
          tc_fence_after();
          if (elect_one()) {
            if (mine) issue_pv(0, vs, j == 0);
            if (next) issue_qk(0, ks);
            umma_commit(bar);
          }
          __syncwarp();
        }
        {
          const bool mine = j < n1, next = j + 1 < n1;
          bool ready = mbar_try_wait(p_full + 1, step & 1);
          if (single && mine) ready &= try_item(v1);
          if (single && next) ready &= mbar_try_wait(full + k1.st, k1.ph);
          if (!__all_sync(0xffffffffu, ready))
            ok = (!single || !mine || wait_item(v1)) && (!single || !next || wait_item(k1)) &&
                 warp_wait(p_full + 1, step & 1, abort_flag, a.status);
          if (!ok) break;
          if (single && mine && v1.look) look_parity ^= 1u << v1.st;
          uint64_t* bar = done + dn;
          dn = dn + 1 == L::kDone ? 0 : dn + 1;
          const int vs = v1.st, ks = k1.st;
          if (j + 1 < count) take0(j + 1);
          tc_fence_after();
          if (elect_one()) {
            if (mine) issue_pv(1, vs, j == 0);
            if (next) issue_qk(1, ks);
            umma_commit(bar);
          }
          __syncwarp();
        }
      }
    }
    if (elect_one()) umma_commit(fin);
    __syncwarp();
    drain_wait(fin, 0);
  } else {
    // ------------------------------------------------------------ softmax
    const int x = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + x * 128 + lane_off;
    const uint32_t tO = tmem + 256 + x * D + lane_off;
    const float sl2 = a.scale_log2;
    // this thread's row of a segment: its token, the head inside the KV head, whether it exists, and
    // the keys it sees (a row that does not exist sees what every row sees and costs no masks)
    struct Row {
      int tok, head, limit;
      bool live;
    };
    auto row_of = [&](const Walk& w) {
      const int t = row / a.heads;
      Row r;
      r.tok = static_cast<int>(min((2LL * w.i + (w.single ? 0 : x)) * a.tokens + t, 0x7fffffffLL));
      r.head = w.head % a.chunks * a.heads + row - t * a.heads;
      r.live = t < a.tokens && r.tok < w.s.n && r.head < group;
      r.limit = r.live && a.causal ? w.s.keys - w.s.n + r.tok + 1 : w.s.keys;
      return r;
    };
    int step = 0;
    uint32_t join_parity = 0;
    bool ok = true;
    for (; ok && more; more = next_segment(a, w)) {
      const Row mine_row = row_of(w);
      const int limit = mine_row.limit;
      const int mine = __all_sync(0xffffffffu, !mine_row.live) ? 0 : steps_of(w, x), count = w.count;
      int ahead = limit - tile_of(w, x, 0) * BN;  // keys that the row sees from the tile's first on
      const int stride = w.single ? 2 * BN : BN;
      const int folded = fold(w, lane);
      float m_run = -INFINITY, l_f32 = 0.f, l_mul = 0.f;
      for (int j = 0; j < count; ++j, ++step, ahead -= stride) {
        if (!wait_batch(j == 0 ? base : base + 2 * j + x - 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (j >= mine) {  // P of these rows is never read, or not used
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full + x);
          continue;
        }
        const int valid = ahead;
        const uint32_t bad = misc.bad[step % kBadSlots][x];
        if (bad != 0 || !__all_sync(0xffffffffu, valid >= BN)) mask_scores(tS, valid, bad);
        float s[64];
        uint32_t* su = reinterpret_cast<uint32_t*>(s);
        tmem_ld32(tS + 64, su);
        tmem_ld32(tS + 96, su + 32);
        tmem_ld_wait();
        const float mx_hi = max64(s);
        tmem_ld32(tS + 0, su);
        tmem_ld32(tS + 32, su + 32);
        tmem_ld_wait();
        const float m_new = fmaxf(max64(s), mx_hi) * sl2;
        // The reference maximum moves only when the tile's exceeds it by more than the
        // threshold; TMEM loads and stores are the whole warp's, so all rows enter when one does.
        const bool need = m_new > m_run + kThreshold<E4M3>;  // (the first maximum of a row, too)
        if (__any_sync(0xffffffffu, need)) {
          if (j > 0) {
            const float f = need ? ex2(m_run - m_new) : 1.f;
            l_f32 *= f;
            l_mul *= f;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tmem_ld16(tO + c * 16, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(f * __uint_as_float(o[i]));
              tmem_st16(tO + c * 16, o);
            }
          }
          if (need) m_run = m_new;
        }
        // p = 2^(s c - m).  Two row sums: the fp32 weights (lse) and the rounded ones the product
        // multiplies by (the output is normalised by those, which keeps its error smaller).
        const float m_ref = m_run == -INFINITY ? 0.f : m_run;
        const uint64_t c2 = f2_pack(sl2, sl2), nm2 = f2_pack(-m_ref, -m_ref);
        uint64_t accf[4] = {0ull, 0ull, 0ull, 0ull}, accb[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 1) {
            tmem_ld32(tS + 64, su);
            tmem_ld32(tS + 96, su + 32);
            tmem_ld_wait();
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float x0, x1;
              f2_unpack(f2_fma(f2_pack(s[32 * c + 2 * i], s[32 * c + 2 * i + 1]), c2, nm2), x0, x1);
              const float p0 = ex2(x0), p1 = ex2(x1);
              pk[i] = E4M3 ? pack_f16(p0, p1) : pack_bf16(p0, p1);
              accf[i & 3] = f2_add(accf[i & 3], f2_pack(p0, p1));
              if constexpr (E4M3) {
                const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&pk[i]));
                accb[i & 3] = f2_add(accb[i & 3], f2_pack(r.x, r.y));
              } else {
                accb[i & 3] = f2_add(accb[i & 3], f2_pack(__uint_as_float(pk[i] << 16), __uint_as_float(pk[i] & 0xFFFF0000u)));
              }
            }
            tmem_st16(tS + h * 32 + c * 16, pk);
          }
        }
        l_f32 += sum8(accf);
        l_mul += sum8(accb);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + x);
      }
      // ---------------------------------------------------------- epilogue
      if (ok) ok = wait_batch(base + 2 * count - 1 + x);
      if (!ok) break;
      w = unfold(folded);
      const Row r = row_of(w);
      const bool idle = __all_sync(0xffffffffu, !r.live), live = r.live;
      const bool had = has_tile(w, x, 0);  // this chain wrote O
      float fa = 1.f, fb = 0.f;
      if (w.single) {  // chain a joins the two
        if (x == 1) {
          s_ml[row] = m_run;
          s_ml[BM + row] = l_mul;
          s_ml[2 * BM + row] = l_f32;
          __syncwarp();
          if (lane == 0) mbar_arrive(joined + (warp & 3));
        } else {
          ok = wait_batch(base + 2 * count) && warp_wait(joined + (warp & 3), join_parity, abort_flag, a.status);
          if (!ok) break;
          join_parity ^= 1;
          const float m_b = s_ml[row], top = fmaxf(m_run, m_b);
          fa = m_run == -INFINITY ? 0.f : ex2(m_run - top);
          fb = m_b == -INFINITY ? 0.f : ex2(m_b - top);
          // (sums of scores that are NaN stay NaN)
          l_mul = fmaf(l_mul, fa, s_ml[BM + row] * fb);
          l_f32 = fmaf(l_f32, fa, s_ml[2 * BM + row] * fb);
          m_run = top;
        }
      }
      tc_fence_after();
      if (!idle && !(w.single && x == 1)) {
        const bool b_too = w.single && has_tile(w, 1, 0);
        const uint32_t tOb = tmem + 256 + D + lane_off;
        const bool goes_on = w.t0 + w.count < w.steps, whole = w.t0 == 0 && !goes_on;
        const size_t out_row = static_cast<size_t>(w.s.cu + r.tok) * a.Hq + w.head / a.chunks * group + r.head;
        const bool finals = whole && a.whole == nullptr;
        // (the value scale by itself: its quotient by the sum may be too small for a normal float)
        const float inv = !finals ? 1.f : l_mul > 0.f || l_mul != l_mul ? 1.f / l_mul : 0.f;
        float* part = nullptr;
        if (!whole) {
          part = a.parts + (2 * static_cast<size_t>(blockIdx.x) + (goes_on ? 1 : 0)) * part_floats(D);
          const int at = x * BM + row;
          if (live) reinterpret_cast<float4*>(part)[at] = make_float4(m_run, l_mul, l_f32, 0.f);
          part += 4 * kPartRows + static_cast<size_t>(at) * D;
        } else if (!finals) {
          part = a.whole + 4 * static_cast<size_t>(a.T) * a.Hq + out_row * D;
          if (live) reinterpret_cast<float4*>(a.whole)[out_row] = make_float4(m_run, l_mul, l_f32, 0.f);
        }
        const int seen = seen_by_all(a, w);
        const bool spoiled = *static_cast<volatile uint32_t*>(misc.any_bad + (w.index & 1)) == bad_mark(w.index);
        const uint32_t* record = records + (w.index & 1) * D;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          float v[32];
          if (had) {
            tmem_ld32(tO + c * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(o[i]) * fa;
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.f;
          }
          if (b_too) {
            tmem_ld32(tOb + c * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = fmaf(__uint_as_float(o[i]), fb, v[i]);
          }
          if (live) {
            if (spoiled) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (first_bad(record, w, seen, c * 32 + i) < r.limit) v[i] = NAN;
            }
            if (finals) {
              uint4* dst = reinterpret_cast<uint4*>(a.out + out_row * D + c * 32);
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = E4M3 ? v[i] * inv * a.v_scale : v[i] * inv;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                dst[e] = make_uint4(pack_bf16(v[8 * e], v[8 * e + 1]), pack_bf16(v[8 * e + 2], v[8 * e + 3]),
                                    pack_bf16(v[8 * e + 4], v[8 * e + 5]), pack_bf16(v[8 * e + 6], v[8 * e + 7]));
            } else {
              float4* dst = reinterpret_cast<float4*>(part + c * 32);
#pragma unroll
              for (int e = 0; e < 8; ++e) dst[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
            }
          }
          __syncwarp();  // TMEM loads are the whole warp's
        }
        if (finals && live && a.lse != nullptr)
          a.lse[out_row] = l_f32 == 0.f ? -INFINITY : (m_run + log2f(l_f32)) * 0.6931471805599453f;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(written + (w.index & 1));
      base += 2 * count + 1;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// Which sequences a common beginning serves.  One CTA: it is a few reads and writes per sequence.
// Bounds that do not ascend from 0 to B leave every sequence by itself; a group of which fewer than
// two sequences reach the beginning's end, too.
constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const SharedPlanArgs a) {
  pdl_begin();
  const int tid = threadIdx.x, lane = lane_id();
  const long long room = static_cast<long long>(a.max_pages) * a.page;
  bool bad = tid == 0 && (a.starts[0] != 0 || a.starts[a.G] != a.B);
  for (int g = tid; g < a.G; g += kPlanThreads) bad = bad || a.starts[g] > a.starts[g + 1];
  for (int b = tid; b < a.B; b += kPlanThreads) {
    const int len = a.lens[b];
    const bool good = len >= 0 && len <= room;
    if (!good) atomicOr(a.status, DEV_BOUNDS);
    a.tail[b] = good ? len : 0;
    a.skip[b] = 0;
    a.group_of[b] = -1;
  }
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) atomicOr(a.status, DEV_BOUNDS);
  for (int g = tid; g <= a.G; g += kPlanThreads) a.cu[g] = bad ? 0 : a.starts[g];
  for (int g = warp_id(); g < a.G; g += kPlanThreads / 32) {
    const int lo = bad ? 0 : a.starts[g], hi = bad ? 0 : a.starts[g + 1], pages = a.shared[g];
    const bool good = pages >= 0 && pages <= a.max_pages;
    const int keys = good ? pages * a.page : 0;
    bool wrong = !good;
    int live = 0, leader = 0x7fffffff;
    for (int b = lo + lane; b < hi; b += 32) {
      const int len = a.tail[b];
      wrong = wrong || (len > 0 && len < keys);
      if (len > 0 && len >= keys) {
        ++live;
        leader = min(leader, b);
      }
    }
    live = __reduce_add_sync(0xffffffffu, live);
    leader = __reduce_min_sync(0xffffffffu, leader);
    if (wrong) atomicOr(a.status, DEV_BOUNDS);
    const bool use = live > 1 && keys > 0;
    if (lane == 0) {
      a.keys[g] = use ? keys : 0;
      a.leader[g] = use ? leader : 0;
    }
    for (int b = lo + lane; use && b < hi; b += 32) {
      const int len = a.tail[b];
      if (len == 0 || len < keys) continue;
      a.tail[b] = len - keys;
      a.skip[b] = pages;
      a.group_of[b] = g;
    }
  }
}

// Joins the parts of the segment that ends in share blockIdx.x / kJoinBlocks and begins in an
// earlier one, in the order of the shares: kJoinRows rows per block, 8 threads to a row.
constexpr int kJoinRows = 32;
constexpr int kJoinBlocks = kPartRows / kJoinRows;
template <int D, bool E4M3>
__global__ void __launch_bounds__(8 * kJoinRows) paged_attn_join_kernel(const PagedAttnArgs a) {
  pdl_begin();
  const int c1 = blockIdx.x / kJoinBlocks, r = blockIdx.x % kJoinBlocks * kJoinRows + threadIdx.x / 8, t = threadIdx.x % 8;
  const int4 end = a.ends[c1];
  if (end.x < 0) return;
  Seq s;
  load_seq(a, end.x, s, false);
  const int group = a.Hq / a.Hkv, pairs = units_of(a, s) / 2;
  const int row = r % BM, row_t = row / a.heads, hh = end.y % a.chunks * a.heads + row - row_t * a.heads;
  const long long tok = static_cast<long long>(2 * end.z + r / BM) * a.tokens + row_t;
  if (row_t >= a.tokens || tok >= s.n || hh >= group || (end.z >= pairs && r >= BM)) return;
  const int c0 = end.w;
  auto part = [&](int c) { return a.parts + (2 * static_cast<size_t>(c) + (c < c1 ? 1 : 0)) * part_floats(D); };
  float top = -INFINITY;
  for (int c = c0; c <= c1; ++c) top = fmaxf(top, reinterpret_cast<const float4*>(part(c))[r].x);
  float l_mul = 0.f, l_f32 = 0.f;
  float4 acc[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int c = c0; c <= c1; ++c) {
    const float* p = part(c);
    const float4 ml = reinterpret_cast<const float4*>(p)[r];
    const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);  // (sums of scores that are NaN stay NaN)
    l_mul = fmaf(ml.y, f, l_mul);
    l_f32 = fmaf(ml.z, f, l_f32);
    const float4* o = reinterpret_cast<const float4*>(p + 4 * kPartRows + static_cast<size_t>(r) * D);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const float4 v = o[t + 8 * i];
      acc[i].x = fmaf(v.x, f, acc[i].x);
      acc[i].y = fmaf(v.y, f, acc[i].y);
      acc[i].z = fmaf(v.z, f, acc[i].z);
      acc[i].w = fmaf(v.w, f, acc[i].w);
    }
  }
  const size_t out_row = static_cast<size_t>(s.cu + static_cast<int>(tok)) * a.Hq + end.y / a.chunks * group + hh;
  const float inv = l_mul > 0.f || l_mul != l_mul ? 1.f / l_mul : 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    float4 y = make_float4(acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv);
    if (E4M3) y.x *= a.v_scale, y.y *= a.v_scale, y.z *= a.v_scale, y.w *= a.v_scale;
    *reinterpret_cast<uint2*>(a.out + out_row * D + 4 * (t + 8 * i)) = make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
  }
  if (t == 0 && a.lse != nullptr)
    a.lse[out_row] = l_f32 == 0.f ? -INFINITY : (top + log2f(l_f32)) * 0.6931471805599453f;
}

template <int D, bool E4M3>
cudaError_t launch(const PagedAttnArgs& a, const CUtensorMap* tq, const CUtensorMap* tk, const CUtensorMap* tv, int grid,
                   cudaStream_t stream) {
  auto kernel = paged_attn_kernel<D, E4M3>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D, E4M3>::kSmem);
  if (e != cudaSuccess) return e;
  if ((e = launch_dependent(kernel, grid, kThreads, Layout<D, E4M3>::kSmem, stream, *tq, *tk, *tv, a)) != cudaSuccess) return e;
  if (a.whole != nullptr) return cudaSuccess;  // joined with what the caller adds
  return launch_dependent(paged_attn_join_kernel<D, E4M3>, grid * kJoinBlocks, 8 * kJoinRows, 0, stream, a);
}

}  // namespace

cudaError_t launch_shared_plan(const SharedPlanArgs& a, cudaStream_t stream) {
  return launch_dependent(shared_plan_kernel, 1, kPlanThreads, 0, stream, a);
}

size_t paged_attn_parts_bytes(int D) { return 2 * kMaxSms * part_floats(D) * sizeof(float); }
size_t paged_attn_ends_bytes() { return kMaxSms * sizeof(int4); }

cudaError_t paged_attn_grid(int* grid) {
  const cudaError_t e = sm_count(grid);
  *grid = std::min(*grid, kMaxSms);
  return e;
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, const CUtensorMap* tq, const CUtensorMap* tk, const CUtensorMap* tv,
                              bool e4m3, cudaStream_t stream) {
  int grid = 0;
  const cudaError_t e = paged_attn_grid(&grid);
  if (e != cudaSuccess) return e;
  if (a.D == 128)
    return e4m3 ? launch<128, true>(a, tq, tk, tv, grid, stream) : launch<128, false>(a, tq, tk, tv, grid, stream);
  return e4m3 ? launch<64, true>(a, tq, tk, tv, grid, stream) : launch<64, false>(a, tq, tk, tv, grid, stream);
}

}  // namespace mcs
