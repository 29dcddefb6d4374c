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
// K and V tile of 128 keys, or its last odd unit, of whose tiles the two softmax chains take 64
// keys each, joined in the CTA.  All segments in a row form one list of tiles, and each of the
// SMs' CTAs takes an equal share of it, whatever the lengths are: few long sequences are so split
// along their keys, many short ones along the list.  What a share holds whole it writes at once;
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
//
// Measured (graph replays; two figures: different GPUs), and what bounds it:
//   a prompt of 16384 tokens, 32 / 8 heads, D = 128: bf16 1372 to 1386 us, 1600 TFLOP/s, 81 % of a
//     matrix product's rate; with the softmax left out it would be 94 %, so the chains' softmax bounds
//     it (two warps per scheduler: maxima, exponentials, sums, rounding, and TMEM on both sides).
//     E4M3 1696 to 1844 us: the conversions take issue slots from it
//   8192 tokens, 40 heads: bf16 512 us, E4M3 577 to 655, 67 and 54 to 61 %: shorter segments, of which each change
//     takes about 4 us: last softmax, product, epilogue, first scores and softmax one after another
//   1024 tokens behind 73552, 40 / 8 heads: bf16 1050 to 1102 us, E4M3 1106 to 1175, 72 to 75 and 67 to 71 %, as the first
//   32 x 5 tokens behind 8000, 32 / 8 heads, bf16 (1.05 GB): 174 to 178 us, 5.9 TB/s, 87 % of a copy
//   the same in E4M3 (0.52 GB): 164 to 173 us, 3.2 TB/s.  A step of an odd unit is a chain of waits (tile there,
//     stage free, converted, scores, weights) of 1.4 us; without the conversions' work it takes 1.1.  Two more
//     tiles ahead, one more f16 stage, and scores a step ahead in S's other half changed nothing each
//   77 tokens, 16 heads, D = 64: 14.6 us, latency: the first use of each role's code and data
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

// Weights are 2^(x - r), x the score in powers of two and r the row's reference: its maximum when that was
// last set, for f16 weights 2^12 below it, since f16 keeps nothing below 2^-25: weights down to 2^-37 of the
// maximum then count, as in the decode, where keys of next to no weight each make up a visible part of the
// output by their number.  (Scores so large that a float cannot tell 12 apart keep the maximum.)
// The reference moves only when the maximum has come to lie 2^16 above it (f16 weights: 2^15 < 65504).
template <bool E4M3>
constexpr float kThreshold = E4M3 ? 15.f : 16.f;
template <bool E4M3>
__device__ __forceinline__ float reference_of(float maximum) {
  return E4M3 && fabsf(maximum) < 0x1p24f ? maximum - 12.f : maximum;
}

template <int D, bool E4M3>
struct Layout {
  static constexpr int kSub = D / 64;                 // 128-byte column sub-tiles of a row
  static constexpr int kSubBytes = BN * 128;
  static constexpr int kTileBytes = kSub * kSubBytes;
  // ring of K and V tiles; E4M3: behind it a ring of tiles as they are in the cache
  static constexpr int kStages = E4M3 ? (D == 128 ? 4 : 8) : D == 128 ? 5 : 12;
  static constexpr int kRawStages = E4M3 ? (D == 128 ? 2 : 8) : 0, kRawBytes = BN * D;
  static constexpr int kRing = 2 * kTileBytes;
  static constexpr int kRaw = kRing + kStages * kTileBytes;
  static constexpr int kBars = kRaw + kRawStages * kRawBytes;
  // MMA batches done, round robin.  A waiter reads the phase of batch n's barrier, which is
  // unambiguous as long as batch n + kDone cannot be done yet.  Loads (and conversions) lag furthest:
  // they wait for the last reader of the item kStages back, and what the kStages - 1 items behind it
  // feed is at most three batches for every two (segments of one step), and three more.
  static constexpr int kDone = D == 128 ? 16 : 32;
  static_assert(kDone >= (kStages - 1) / 2 * 3 + 5, "batch barriers must outnumber the lag");
  static constexpr int kAside = E4M3 ? kRawStages : kStages;
  static constexpr int kNumBars = kStages + 2 * kAside + kDone + 10;
  static constexpr int kBadKey = kBars + kNumBars * 8;           // [2][D] words
  static constexpr int kMl = kBadKey + 2 * D * 4;                // [2][128] floats
  static constexpr int kMisc = kMl + 2 * BM * 4;                 // Misc
  static constexpr int kSmem = kMisc + 80;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert((kStages + kRawStages) / 2 + 2 <= kBadSlots, "bad slots");
};

// ------------------------------------------------------------------ the list

// A walk over a CTA's share, segment by segment; every role makes it by itself.
struct Walk {
  Seq s;
  int units;
  int g, kv, chunk, i;  // sequence, KV head and its chunk of query heads, pair (the last odd unit behind them)
  bool single;     // an odd unit, whose tiles the chains halve
  int steps, steps_a;  // tiles of the segment; of a pair's first unit
  int t0, count;   // the share's tiles of it: [t0, t0 + count)
  long long left;  // positions from t0 to the share's end
  int index;       // segments of the share in front of this one
};
__device__ __forceinline__ void set_segment(const PagedAttnArgs& a, Walk& w) {
  w.single = w.i >= w.units / 2;
  if (w.single) {
    w.steps = w.steps_a = tiles_until(a, w.s, w.s.n);
  } else {
    const long long e = (2LL * w.i + 2) * a.tokens;
    w.steps = tiles_until(a, w.s, static_cast<int>(min(e, static_cast<long long>(w.s.n))));
    w.steps_a = tiles_until(a, w.s, static_cast<int>(e - a.tokens));
  }
}
__device__ __forceinline__ bool next_segment(const PagedAttnArgs& a, Walk& w) {
  w.left -= w.steps + kSegCost - w.t0;
  if (w.left <= 0) return false;
  if (++w.i >= w.units / 2 + (w.units & 1)) {
    w.i = 0;
    if (++w.chunk == a.chunks) {
      w.chunk = 0;
      if (++w.kv == a.Hkv) {
        w.kv = 0;
        do {  // (there is one, unless the lengths change under the kernel)
          if (++w.g >= a.G) return false;
        } while (!load_seq(a, w.g, w.s, false));
        w.units = units_of(a, w.s);
      }
    }
  }
  set_segment(a, w);
  w.t0 = 0;
  w.count = static_cast<int>(min(static_cast<long long>(w.steps), w.left));
  ++w.index;
  return true;
}

// A walk in one register of a warp's lanes, while the softmax needs the registers.
__device__ __forceinline__ int fold(const Walk& w, int lane) {
  const int f[15] = {w.s.cu, w.s.n, w.s.keys, w.units, w.g, w.kv, w.chunk, w.i, w.single, w.steps, w.steps_a, w.t0, w.index,
                     static_cast<int>(w.left), static_cast<int>(w.left >> 32)};
  int x = w.count;
#pragma unroll
  for (int k = 0; k < 15; ++k)
    if (lane == k) x = f[k];
  return x;
}
__device__ __forceinline__ Walk unfold(int x) {
  int f[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) f[k] = __shfl_sync(0xffffffffu, x, k);
  return {{f[0], f[1], f[2]}, f[3], f[4], f[5], f[6], f[7], f[8] != 0, f[9], f[10], f[11], f[15],
          static_cast<long long>(static_cast<uint32_t>(f[13])) | (static_cast<long long>(f[14]) << 32), f[12]};
}

// How many of the share's tiles chain x works on: the first ones (a pair's first unit ends earlier).
__device__ __forceinline__ int steps_of(const Walk& w, int x) {
  return max(0, min(w.count, (x == 0 ? w.steps_a : w.steps) - w.t0));
}

// Lane q of four holds r[i]: piece i of its row.  Then it holds piece q of the rows of lanes i, and stores of
// r[i] fill 64 bytes of a row instead of 16 of four (which took a third of an epilogue).
__device__ __forceinline__ void turn(uint4 (&r)[4], int lane) {
#pragma unroll
  for (int d = 1; d <= 2; d <<= 1) {
    const bool odd = (lane & d) != 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = d == 1 ? 2 * k : k;
      uint4 x = odd ? r[i] : r[i + d];
      x.x = __shfl_xor_sync(0xffffffffu, x.x, d);
      x.y = __shfl_xor_sync(0xffffffffu, x.y, d);
      x.z = __shfl_xor_sync(0xffffffffu, x.z, d);
      x.w = __shfl_xor_sync(0xffffffffu, x.w, d);
      (odd ? r[i] : r[i + d]) = x;
    }
  }
}

// Keys that every row of the segment sees: tiles behind it are looked through.
__device__ __forceinline__ int seen_by_all(const PagedAttnArgs& a, const Walk& w) {
  return a.causal ? w.s.keys - w.s.n + 2 * w.i * a.tokens + 1 : w.s.keys;
}

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
__device__ __noinline__ void mask_scores(uint32_t tS, int keys, int valid, uint32_t bad) {
#pragma unroll 1
  for (int c0 = 0; c0 < keys; c0 += 32) {
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
  uint8_t bad[kBadSlots];  // slabs of each step's tile whose pages lie outside the cache
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
  // bf16: [NS] V tile loaded that is to be looked through, and looked through; E4M3: [kRawStages] tile
  // loaded, and converted
  uint64_t* raw = full + NS;
  uint64_t* past = raw + L::kAside;
  uint64_t* q_full = past + L::kAside;                           // queries loaded
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
    for (int s = 0; s < NS; ++s) mbar_init(full + s, E4M3 ? kLoaders - 1 : 1);
    for (int s = 0; s < L::kAside; ++s) {
      mbar_init(raw + s, 1);
      mbar_init(past + s, kLoaders - 1);
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
  if (tid < kBadSlots) misc.bad[tid] = 0;
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
  const long long lo = busy ? share_begin(blockIdx.x, all, shares) : 0, hi = busy ? share_begin(blockIdx.x + 1, all, shares) : 0;
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
        misc.start.head = static_cast<int>(quotient(in, size));
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
    w.kv = misc.start.head / a.chunks;
    w.chunk = misc.start.head - w.kv * a.chunks;
    w.i = misc.start.i;
    load_seq(a, w.g, w.s, false);
    w.units = units_of(a, w.s);
    w.i = min(w.i, w.units / 2 + (w.units & 1) - 1);
    set_segment(a, w);
    w.t0 = static_cast<int>(misc.start.offset);
    w.left = hi - lo;
    w.count = static_cast<int>(min(static_cast<long long>(w.steps - w.t0), w.left));
    if (w.t0 > 0 && w.count > 0 && w.t0 + w.count == w.steps) {
      part_from = share_of(lo - w.t0, all, shares);
    }
    if (tid == 0) {
      a.ends[blockIdx.x] = make_int4(part_from >= 0 ? w.g : -1, w.kv * a.chunks + w.chunk, w.i, part_from);
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
    // Ring items of a segment, in the order in which the MMA warp asks for them: K(0), then V(j) and
    // K(j + 1) of every step.  K(j) and, of the step in front, V(j - 1) are read last by batch base + 2 j.
    int it = 0;  // items so far
    int reader = 0, q_reader = 0;  // lane i: the last batch that reads stage i; the last that reads the queries
    if (warp == kFirstLoader) {
      // ---------------------------------------------------------- TMA
      if (elect_one()) {
        if (!E4M3) tma_prefetch_desc(&tq);
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
      }
      __syncwarp();
      // Pages of kWindow tiles at a time: lane i has the row in the caches of the i-th slab, -1 where
      // there is nothing; those of the next ones are asked for when a window is begun.
      const int slabs_per_page = a.page / kSlab, shift = 31 - __clz(slabs_per_page);
      auto look_up = [&](int window, int& row, uint32_t& outside) {
        const long long slab = static_cast<long long>(window) * 32 + lane;
        row = -1;
        bool out = false;
        if (slab * kSlab < w.s.keys) {
          const int at = a.row_of != nullptr ? a.row_of[w.g] : w.g;
          const int pid = a.table[static_cast<size_t>(at) * a.max_pages + static_cast<int>(slab >> shift)];
          out = pid < 0 || pid >= a.num_pages;
          if (!out) row = (pid * a.Hkv + w.kv) * a.page + (static_cast<int>(slab) & (slabs_per_page - 1)) * kSlab;
        }
        outside = __ballot_sync(0xffffffffu, out);  // slabs inside the sequence whose page is none
      };
      // a lane per box: a page's rows, 128 bytes wide (E4M3: all of a row's)
      constexpr int kBoxSubs = E4M3 ? 1 : L::kSub, kBoxBytes = E4M3 ? D : 128;
      constexpr int kSlots = E4M3 ? L::kRawStages : NS, kSlotBytes = E4M3 ? L::kRawBytes : L::kTileBytes;
      const int box = lane / kBoxSubs, sub = lane % kBoxSubs, boxes = BN / a.page;
      const int box_slab = box < boxes ? box * slabs_per_page : 0;
      const uint32_t to = smem_u32(E4M3 ? smem + L::kRaw : ring) + sub * L::kSubBytes + box * a.page * kBoxBytes;
      int st = 0, step = 0;
      uint32_t turn = 0;  // of the slots, parity
      uint32_t raw_used = 0, raw_parity = 0;  // bf16, of each stage: a tile went to `raw`; the last one's parity
      uint32_t dirty = 0;                     // steps whose `bad` is not zero
      // Bytes may arrive in front of their announcement: the phase waits for the arrival.
      auto load = [&](const CUtensorMap* tm, int row, bool look, int read_by) -> bool {
        if (it >= kSlots) {
          const bool ok = E4M3 ? warp_wait(past + st, turn ^ 1, abort_flag, a.status) : wait_batch(__shfl_sync(0xffffffffu, reader, st));
          if (!ok) return false;
        }
        uint64_t* bar = (E4M3 || look ? raw : full) + st;
        if (box < boxes)  // (a row past the tensor's end reads zeros)
          tma_load_2d_at(to + st * kSlotBytes, tm, sub * 64, row < 0 ? a.rows : row, bar);
        if (lane == 0) {
          mbar_expect_tx(bar, kSlotBytes);
          if (look) mbar_arrive(full + st);  // `full` keeps its turn: such tiles complete it empty
        }
        if (look) {
          raw_parity ^= ((raw_used >> st) & 1u) << st;
          raw_used |= 1u << st;
        }
        if (lane == st) reader = read_by;
        ++it;
        if (++st == kSlots) st = 0, turn ^= 1;
        return true;
      };
      bool ok = true;
      for (; ok && more; more = next_segment(a, w)) {
        const int count = w.count, t0 = w.t0, look_from = E4M3 ? count : seen_by_all(a, w) / BN - t0;
        int window = t0 / kWindow, slab0 = t0 % kWindow * kSlabs, rows, next_rows;
        uint32_t outside, next_outside;
        look_up(window, rows, outside);
        look_up(window + 1, next_rows, next_outside);
        if (w.index > 0 && !E4M3) ok = wait_batch(q_reader);
        if (!ok) break;
        if (!E4M3 && elect_one()) {
          // a box is tokens x heads rows; tokens behind the sequence's are other ones' or zeros
          const int units = w.single ? 1 : 2;
          mbar_expect_tx(q_full, units * L::kSub * 128 * a.heads * a.tokens);
          const int head = w.kv * group + w.chunk * a.heads;
          for (int u = 0; u < units; ++u)
            for (int s = 0; s < L::kSub; ++s)
              tma_load_3d(qs + u * L::kTileBytes + s * L::kSubBytes, &tq, s * 64, head, w.s.cu + (2 * w.i + u) * a.tokens, q_full);
        }
        __syncwarp();
#pragma unroll 1
        for (int j = 0; ok && j < count; ++j) {
          if (slab0 == 32) {
            slab0 = 0;
            rows = next_rows, outside = next_outside;
            look_up(++window + 1, next_rows, next_outside);
          }
          const int row = __shfl_sync(0xffffffffu, rows, slab0 + box_slab);
          const uint32_t out = (outside >> slab0) & 0xffu, bit = 1u << ((step + j) % kBadSlots);
          slab0 += kSlabs;
          if (out != 0 || (dirty & bit) != 0) {  // for the softmax; in front of the load that it goes with
            dirty = out ? dirty | bit : dirty & ~bit;
            if (lane == 0) {
              misc.bad[(step + j) % kBadSlots] = static_cast<uint8_t>(out);
              if (out) atomicOr(a.status, DEV_BOUNDS);
            }
            __syncwarp();
          }
          ok = load(&tk, row, false, base + 2 * j);
          if (a.fault) ok = false;  // test only: starve the MMA warp
          ok = ok && load(&tv, row, j >= look_from, base + 2 * j + 2);
        }
        step += count;
        q_reader = base + 2 * (count - 1);
        base += 2 * count + 1;
      }
      if (*abort_flag)
        for (int i = max(it - kSlots, 0); i < it; ++i) {
          drain_wait((E4M3 ? raw : full) + i % kSlots, (i / kSlots) & 1);
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
      bool ok = true;
      for (; ok && more; more = next_segment(a, w)) {
        const int count = w.count, t0 = w.t0, keys = w.s.keys, first_look = seen_by_all(a, w) / BN, mark = w.index & 1;
        // A record's last segment, two back, has been read when this one's is begun.  Waited for whether or not
        // there are tiles to look through: a wait left out would put the next one two phases behind, where the
        // barrier's parity says the opposite.
        if (w.index >= 2) ok = warp_wait(written + mark, ((w.index - 2) / 2) & 1, abort_flag, a.status);
        if (!ok) break;
        if constexpr (!E4M3) {
          for (int j = max(0, first_look - t0); ok && j < count; ++j) {
            const int tile = t0 + j, st = (it + 2 * j + 1) % NS;
            ok = warp_wait(raw + st, (raw_parity >> st) & 1u, abort_flag, a.status);
            if (!ok) break;
            raw_parity ^= 1u << st;
            uint8_t* v = ring + st * L::kTileBytes;
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
            if (lane == 0) mbar_arrive(past + st);
          }
          it += 2 * count;
        } else {
          if (w.index > 0) ok = wait_batch(q_reader);
          if (!ok) break;
          // queries: bf16 to f16 through registers, kAtOnce chunks side by side
          constexpr int kChunks = BM * kSegsRow, kAtOnce = 6;
          const int chunk0 = w.chunk * a.heads, head = w.kv * group + chunk0;
#pragma unroll 1
          for (int c0 = me; c0 < (w.single ? 1 : 2) * kChunks; c0 += kAtOnce * kHelp) {
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
          // rows in 16-byte pieces, a row per kSegs lanes
          constexpr int kSegs = D / 16, kRows = 32 / kSegs, kGroups = BN / kRows, kTurns = (kGroups + kLoaders - 2) / (kLoaders - 1);
          const int sub = lane / kSegs, seg = lane % kSegs;
#pragma unroll 1
          for (int i = 0; ok && i < 2 * count; ++i) {
            const int j = i >> 1, tile = t0 + j, st = it % NS, slot = it % L::kRawStages;
            const bool is_k = !(i & 1);
            ok = warp_wait(raw + slot, (it / L::kRawStages) & 1, abort_flag, a.status);
            if (!ok) break;
            uint8_t* from = smem + L::kRaw + slot * L::kRawBytes;
            uint8_t* stage = ring + st * L::kTileBytes;
            uint4 v[kTurns];
#pragma unroll
            for (int k = 0; k < kTurns; ++k)
              if (hw + (kLoaders - 1) * k < kGroups) v[k] = ld_shared16(from + ((hw + (kLoaders - 1) * k) * kRows + sub) * D + seg * 16);
            // (looked through in registers: nothing is written to memory that the next copy overwrites)
            if (!is_k && tile >= first_look) {
#pragma unroll
              for (int k = 0; k < kTurns; ++k) {
                if (hw + (kLoaders - 1) * k >= kGroups) continue;
                const int r = (hw + (kLoaders - 1) * k) * kRows + sub;
                if (r >= keys - tile * BN)
                  v[k] = make_uint4(0u, 0u, 0u, 0u);
                else if (has_bad<true>(v[k]))  // NaN codes (there are no infinities)
                  v[k] = note_bad<true>(v[k], records + mark * D + seg * 16, misc.any_bad + mark, bad_mark(w.index),
                                        (tile - first_look) * BN + r);
              }
            }
            if (it >= NS) ok = wait_batch(__shfl_sync(0xffffffffu, reader, st));
            if (!ok) break;
            if (lane == st) reader = base + 2 * j + (is_k ? 0 : 2);
            ++it;
            __syncwarp();  // every lane has its pieces
            if (lane == 0) mbar_arrive(past + slot);
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
    constexpr uint32_t idesc_half = E4M3 ? idesc_f16(BM, BN / 2, false, false) : idesc_bf16(BM, BN / 2, false, false);
    constexpr uint32_t idesc_pv = E4M3 ? idesc_f16(BM, D, false, true) : idesc_bf16(BM, D, false, true);
    // The tensor core holds one or two MMAs ahead and the issue of a batch ends as its last ones
    // begin: whatever stands between that and the next batch's issue leaves it idle.  So stages,
    // parities and barriers of the next batch are worked out in front of the present one's issue.
    const uint32_t ring_addr = smem_u32(ring), q_addr = smem_u32(qs);
    uint32_t look_parity = 0;       // of each stage's `past` (bf16)
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
      return i.look ? mbar_try_wait(past + i.st, (look_parity >> i.st) & 1) : mbar_try_wait(full + i.st, i.ph);
    };
    auto wait_item = [&](const Item& i) {
      return i.look ? warp_wait(past + i.st, (look_parity >> i.st) & 1, abort_flag, a.status)
                    : warp_wait(full + i.st, i.ph, abort_flag, a.status);
    };
    // S_x = Q_x K^T; an odd unit's chains take the tile's first and last 64 keys
    auto issue_qk = [&](int x, int st, bool single) {
      const uint32_t kb = ring_addr + st * L::kTileBytes + (single ? x * (BN / 2) * 128 : 0);
      const uint32_t qb = q_addr + (single ? 0 : x) * L::kTileBytes, idesc = single ? idesc_half : idesc_qk;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk >> 2) * L::kSubBytes + (kk & 3) * 32;
        umma_ss(tmem + x * 128, sdesc_sw128(qb + off, 16, 1024), sdesc_sw128(kb + off, 16, 1024), idesc, kk > 0);
      }
    };
    // O_x (+)= P_x V
    auto issue_pv = [&](int x, int st, bool first, bool single) {
      const uint32_t vb = ring_addr + st * L::kTileBytes + (single ? x * (BN / 2) * 128 : 0);
#pragma unroll
      for (int kk = 0; kk < BN / 16; ++kk)
        if (kk < BN / 32 || !single)
          umma_ts(tmem + 256 + x * D, tmem + x * 128 + kk * 8, sdesc_sw128(vb + kk * 16 * 128, L::kSubBytes, 1024), idesc_pv,
                  (!first || kk > 0) ? 1u : 0u);
    };
    bool ok = true;
    for (; ok && more; more = next_segment(a, w)) {
      const bool single = w.single;
      const int count = w.count, n0 = steps_of(w, 0);  // (chain b works on every tile)
      const int look_from = E4M3 ? count : seen_by_all(a, w) / BN - w.t0;
      Item k = take(false), v = take(0 >= look_from);
      ok = warp_wait(q_full, w.index & 1, abort_flag, a.status) && wait_item(k);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        if (n0 > 0) issue_qk(0, k.st, single);
        issue_qk(1, k.st, single);
        umma_commit(done + dn);
      }
      __syncwarp();
      dn = (dn + 1) % L::kDone;
      if (count > 1) k = take(false);
#pragma unroll 1
      for (int j = 0; ok && j < count; ++j, ++step) {
        const bool last = j + 1 == count;
        {
          const bool mine = j < n0, next = j + 1 < n0;
          bool ready = mbar_try_wait(p_full, step & 1);
          ready &= try_item(v);
          if (!last) ready &= mbar_try_wait(full + k.st, k.ph);
          if (!__all_sync(0xffffffffu, ready))
            ok = wait_item(v) && (last || wait_item(k)) && warp_wait(p_full, step & 1, abort_flag, a.status);
          if (!ok) break;
          if (v.look) look_parity ^= 1u << v.st;
          uint64_t* bar = done + dn;
          dn = (dn + 1) % L::kDone;
          tc_fence_after();
          if (elect_one()) {
            if (mine) issue_pv(0, v.st, j == 0, single);
            if (next) issue_qk(0, k.st, single);
            umma_commit(bar);
          }
          __syncwarp();
        }
        const bool ready = mbar_try_wait(p_full + 1, step & 1);
        if (!__all_sync(0xffffffffu, ready)) ok = warp_wait(p_full + 1, step & 1, abort_flag, a.status);
        if (!ok) break;
        uint64_t* bar = done + dn;
        dn = (dn + 1) % L::kDone;
        const int vs = v.st, ks = k.st;
        if (!last) v = take(j + 1 >= look_from);
        if (j + 2 < count) k = take(false);
        tc_fence_after();
        if (elect_one()) {
          issue_pv(1, vs, j == 0, single);
          if (!last) issue_qk(1, ks, single);
          umma_commit(bar);
        }
        __syncwarp();
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
    const int row_t = row / a.heads;
    auto row_of = [&](const Walk& w) {
      const int t = row_t;
      Row r;
      r.tok = static_cast<int>(min((2LL * w.i + (w.single ? 0 : x)) * a.tokens + t, 0x7fffffffLL));
      r.head = w.chunk * a.heads + row - t * a.heads;
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
      // an odd unit's chains see half a tile each: its first, its last 64 keys
      const bool single = w.single;
      int ahead = limit - w.t0 * BN - (single ? x * (BN / 2) : 0);  // keys that the row sees from the chain's first on
      const int folded = fold(w, lane);
      float m_run = -INFINITY, l_run = 0.f;
      for (int j = 0; j < count; ++j, ++step, ahead -= BN) {
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
        const uint32_t bad = misc.bad[step % kBadSlots] >> (single ? x * (kSlabs / 2) : 0);
        const int keys = single ? BN / 2 : BN;
        if (bad != 0 || !__all_sync(0xffffffffu, ahead >= keys)) mask_scores(tS, keys, ahead, bad);
        float s[64];
        uint32_t* su = reinterpret_cast<uint32_t*>(s);
        float mx_hi = -INFINITY;
        if (!single) {
          tmem_ld32(tS + 64, su);
          tmem_ld32(tS + 96, su + 32);
          tmem_ld_wait();
          mx_hi = max64(s);
        }
        tmem_ld32(tS + 0, su);
        tmem_ld32(tS + 32, su + 32);
        tmem_ld_wait();
        const float m_new = fmaxf(max64(s), mx_hi) * sl2;
        // The reference moves only when the tile's maximum exceeds it by more than the
        // threshold; TMEM loads and stores are the whole warp's, so all rows enter when one does.
        const bool need = m_new > m_run + kThreshold<E4M3>;  // (the first maximum of a row, too)
        if (__any_sync(0xffffffffu, need)) {
          const float ref = reference_of<E4M3>(m_new);
          if (j > 0) {
            const float f = need ? ex2(m_run - ref) : 1.f;
            l_run *= f;
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
          if (need) m_run = ref;
        }
        // p = 2^(s c - m), rounded to bf16 or f16 for the product and summed in fp32 as they were, for lse
        // and output: a weight's rounding then counts once in the output, by at most 2^-8 (f16: 2^-11, and
        // 2^-37 of the largest weight) of the weight times its value.  (A second sum of the rounded weights makes equal values come out unrounded,
        // but no bound smaller, and cost 4 to 9 % of a prompt's time.)
        const float m_ref = m_run == -INFINITY ? 0.f : m_run;
        const uint64_t c2 = f2_pack(sl2, sl2), nm2 = f2_pack(-m_ref, -m_ref);
        uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 1) {
            if (single) break;
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
              acc[i & 3] = f2_add(acc[i & 3], f2_pack(p0, p1));
            }
            tmem_st16(tS + h * 32 + c * 16, pk);
          }
        }
        l_run += sum8(acc);
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
      const bool had = steps_of(w, x) > 0;  // this chain wrote O
      float fa = 1.f, fb = 0.f;
      if (w.single) {  // chain a joins the two
        if (x == 1) {
          s_ml[row] = m_run;
          s_ml[BM + row] = l_run;
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
          l_run = fmaf(l_run, fa, s_ml[BM + row] * fb);
          m_run = top;
        }
      }
      tc_fence_after();
      if (!idle && !(w.single && x == 1)) {
        const uint32_t tOb = tmem + 256 + D + lane_off;
        const bool goes_on = w.t0 + w.count < w.steps, whole = w.t0 == 0 && !goes_on;
        const int out_row = live ? (w.s.cu + r.tok) * a.Hq + w.kv * group + r.head : 0;
        const bool finals = whole && a.whole == nullptr;
        // (the value scale by itself: its quotient by the sum may be too small for a normal float)
        if (finals) {
          const float inv = l_run > 0.f || l_run != l_run ? 1.f / l_run : 0.f;
          fa *= inv;
          fb *= inv;
        }
        float* part = a.parts + (2 * static_cast<size_t>(blockIdx.x) + (goes_on ? 1 : 0)) * part_floats(D);
        float* const sums = whole ? a.whole + static_cast<size_t>(a.T) * a.Hq * D : part;
        const int at = whole ? out_row : x * BM + row;
        if (live && !finals) reinterpret_cast<float2*>(sums)[at] = make_float2(m_run, l_run);
        part = whole ? a.whole : part + 2 * kPartRows;
        int ats[4];  // of this lane's four, -1: none
#pragma unroll
        for (int i = 0; i < 4; ++i) ats[i] = __shfl_sync(0xffffffffu, live ? at : -1, (lane & 28) + i);
        const int seen = seen_by_all(a, w);
        const bool spoiled = *static_cast<volatile uint32_t*>(misc.any_bad + (w.index & 1)) == bad_mark(w.index);
        const uint32_t* record = records + (w.index & 1) * D;
#pragma unroll 1  // (once per segment: short code is there sooner)
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
          if (w.single) {
            tmem_ld32(tOb + c * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = fmaf(__uint_as_float(o[i]), fb, v[i]);
          }
          if (__builtin_expect(spoiled, 0)) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (first_bad(record, w, seen, c * 32 + i) < r.limit) v[i] = NAN;
          }
          const size_t col = c * 32 + (lane & 3) * (finals ? 8 : 4);
          uint4 p[4];
          if (finals) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = E4M3 ? v[i] * a.v_scale : v[i];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              p[e] = make_uint4(pack_bf16(v[8 * e], v[8 * e + 1]), pack_bf16(v[8 * e + 2], v[8 * e + 3]),
                                pack_bf16(v[8 * e + 4], v[8 * e + 5]), pack_bf16(v[8 * e + 6], v[8 * e + 7]));
            turn(p, lane);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (ats[i] >= 0) *reinterpret_cast<uint4*>(a.out + static_cast<size_t>(ats[i]) * D + col) = p[i];
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float* f = v + 16 * h + 4 * e;
                p[e] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
              }
              turn(p, lane);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (ats[i] >= 0) *reinterpret_cast<uint4*>(part + static_cast<size_t>(ats[i]) * D + col + 16 * h) = p[i];
            }
          }
          __syncwarp();  // TMEM loads are the whole warp's
        }
        if (finals && live && a.lse != nullptr)
          a.lse[out_row] = l_run == 0.f ? -INFINITY : (m_run + log2f(l_run)) * 0.6931471805599453f;
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
// two sequences reach the beginning's end, too; and so does a batch in which reading the beginnings
// once saves too few bytes (see SharedPlanArgs).  Without `tail` it only checks.
constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const SharedPlanArgs a) {
  __shared__ unsigned long long s_saved, s_once;
  const int tid = threadIdx.x, lane = lane_id();
  if (tid == 0) s_saved = s_once = 0;
  pdl_begin();
  const long long room = static_cast<long long>(a.max_pages) * a.page;
  bool bad = tid == 0 && (a.starts[0] != 0 || a.starts[a.G] != a.B);
  for (int g = tid; g < a.G; g += kPlanThreads) bad = bad || a.starts[g] > a.starts[g + 1];
  const bool writes = a.tail != nullptr;
  for (int b = tid; b < a.B; b += kPlanThreads) {
    const int len = a.lens[b];
    const bool good = len >= 0 && len <= room;
    if (!good) atomicOr(a.status, DEV_BOUNDS);
    if (!writes) continue;
    a.tail[b] = good ? len : 0;
    a.skip[b] = 0;
    a.group_of[b] = -1;
  }
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) atomicOr(a.status, DEV_BOUNDS);
  for (int g = tid; writes && g <= a.G; g += kPlanThreads) a.cu[g] = bad ? 0 : a.starts[g];
  for (int g = warp_id(); g < a.G; g += kPlanThreads / 32) {
    const int lo = bad ? 0 : a.starts[g], hi = bad ? 0 : a.starts[g + 1], pages = a.shared[g];
    const bool good = pages >= 0 && pages <= a.max_pages;
    const int keys = good ? pages * a.page : 0;
    bool wrong = !good;
    int live = 0, leader = 0x7fffffff;
    for (int b = lo + lane; b < hi; b += 32) {
      const int given = a.lens[b], len = given <= room ? given : 0;
      wrong = wrong || (len > 0 && len < keys);
      if (len > 0 && len >= keys) {
        ++live;
        leader = min(leader, b);
      }
    }
    live = __reduce_add_sync(0xffffffffu, live);
    leader = __reduce_min_sync(0xffffffffu, leader);
    if (wrong) atomicOr(a.status, DEV_BOUNDS);
    if (writes && lane == 0) {
      const bool use = live > 1 && keys > 0;
      a.keys[g] = use ? keys : 0;
      a.leader[g] = use ? leader : 0;
      if (use) {
        atomicAdd(&s_saved, (live - 1ull) * keys * a.row_bytes);
        atomicAdd(&s_once, keys * a.row_bytes);
      }
    }
  }
  if (!writes) return;
  __syncthreads();
  const unsigned long long close = min(s_once, a.near);
  const bool worth = s_saved >= a.worth + close + a.beyond * (s_once - close);
  for (int g = warp_id(); g < a.G; g += kPlanThreads / 32) {
    const int keys = a.keys[g];
    __syncwarp();
    if (keys == 0) continue;
    if (!worth) {
      if (lane == 0) a.keys[g] = 0;
      continue;
    }
    for (int b = a.starts[g] + lane; b < a.starts[g + 1]; b += 32) {
      const int len = a.tail[b];
      if (len < keys) continue;
      a.tail[b] = len - keys;
      a.skip[b] = a.shared[g];
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
  for (int c = c0; c <= c1; ++c) top = fmaxf(top, reinterpret_cast<const float2*>(part(c))[r].x);
  float sum = 0.f;
  float4 acc[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int c = c0; c <= c1; ++c) {
    const float* p = part(c);
    const float2 ml = reinterpret_cast<const float2*>(p)[r];
    const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);  // (sums of scores that are NaN stay NaN)
    sum = fmaf(ml.y, f, sum);
    const float4* o = reinterpret_cast<const float4*>(p + 2 * kPartRows + static_cast<size_t>(r) * D);
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
  const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    float4 y = make_float4(acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv);
    if (E4M3) y.x *= a.v_scale, y.y *= a.v_scale, y.z *= a.v_scale, y.w *= a.v_scale;
    *reinterpret_cast<uint2*>(a.out + out_row * D + 4 * (t + 8 * i)) = make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
  }
  if (t == 0 && a.lse != nullptr)
    a.lse[out_row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
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
