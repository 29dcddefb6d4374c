// Attention of one token per sequence over a paged cache, split over the
// cache's length and joined.
//
// For query head i of KV head h: s_j = scale q_i . k_j, o_i = sum_j
// exp(s_j - m) v_j / l with the running maximum m and sum l, one pass over the
// keys.  Every key and value row is read once from HBM for up to 16 query heads
// that share it (more heads are further segments, and a cache larger than L2 is read
// again for each 16: 16 x 32768 tokens of 4 KV heads, bf16, 1.07 GB, takes 181 us for 16
// heads each and 304 for 20 or 32): 4 * group flops per 2 * element-size bytes, 8 to 64 flop/byte,
// far below the tensor cores' balance and above the FP32 pipes', so the bound
// is HBM and the products run on mma.sync m16n8k16 with the (up to 16) query
// heads of a KV head as the 16 rows.  tcgen05 would want 128 rows of queries,
// or 128 keys as rows with the softmax across TMEM lanes; at one token per
// sequence the legacy instruction needs a small part of its rate and leaves
// scores and weights in registers.
//
// Split: the keys of all (sequence, KV head) pairs, in tiles of 8 KB (K and V
// together), form one list, and each warp of the machine takes an equal piece
// of it whatever the lengths are.  A warp works alone: a ring of 3 tiles of its
// own, filled by 16-byte cp.async (8 warps per SM, two CTAs: 192 KB in flight), no
// barrier after the shares are known, so that the latencies of one warp's new sequence
// (page numbers, queries) hide behind the other warps' loads.  What a warp holds
// whole it writes at once.  Neighbouring warps' pieces of one segment are joined in
// shared memory when the CTA is done, what crosses CTAs goes to the workspace, and a
// second, programmatically dependent launch joins that in the order of the tiles.
//
// SMs do not get equal parts of the bandwidth: with equal shares the same ones always
// ended up to 15 % later.  So the last eighth of a long list is cut into shares of
// 16 tiles or more for CTAs behind the resident ones, which go to the SMs that are
// done first: 12 x 75600 tokens of 8 KV heads, E4M3 289 -> 283 us, 32 x 30000, bf16 565 ->
// 552 us, 48 sequences up to 16001 120.5 -> 117 us.  From 64 tiles per warp on: at 43
// it was 76.5 us against 74.3, at 55 even, since a share costs 4 us until its first tile
// is there, and finer cuts cost parts (a quarter of the list in shares of 12: 123 us).
// Which CTA does a share changes no result.  Handing shares out by a counter (a launch to
// clear it, three times the parts) had given all of this back.
//
// Measured: 12 x 75600 tokens of 8 KV heads, D = 128, E4M3 (1.86 GB) 283 us;
// 1 x 1023 (4.2 MB) 8.3 us, all of it latency (shares 1.3 us, page numbers and first
// tile 1.2, its products and the CTA's join 1.9, the launch behind it 0.7 and its join 2).
#include <cuda_fp16.h>

#include <algorithm>

#include "internal.h"
#include "launch.cuh"
#include "paged_list.cuh"
#include "ptx.cuh"

namespace mcs {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 3;
constexpr int kHalfStage = 4096;              // bytes of K (and of V) in a tile
constexpr int kStageBytes = 2 * kHalfStage;
constexpr int kMaxSms = 160;
constexpr int kTailCut = 8;                   // CTAs behind the resident ones: a part of the list,
constexpr int kTailMin = 64;                  // from so many positions per resident warp on,
constexpr int kTailShare = 16;                // so many per warp and more,
constexpr int kTailPerSm = 2;                 // and so many CTAs per SM at most
constexpr int kMaxCtas = (2 + kTailPerSm) * kMaxSms;  // parts in the workspace: two per warp
constexpr int kSegCost = 1;                   // what starting a segment costs, in tiles
constexpr int kHeads = 16;                    // query heads per pass over a KV head
constexpr int kPidBits = 27;                  // num_pages * page < 2^31, page >= 16

template <int D, bool E4M3>
struct Geo {
  static constexpr int RB = D * (E4M3 ? 1 : 2);  // bytes of a row
  static constexpr int TK = kHalfStage / RB;     // keys per tile: 16, 32 or 64
  static constexpr int NS = TK / 16;             // 16-key slabs per tile, each inside one page
  static constexpr int CPR = RB / 16;            // 16-byte chunks per row
  static constexpr int RPI = 32 / CPR;           // rows one warp instruction copies
};

// Shared-memory offset of 16-byte chunk c of row r: eight rows of one chunk
// column fall on eight different 16-byte banks groups.
template <int RB>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  if (RB == 64) return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
  return static_cast<uint32_t>(r * RB + ((c ^ (r & 7)) << 4));
}

__device__ __forceinline__ void ldm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Workspace: exclusive sums of the sequences' positions [B + 1] (see below), then
// the parts: (log2 maximum, sum) of each row and the rows' D sums.
__host__ __device__ constexpr size_t parts_offset() { return ((4096 + 1) * 8 + 255) / 256 * 256; }
__host__ __device__ constexpr size_t part_floats(int D, bool wide) { return (wide ? 16 : 8) * (2 + D); }

// Pages are powers of two.
__device__ __forceinline__ int page_log2(const DecodeArgs& a) { return 31 - __clz(a.page); }
__device__ __forceinline__ int pages_of(const DecodeArgs& a, int len) {
  return (len + a.page - 1) >> page_log2(a);
}

// Rows of a sequence's key list (dense: its tokens; sparse: whole listed
// pages), 0 for a length the table cannot hold.
__device__ __forceinline__ int list_rows(const DecodeArgs& a, int len) {
  if (len <= 0 || static_cast<long long>(len) > static_cast<long long>(a.max_pages) * a.page)
    return 0;
  if (a.sel == nullptr) return len;
  return min(pages_of(a, len), a.select) * a.page;
}
template <int TK>
__device__ __forceinline__ int tiles_of(const DecodeArgs& a, int len) {
  return (list_rows(a, len) + TK - 1) / TK;
}

// The list of all segments (a segment: one sequence, one KV head, up to 16
// query heads) has tiles + kSegCost positions for each that has tiles.  It is
// cut into one share per warp, and a warp takes the tiles that begin in its
// share: the first `big` warps equal parts of [0, cut), the others of [cut, all).
template <int TK>
__device__ __forceinline__ int positions_of(const DecodeArgs& a, int len) {
  const int tiles = tiles_of<TK>(a, len);
  return tiles > 0 ? tiles + kSegCost : 0;
}
__device__ __forceinline__ uint64_t divide(uint64_t x, uint64_t y) {
  return ((x | y) >> 32) == 0 ? static_cast<uint32_t>(x) / static_cast<uint32_t>(y) : x / y;
}
struct Shares {
  long long all, cut;
  int big, small;  // warps
  // the first position of share i: floor(i * cut / big), and so on (i, big, small < 2^15)
  __device__ __forceinline__ long long begin(int i) const {
    const bool first = i <= big;
    const long long x = first ? cut : all - cut;
    const unsigned n = first ? big : small, k = first ? i : i - big;
    const long long q = divide(x, n);
    return (first ? 0 : cut) + k * q + k * static_cast<unsigned>(x - q * n) / n;
  }
  // the share that holds position x
  __device__ __forceinline__ int of(long long x) const {
    const bool first = x < cut;
    const long long size = first ? cut : all - cut, n = first ? big : small;
    if (!first) x -= cut;
    // the largest i with i * size < (x + 1) * n: an estimate that is off by one at most, then
    // exact products
    const long long y = (x + 1) * n;
    int i = static_cast<int>(static_cast<float>(x) * (static_cast<float>(n) / static_cast<float>(size)));
    while (i > 0 && i * size >= y) --i;
    while ((i + 1) * size < y) ++i;
    return first ? i : i + big;
  }
};
// `tail` of the grid's `ctas` CTAs are the last ones.
__device__ __forceinline__ Shares shares_of(long long all, int ctas, int tail) {
  const int warps = (ctas - tail) * kWarps;
  if (tail == 0 || all < static_cast<long long>(warps) * kTailMin)
    return {all, all, static_cast<int>(min(all, static_cast<long long>(warps))), 0};
  const long long last = all / kTailCut;
  return {all, all - last, warps, static_cast<int>(min(divide(last, kTailShare), static_cast<uint64_t>(tail * kWarps)))};
}

// A walk over a warp's share, segment by segment.
struct Walk {
  int b, seg;       // sequence, segment inside it
  int tb;           // tiles of each segment of the sequence
  int t0, count;    // the warp's tiles of this segment: [t0, t0 + count)
  long long left;   // positions from t0 to the end of the share
};
// What a kernel reads that may begin before the one in front has ended (see paged_decode_kernel): from L2.
template <bool SHARED>
__device__ __forceinline__ int load(const int32_t* p) { return SHARED ? __ldcg(p) : *p; }

// To the next segment; false at the end of the share.
template <int TK, bool SHARED>
__device__ __forceinline__ bool next_segment(Walk& w, const DecodeArgs& a, int segs) {
  w.left -= w.tb + kSegCost - w.t0;
  if (w.left <= 0) return false;
  if (++w.seg == segs) {
    w.seg = 0;
    do {  // (there is one, unless the lengths change under the kernel)
      if (++w.b >= a.B) return false;
      w.tb = tiles_of<TK>(a, load<SHARED>(a.lens + w.b));
    } while (w.tb == 0);
  }
  w.t0 = 0;
  w.count = static_cast<int>(min(static_cast<long long>(w.tb), w.left));
  return true;
}

// A thread's values of row r (0: g, 1: g + 8), times f, to their columns.
template <int D, bool E4M3>
__device__ __forceinline__ void store_rows(float* to, const float (*o)[4], int r, float f, int t) {
#pragma unroll
  for (int c = 0; c < D / 8; c += 2) {
    if (E4M3) {
      *reinterpret_cast<float4*>(to + 8 * c + 4 * t) =
          make_float4(o[c][2 * r] * f, o[c + 1][2 * r] * f, o[c][2 * r + 1] * f, o[c + 1][2 * r + 1] * f);
    } else {
      *reinterpret_cast<float2*>(to + 8 * c + 2 * t) = make_float2(o[c][2 * r] * f, o[c][2 * r + 1] * f);
      *reinterpret_cast<float2*>(to + 8 * c + 8 + 2 * t) =
          make_float2(o[c + 1][2 * r] * f, o[c + 1][2 * r + 1] * f);
    }
  }
}

// WIDE: more than 8 query heads in a segment.  SHARED: the sequences' own tails behind a common
// beginning of skip[b] pages (lens are the tails'), whose rows are joined with the beginning's
// afterwards: what a warp holds whole it leaves unnormalised.
template <int D, bool E4M3, bool WIDE, bool SHARED = false>
__global__ void __launch_bounds__(kThreads, 2)
    paged_decode_kernel(const DecodeArgs a, int chunks, int tail) {
  using G = Geo<D, E4M3>;
  constexpr int RB = G::RB, TK = G::TK, NS = G::NS, CPR = G::CPR, RPI = G::RPI;
  constexpr float kShift = E4M3 ? 12.f : 0.f;   // weights carry 2^12 so that f16 holds small ones
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_cnt[kWarps][kStages];
  __shared__ int s_seg[kWarps];
  __shared__ float s_m[kWarps][kHeads], s_l[kWarps][kHeads];

  const int tid = threadIdx.x, lane = lane_id(), w = warp_id();
  const int g = lane >> 2, t = lane & 3;
  const int group = a.Hq / a.Hkv, segs = a.Hkv * chunks;
  long long* prefix = static_cast<long long*>(a.ws);
  float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + parts_offset());

  // (SHARED: the kernel in front, over the beginnings, has nothing that this one reads and writes
  // nothing that it does; what this one reads was there when that one began.  So they run side by
  // side, this one on the SMs that are free or become so, and it waits before it ends.  Its loads are
  // from L2: an L1 may hold older lines.)
  if (SHARED)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  else
    pdl_begin();

  // ---- this warp's share, found by itself: lane i sums sequences [i * per, (i + 1) * per),
  // one scan over the lanes, and one over the sequences of the lane that holds the start
  const int per = (a.B + 31) / 32, b_lane = lane * per;
  long long own = 0;
#pragma unroll 4
  for (int i = 0; i < per; ++i)
    if (b_lane + i < a.B) own += positions_of<TK>(a, load<SHARED>(a.lens + b_lane + i));
  auto scan = [&](long long x) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    return x;
  };
  const long long upto = scan(own), all = __shfl_sync(0xffffffffu, upto, 31) * segs;
  if (blockIdx.x == 0 && w == 0) {
    long long sum = upto - own;
    for (int b = b_lane; b < min(a.B, b_lane + per); ++b) {
      const int len = load<SHARED>(a.lens + b), x = positions_of<TK>(a, len);
      if (x == 0 && len != 0) atomicOr(a.status, DEV_BOUNDS);
      prefix[b] = sum;
      sum += x;
    }
    if (lane == 31) prefix[a.B] = upto;
  }
  const Shares shares = shares_of(all, gridDim.x, tail);
  const int warps = shares.big + shares.small, me = blockIdx.x * kWarps + w;
  if (static_cast<int>(blockIdx.x) * kWarps >= warps) {  // a CTA without a share
    if (SHARED) asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  Walk here = {};
  bool busy = me < warps;
  if (busy) {
    const long long ends = shares.begin(me + (lane & 1));
    const long long lo = __shfl_sync(0xffffffffu, ends, 0), hi = __shfl_sync(0xffffffffu, ends, 1);
    // (all > 0: some lane's sequences hold position lo)
    const int from = per == 1 ? 0 : __ffs(__ballot_sync(0xffffffffu, lo < upto * segs)) - 1;
    long long base = per == 1 ? 0 : __shfl_sync(0xffffffffu, upto - own, from);
    busy = false;
    for (int b0 = from * per; from >= 0 && b0 < a.B; b0 += 32) {
      const int b = b0 + lane;
      long long x = own, y = upto;  // (a sequence per lane: known already)
      if (per > 1) {
        x = b < a.B && b < (from + 1) * per ? positions_of<TK>(a, load<SHARED>(a.lens + b)) : 0;
        y = scan(x);
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, lo < (base + y) * segs);
      if (hit != 0) {
        const int at = __ffs(hit) - 1;
        const long long first = (base + __shfl_sync(0xffffffffu, y - x, at)) * segs;
        const long long size = __shfl_sync(0xffffffffu, x, at);
        here.b = b0 + at;
        here.tb = static_cast<int>(size) - kSegCost;
        here.seg = static_cast<int>(divide(lo - first, size));
        here.t0 = static_cast<int>(lo - first - here.seg * size);
        busy = true;
        break;
      }
      base += __shfl_sync(0xffffffffu, y, 31);
    }
    here.left = hi - lo;
    here.count = static_cast<int>(min(static_cast<long long>(here.tb - here.t0), here.left));
    if (busy && here.count <= 0) busy = next_segment<TK, SHARED>(here, a, segs);
  }

  // ---- the warp's ring: its tiles, three ahead
  uint8_t* ring = smem + w * (kStages * kStageBytes);
  const uint32_t ring_s = smem_u32(ring);
  Walk ahead = here;
  int k_next = 0;          // next tile of `ahead` to load: t0 + k_next
  uint32_t found = 0;      // lane i: page and rows of the i-th 16-key slab from a window's start
  bool more = busy;
  const int l_row = lane / CPR, l_chunk = lane % CPR;

  auto look_up = [&](int k) {
    const long long row0 = static_cast<long long>(ahead.t0 + k) * TK + lane * 16;
    found = 0;
    if (k + lane / NS >= ahead.count) return;
    const int len = load<SHARED>(a.lens + ahead.b);
    if (row0 >= list_rows(a, len)) return;
    const int h = ahead.seg / chunks;
    const int at = static_cast<int>(row0 >> page_log2(a)), inner = static_cast<int>(row0) & (a.page - 1);
    int j = at;
    if (a.sel != nullptr) {
      j = a.sel[(static_cast<size_t>(ahead.b) * a.Hkv + h) * a.select + at];
      if (j == -1) return;
      if (j < 0 || j >= pages_of(a, len)) {
        atomicOr(a.status, DEV_BOUNDS);
        return;
      }
    }
    const int pid = load<SHARED>(a.table + static_cast<size_t>(ahead.b) * a.max_pages + j + (SHARED ? __ldcg(a.skip + ahead.b) : 0));
    if (pid < 0 || pid >= a.num_pages) {
      atomicOr(a.status, DEV_BOUNDS);
      return;
    }
    const int rows = min(16, max(0, len - j * a.page - inner));
    found = static_cast<uint32_t>(pid) | (static_cast<uint32_t>(rows) << kPidBits);
  };

  auto load_next = [&](int stage) {
    if (more && k_next >= ahead.count) {
      more = next_segment<TK, SHARED>(ahead, a, segs);
      k_next = 0;
    }
    if (more) {
      constexpr int kWindow = 32 / NS;
      if (k_next % kWindow == 0) look_up(k_next);
      const int h = ahead.seg / chunks;
      const int row0 = (ahead.t0 + k_next) * TK & (a.page - 1);
      const uint32_t dst = ring_s + stage * kStageBytes;
      uint32_t counts = 0;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const uint32_t f = __shfl_sync(0xffffffffu, found, k_next % kWindow * NS + s);
        const int rows = f >> kPidBits, pid = f & ((1u << kPidBits) - 1u);
        counts |= static_cast<uint32_t>(rows) << (8 * s);
        // rows of the slab in the caches (below 2^31), then bytes in 64 bits
        const int row = (pid * a.Hkv + h) * a.page + ((row0 + 16 * s) & (a.page - 1)) + l_row;
        const size_t at = static_cast<size_t>(row) * RB + l_chunk * 16;
        const uint8_t* ks = static_cast<const uint8_t*>(a.k) + at;
        const uint8_t* vs = static_cast<const uint8_t*>(a.v) + at;
#pragma unroll
        for (int i = 0; i < 16 / RPI; ++i) {
          const int r = i * RPI + l_row;
          const uint32_t to = dst + swz<RB>(16 * s + r, l_chunk);
          const int bytes = r < rows ? 16 : 0;  // rows that hold no token become zeros
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to),
                       "l"(ks + i * (RPI * RB)), "r"(bytes)
                       : "memory");
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + kHalfStage),
                       "l"(vs + i * (RPI * RB)), "r"(bytes)
                       : "memory");
        }
      }
      if (lane == 0) s_cnt[w][stage] = static_cast<int>(counts);
      ++k_next;
    }
    cp_async_commit();
  };

#pragma unroll
  for (int i = 0; i < kStages; ++i) load_next(i);
  int stage = 0;

  constexpr int QK = D / 16;         // k-steps of the score product
  constexpr int NT = D / 8;          // 8-column tiles of the output
  constexpr uint32_t kFull = NS == 1 ? 16u : NS == 2 ? 0x1010u : 0x10101010u;

  float o[NT][4];
  float m[2], l[2];
  bool goes_on = false;  // the last segment continues in the next warp's share

  while (busy) {
    const int h = here.seg / chunks, q0 = here.seg % chunks * kHeads;
    const int heads = min(kHeads, group - q0);
    const __nv_bfloat16* q = a.q + here.b * a.q_stride + static_cast<size_t>(h * group + q0) * D;
    // queries as the A operand; E4M3: a thread's four values of a 16-value
    // chunk are consecutive, as ldmatrix hands out the bytes of K
    uint32_t qa[QK][4];
#pragma unroll
    for (int i = 0; i < QK; ++i) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t x = 0, y = 0;
        if ((WIDE || r == 0) && g + 8 * r < heads) {
          const __nv_bfloat16* p = q + (g + 8 * r) * D + 16 * i;
          if (E4M3) {
            const uint2 v = SHARED ? __ldcg(reinterpret_cast<const uint2*>(p + 4 * t)) : *reinterpret_cast<const uint2*>(p + 4 * t);
            x = bf16x2_to_f16x2(v.x);
            y = bf16x2_to_f16x2(v.y);
          } else {
            x = load<SHARED>(reinterpret_cast<const int32_t*>(p + 2 * t));
            y = load<SHARED>(reinterpret_cast<const int32_t*>(p + 8 + 2 * t));
          }
        }
        qa[i][r] = x;
        qa[i][r + 2] = y;
      }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;

    for (int k = 0; k < here.count; ++k) {
      cp_async_wait_group<kStages - 1>();
      __syncwarp();
      const uint32_t ks = ring_s + stage * kStageBytes, vs = ks + kHalfStage;
      const uint32_t counts = static_cast<uint32_t>(s_cnt[w][stage]);
      float s[2 * NS][4] = {};
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        if (E4M3) {
          // matrices: keys 0-7 and 8-15 of chunk c, then of chunk c + 1
          const int r = 16 * i + (lane & 15);
#pragma unroll
          for (int c = 0; c < QK; c += 2) {
            uint32_t f[4], lo, hh;
            ldm4(ks + swz<RB>(r, c + (lane >> 4)), f);
            e4m3x4_to_f16x4(f[0], lo, hh);
            mma<true>(s[2 * i], qa[c], lo, hh);
            e4m3x4_to_f16x4(f[1], lo, hh);
            mma<true>(s[2 * i + 1], qa[c], lo, hh);
            e4m3x4_to_f16x4(f[2], lo, hh);
            mma<true>(s[2 * i], qa[c + 1], lo, hh);
            e4m3x4_to_f16x4(f[3], lo, hh);
            mma<true>(s[2 * i + 1], qa[c + 1], lo, hh);
          }
        } else {
          // matrices: keys 0-7, both halves of the k-step, then keys 8-15
          const int r = 16 * i + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
          for (int c = 0; c < QK; ++c) {
            uint32_t f[4];
            ldm4(ks + swz<RB>(r, 2 * c + ((lane >> 3) & 1)), f);
            mma<false>(s[2 * i], qa[c], f[0], f[1]);
            mma<false>(s[2 * i + 1], qa[c], f[2], f[3]);
          }
        }
      }
      if (counts != kFull) {
#pragma unroll
        for (int j = 0; j < 2 * NS; ++j) {
          const int rows = (counts >> (8 * (j >> 1))) & 255, c0 = (j & 1) * 8 + 2 * t;
          if (c0 >= rows) s[j][0] = s[j][2] = -INFINITY;
          if (c0 + 1 >= rows) s[j][1] = s[j][3] = -INFINITY;
        }
      }
      // running maximum, over the four threads of a row
      float mx[2] = {m[0], m[1]};
#pragma unroll
      for (int j = 0; j < 2 * NS; ++j) {
        mx[0] = fmax3(mx[0], s[j][0], s[j][1]);
        if (WIDE) mx[1] = fmax3(mx[1], s[j][2], s[j][3]);
      }
#pragma unroll
      for (int r = 0; r < (WIDE ? 2 : 1); ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
      }
      if (__any_sync(0xffffffffu, mx[0] > m[0] || (WIDE && mx[1] > m[1]))) {
#pragma unroll
        for (int r = 0; r < (WIDE ? 2 : 1); ++r) {
          const float f = m[r] == mx[r] ? 1.f : ex2((m[r] - mx[r]) * a.scale_log2);
          l[r] *= f;
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            o[j][2 * r] *= f;
            o[j][2 * r + 1] *= f;
          }
          m[r] = mx[r];
        }
      }
      // weights in two parts (bf16: 2^-16 off; f16: 2^-22, and 2^-37 of the largest weight), so that
      // their rounding stays below fp32 sums' or the output's; one f16 part, 2^-11 off, showed
      // wherever values cancel.  The low f16 parts of up to 8 heads are rows 8 to 15 of the high
      // parts' product and cost nothing; those of more heads take products of their own (16 x 65536
      // tokens of 4 KV heads with 16 query heads each: 179 -> 198 us; in products of their own
      // with 8 heads: 167 -> 175).
      const float off0 = kShift - (m[0] == -INFINITY ? 0.f : m[0] * a.scale_log2);
      const float off1 = kShift - (m[1] == -INFINITY ? 0.f : m[1] * a.scale_log2);
      constexpr int GS = E4M3 ? (WIDE ? NS : 2) : 1;  // slabs at a time
#pragma unroll
      for (int i0 = 0; i0 < NS; i0 += GS) {
        uint32_t p[GS][4], pl[GS][4];
#pragma unroll
        for (int i = 0; i < GS; ++i) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float* x = s[2 * (i0 + i) + j];
#pragma unroll
            for (int e = 0; e < (WIDE ? 4 : 2); ++e) {
              x[e] = ex2(fmaf(x[e], a.scale_log2, e < 2 ? off0 : off1));
              l[e >> 1] += x[e];
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              if (r == 1 && !WIDE) {
                if (!E4M3) p[i][2 * j + 1] = 0;
                pl[i][2 * j + 1] = 0;
              } else if (E4M3) {
                uint32_t hw = pack_f16(x[2 * r], x[2 * r + 1]);
                const float2 hf = __half22float2(*reinterpret_cast<__half2*>(&hw));
                p[i][2 * j + r] = hw;
                (WIDE ? pl[i][2 * j + r] : p[i][2 * j + 1]) = pack_f16(x[2 * r] - hf.x, x[2 * r + 1] - hf.y);
              } else {
                const uint32_t hb = pack_bf16(x[2 * r], x[2 * r + 1]);
                p[i][2 * j + r] = hb;
                pl[i][2 * j + r] = pack_bf16(x[2 * r] - __uint_as_float(hb << 16),
                                             x[2 * r + 1] - __uint_as_float(hb & 0xFFFF0000u));
              }
            }
          }
        }
#pragma unroll
        for (int c = 0; c < CPR; c += 2) {
          // E4M3: the slabs' sums by themselves, added to the running ones afterwards: the tensor
          // cores cut their sums off, and 700 products behind one another came out 2^-16 too small
          float sums[4][4] = {};
#pragma unroll
          for (int i = 0; i < GS; ++i) {
            uint32_t f[4];
            ldm4t(vs + swz<RB>(16 * (i0 + i) + (lane & 15), c + (lane >> 4)), f);
            if (E4M3) {
              // bytes (key 2t, values 2g and 2g + 1), (key 2t + 1, the same): even
              // and odd values become two 8-column tiles
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                uint32_t a0, a1, b0, b1;
                e4m3x4_to_f16x4(f[2 * u], a0, a1);
                e4m3x4_to_f16x4(f[2 * u + 1], b0, b1);
                const uint32_t even0 = __byte_perm(a0, a1, 0x5410), even1 = __byte_perm(b0, b1, 0x5410);
                const uint32_t odd0 = __byte_perm(a0, a1, 0x7632), odd1 = __byte_perm(b0, b1, 0x7632);
                mma<true>(sums[2 * u], p[i], even0, even1);
                mma<true>(sums[2 * u + 1], p[i], odd0, odd1);
                if (WIDE) {
                  mma<true>(sums[2 * u], pl[i], even0, even1);
                  mma<true>(sums[2 * u + 1], pl[i], odd0, odd1);
                }
              }
            } else {
              mma<false>(o[c], p[i], f[0], f[1]);
              mma<false>(o[c + 1], p[i], f[2], f[3]);
              mma<false>(o[c], pl[i], f[0], f[1]);
              mma<false>(o[c + 1], pl[i], f[2], f[3]);
            }
          }
          if (E4M3) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              float* to = o[2 * c + u];
              if (WIDE) {
                f2_unpack(f2_add(f2_pack(to[0], to[1]), f2_pack(sums[u][0], sums[u][1])), to[0], to[1]);
                f2_unpack(f2_add(f2_pack(to[2], to[3]), f2_pack(sums[u][2], sums[u][3])), to[2], to[3]);
              } else {
                to[0] += sums[u][0] + sums[u][2];
                to[1] += sums[u][1] + sums[u][3];
              }
            }
          }
        }
      }
      __syncwarp();
      load_next(stage);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }

#pragma unroll
    for (int r = 0; r < (WIDE ? 2 : 1); ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      m[r] *= a.scale_log2;
    }
    goes_on = here.t0 + here.count < here.tb;
    if (goes_on) break;
    // ---- the segment ends here: its rows, or the last part of them
    float* part = parts + 2 * static_cast<size_t>(me) * part_floats(D, WIDE);
#pragma unroll
    for (int r = 0; r < (WIDE ? 2 : 1); ++r) {
      const int head = g + 8 * r;
      if (head >= heads) continue;
      if (SHARED && here.t0 == 0) {
        const size_t at = static_cast<size_t>(here.b) * a.Hq + h * group + q0 + head;
        if (t == 0) reinterpret_cast<float2*>(a.own + static_cast<size_t>(a.B) * a.Hq * D)[at] = make_float2(m[r], l[r]);
        store_rows<D, E4M3>(a.own + at * D, o, r, 1.f, t);
      } else if (here.t0 == 0) {
        // (the value scale by itself: its quotient by l may be too small for a normal float)
        const float inv = l[r] > 0.f || l[r] != l[r] ? 1.f / l[r] : 0.f;
        const size_t at = static_cast<size_t>(here.b) * a.Hq + h * group + q0 + head;
        __nv_bfloat16* to = a.out + at * D;
#pragma unroll
        for (int c = 0; c < NT; c += 2) {
          float x0 = o[c][2 * r] * inv, x1 = o[c][2 * r + 1] * inv;
          float y0 = o[c + 1][2 * r] * inv, y1 = o[c + 1][2 * r + 1] * inv;
          if (E4M3) x0 *= a.v_scale, x1 *= a.v_scale, y0 *= a.v_scale, y1 *= a.v_scale;
          if (E4M3) {
            *reinterpret_cast<uint2*>(to + 8 * c + 4 * t) = make_uint2(pack_bf16(x0, y0), pack_bf16(x1, y1));
          } else {
            *reinterpret_cast<uint32_t*>(to + 8 * c + 2 * t) = pack_bf16(x0, x1);
            *reinterpret_cast<uint32_t*>(to + 8 * c + 8 + 2 * t) = pack_bf16(y0, y1);
          }
        }
        if (a.lse != nullptr && t == 0)
          a.lse[at] = l[r] == 0.f ? -INFINITY : (m[r] + (log2f(l[r]) - kShift)) * 0.6931471805599453f;
      } else {
        if (t == 0) *reinterpret_cast<float2*>(part + 2 * head) = make_float2(m[r], l[r]);
        store_rows<D, E4M3>(part + 2 * (WIDE ? 16 : 8) + head * D, o, r, 1.f, t);
      }
    }
    busy = next_segment<TK, SHARED>(here, a, segs);
  }

  // ---- join the warps whose last segment is the same and goes on
  cp_async_wait_group<0>();
  if (lane == 0) s_seg[w] = goes_on ? here.b * segs + here.seg : -1;
  if (goes_on && t == 0) {
    s_m[w][g] = m[0];
    s_l[w][g] = l[0];
    if (WIDE) {
      s_m[w][g + 8] = m[1];
      s_l[w][g + 8] = l[1];
    }
  }
  __syncthreads();  // also: every ring is idle, and is the join's buffer from here
  constexpr int ROWS = WIDE ? 16 : 8, OS = D + 4;
  float* s_o = reinterpret_cast<float*>(smem);  // [warp][row][OS]
  if (goes_on) {
#pragma unroll
    for (int r = 0; r < (WIDE ? 2 : 1); ++r) {
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < kWarps; ++i)
        if (s_seg[i] == s_seg[w]) top = fmaxf(top, s_m[i][g + 8 * r]);
      store_rows<D, E4M3>(s_o + (w * ROWS + g + 8 * r) * OS, o, r, m[r] == -INFINITY ? 0.f : ex2(m[r] - top), t);
    }
  }
  __syncthreads();
  for (int first = 0; first < kWarps; ++first) {
    const int id = s_seg[first];
    if (id < 0 || (first > 0 && s_seg[first - 1] == id)) continue;
    float* part = parts + (2 * (static_cast<long long>(blockIdx.x) * kWarps + first) + 1) * part_floats(D, WIDE);
    for (int e = tid; e < ROWS * D / 4; e += kThreads) {
      const int row = e / (D / 4), col = e % (D / 4) * 4;
      float top = -INFINITY, sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kWarps; ++i)
        if (s_seg[i] == id) top = fmaxf(top, s_m[i][row]);
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        if (s_seg[i] != id) continue;
        const float4 v = *reinterpret_cast<const float4*>(s_o + (i * ROWS + row) * OS + col);
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
        sum += s_m[i][row] == -INFINITY ? 0.f : s_l[i][row] * ex2(s_m[i][row] - top);
      }
      if (col == 0) *reinterpret_cast<float2*>(part + 2 * row) = make_float2(top, sum);
      *reinterpret_cast<float4*>(part + 2 * ROWS + row * D + col) = acc;
    }
  }
  if (SHARED) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Joins the parts of a segment if several shares hold tiles of it, in
// the order of the tiles, and writes the rows of sequences that hold nothing.
// All rows of a part are read together, SIDES parts at a time; a thread's first
// six parts are on their way while the maxima and weights are found.  Few segments, which
// may have a part of every CTA each, take blocks of two rows and 512 threads (one
// sequence of 131072 tokens and one KV head: 36 us with one block for its 8 rows, 24 so).
// Many segments, of which most are whole, share blocks.
constexpr int kJoinFew = 512;
constexpr int kJoinMost = 32;  // segments a block looks at
__host__ __device__ constexpr int join_rows(bool wide, int threads) { return threads == kJoinFew ? 2 : wide ? 16 : 8; }
template <int D, bool E4M3, bool WIDE, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == kJoinFew ? 2 : WIDE && D == 128 ? 3 : 4)
    paged_join_kernel(const DecodeArgs a, int chunks, int grid, int tail, int count, bool early) {
  constexpr int ALL = WIDE ? 16 : 8, ROWS = join_rows(WIDE, THREADS);  // rows of a part, and of those the block's
  constexpr int E = ROWS * D / 4;                                     // fours of these
  constexpr int EPT = E > THREADS ? E / THREADS : 1, SIDES = E > THREADS ? 1 : THREADS / E;
  constexpr int CHUNK = THREADS / ROWS, WARPS = THREADS / 32;         // parts weighed at a time
  constexpr int TK = Geo<D, E4M3>::TK, kAtOnce = 6;  // parts a thread loads side by side
  constexpr float kShift = E4M3 ? 12.f : 0.f;
  __shared__ float s_red[WARPS][ROWS], s_top[ROWS];
  __shared__ float2 s_f[CHUNK][ROWS];  // a part's weight, and its sum times that
  __shared__ float4 s_acc[SIDES][SIDES > 1 ? E : 1];
  __shared__ float s_sums[SIDES][SIDES > 1 ? E : 1];
  __shared__ long long s_before[WARPS][2];
  struct Segment {
    int b, seg, c0, c1;  // the shares of its first and last tile (no tiles: c1 < 0)
  };
  __shared__ Segment s_todo[kJoinMost];
  const int tid = threadIdx.x, lane = lane_id(), w = warp_id();
  const int group = a.Hq / a.Hkv, segs = a.Hkv * chunks;
  const int at = static_cast<int>(blockIdx.x / (ALL / ROWS)) * count, row0 = static_cast<int>(blockIdx.x % (ALL / ROWS)) * ROWS;
  const float* parts = reinterpret_cast<const float*>(static_cast<const uint8_t*>(a.ws) + parts_offset());
  // Where the segments lie follows from the lengths.  The attention kernel neither writes
  // them nor begins before what does has ended, so they are read before it ends (1.5 us of
  // sums and divisions off the chain), from L2, since an L1 may hold older ones until the
  // wait; where there are more blocks than can wait for it, from the sums that it has left.
  {
    int b = at / segs, seg = at - b * segs + tid;
    long long p0 = 0, all = 0;
    const long long* prefix = static_cast<const long long*>(a.ws);
    if (early) {
      const long long x = tid < a.B ? positions_of<TK>(a, __ldcg(a.lens + tid)) : 0;
      long long before = tid < b ? x : 0, total = x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, o);
        total += __shfl_xor_sync(0xffffffffu, total, o);
      }
      if (lane == 0) s_before[w][0] = before, s_before[w][1] = total;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < WARPS; ++i) p0 += s_before[i][0], all += s_before[i][1];
    } else {
      pdl_begin();
      p0 = prefix[b];
      all = prefix[a.B];
    }
    all *= segs;
    // thread i: the block's i-th segment
    if (tid < count) {
      Segment todo = {a.B, 0, 0, 0};
      auto size_of = [&](int i) {
        return early ? static_cast<long long>(positions_of<TK>(a, __ldcg(a.lens + i))) : prefix[i + 1] - prefix[i];
      };
      long long size = b < a.B ? size_of(b) : 0;
      for (; seg >= segs && b < a.B; seg -= segs) {
        p0 += size;
        size = ++b < a.B ? size_of(b) : 0;
      }
      if (b < a.B) {
        todo = {b, seg, 0, -1};
        if (size > 0) {
          const Shares shares = shares_of(all, grid, tail);
          const long long first = p0 * segs + seg * size;
          todo.c0 = shares.of(first);
          todo.c1 = shares.of(first + size - kSegCost - 1);
        }
      }
      s_todo[tid] = todo;
    }
    if (early) pdl_begin();
    __syncthreads();
  }
#pragma unroll 1
  for (int j = 0; j < count; ++j) {
    const Segment todo = s_todo[j];
    const int b = todo.b, h = todo.seg / chunks, q0 = (todo.seg - h * chunks) * kHeads + row0, heads = min(ROWS, group - q0);
    if (b >= a.B || heads <= 0 || todo.c0 == todo.c1) continue;
    const int c0 = todo.c0, c1 = todo.c1;
    const size_t out_row = static_cast<size_t>(b) * a.Hq + h * group + q0;
    if (c1 < 0) {
      uint2* out = reinterpret_cast<uint2*>(a.out + out_row * D);
      for (int i = tid; i < heads * D / 4; i += THREADS) out[i] = make_uint2(0, 0);
      if (a.lse != nullptr && tid < heads) a.lse[out_row + tid] = -INFINITY;
      continue;
    }
    // shares c0 to c1 - 1 go on to the next one and are joined per CTA (the second
    // part of the CTA's first such warp); share c1 ends the segment (its first part)
    const int k0 = c0 / kWarps, n = (c1 - 1) / kWarps - k0 + 2;
    auto part = [&](int i) {
      const int c = i == n - 1 ? c1 : max(c0, (k0 + i) * kWarps);
      return parts + (2 * static_cast<size_t>(c) + (i < n - 1)) * part_floats(D, WIDE);
    };
    const int side = tid / E, e0 = SIDES > 1 ? tid % E : tid;
    auto values = [&](int i, int k) {
      return *reinterpret_cast<const float4*>(part(i) + 2 * ALL + row0 * D + 4 * (e0 + k * THREADS));
    };
    auto row_of = [&](int k) { return (e0 + k * THREADS) / (D / 4); };
    float4 x[kAtOnce][EPT];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
#pragma unroll
      for (int k = 0; k < EPT; ++k) {
        x[u][k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (side + u * SIDES < n && row_of(k) < heads) x[u][k] = values(side + u * SIDES, k);
      }
    }
    // maxima and weights: thread (part, row r)
    const int r = tid % ROWS, i_ml = tid / ROWS;
    auto max_and_sum = [&](int i) {
      return r < heads && i < n ? *reinterpret_cast<const float2*>(part(i) + 2 * (row0 + r)) : make_float2(-INFINITY, 0.f);
    };
    const float2 mine = max_and_sum(i_ml);
    float top = mine.x;
    for (int i = i_ml + CHUNK; i < n; i += CHUNK) top = fmaxf(top, max_and_sum(i).x);
#pragma unroll
    for (int o = 16; o >= ROWS; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane < ROWS) s_red[w][lane] = top;
    __syncthreads();
    for (int row = w; row < ROWS; row += WARPS) {  // a warp per row
      float v = lane < WARPS ? s_red[lane][row] : -INFINITY;
#pragma unroll
      for (int o = WARPS / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
      if (lane == 0) s_top[row] = v;
    }
    __syncthreads();
    top = s_top[r];
    float4 acc[EPT];
    float sum[EPT];
#pragma unroll
    for (int k = 0; k < EPT; ++k) {
      acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      sum[k] = 0.f;
    }
    auto add = [&](const float4& v, float2 f, int k) {
      acc[k].x = fmaf(v.x, f.x, acc[k].x);
      acc[k].y = fmaf(v.y, f.x, acc[k].y);
      acc[k].z = fmaf(v.z, f.x, acc[k].z);
      acc[k].w = fmaf(v.w, f.x, acc[k].w);
      sum[k] += f.y;
    };
    for (int i0 = 0; i0 < n; i0 += CHUNK) {
      const float2 ml = i0 == 0 ? mine : max_and_sum(i0 + i_ml);
      const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);
      s_f[i_ml][r] = make_float2(f, ml.y * f);
      __syncthreads();
      const int end = min(n, i0 + CHUNK);
      int i = i0 + side;
      if (i0 == 0) {
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u, i += SIDES) {
#pragma unroll
          for (int k = 0; k < EPT; ++k)
            if (i < end) add(x[u][k], s_f[i][row_of(k)], k);
        }
      }
      for (; i < end; i += kAtOnce * SIDES) {
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
          for (int k = 0; k < EPT; ++k)
            if (i + u * SIDES < end && row_of(k) < heads) x[u][k] = values(i + u * SIDES, k);
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
          for (int k = 0; k < EPT; ++k)
            if (i + u * SIDES < end) add(x[u][k], s_f[i + u * SIDES - i0][row_of(k)], k);
      }
      __syncthreads();
    }
    if (SIDES > 1) {
      s_acc[side][e0] = acc[0];
      s_sums[side][e0] = sum[0];
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < EPT; ++k) {
      const int row = row_of(k), col = (e0 + k * THREADS) % (D / 4) * 4;
      if (row >= heads || side > 0) continue;
      if (SIDES > 1) {
#pragma unroll
        for (int i = 1; i < SIDES; ++i) add(s_acc[i][e0], make_float2(1.f, s_sums[i][e0]), k);
      }
      const float total = sum[k], inv = total > 0.f || total != total ? 1.f / total : 0.f;
      float4 y = make_float4(acc[k].x * inv, acc[k].y * inv, acc[k].z * inv, acc[k].w * inv);
      if (E4M3) y.x *= a.v_scale, y.y *= a.v_scale, y.z *= a.v_scale, y.w *= a.v_scale;
      *reinterpret_cast<uint2*>(a.out + (out_row + row) * D + col) = make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
      if (a.lse != nullptr && col == 0)
        a.lse[out_row + row] =
            total == 0.f ? -INFINITY : (s_top[row] + (log2f(total) - kShift)) * 0.6931471805599453f;
    }
    __syncthreads();  // s_top, s_acc and s_f are the next one's
  }
}

// Joins, for every sequence and query head, what the tail's shares left with what the common
// beginning's did (PagedAttnArgs): parts in the order of the keys, the beginning's first.  A warp per
// row, a lane per D / 32 values.
template <int D, bool E4M3, bool WIDE>
__global__ void __launch_bounds__(256) paged_shared_join_kernel(const DecodeArgs a, const SharedArgs p, int chunks, int grid, int tail) {
  constexpr int TK = Geo<D, E4M3>::TK, ROWS = WIDE ? 16 : 8, V = D / 32;
  constexpr float kShift = E4M3 ? 12.f : 0.f;
  pdl_begin();
  const int lane = lane_id();
  const int row = blockIdx.x * 8 + warp_id();
  if (row >= a.B * a.Hq) return;
  const int b = row / a.Hq, head = row - b * a.Hq, group = a.Hq / a.Hkv, h = head / group, hh = head - h * group;
  // the row's parts: those of the beginning, then those of the tail
  const int own = a.lens[b];
  PagedAttnPlace at = {0, -1, 0};
  if (a.skip[b] > 0) at = paged_attn_place(p, b, h, hh);
  int c0 = 0, c1 = -1, k0 = 0, tails = 0;
  if (own > 0) {
    const int segs = a.Hkv * chunks, seg = h * chunks + hh / kHeads;
    const long long* prefix = static_cast<const long long*>(a.ws);
    const Shares shares = shares_of(prefix[a.B] * segs, grid, tail);
    const long long size = positions_of<TK>(a, own), first = prefix[b] * segs + seg * size;
    c0 = shares.of(first);
    c1 = shares.of(first + size - kSegCost - 1);
    k0 = c0 / kWarps;
    tails = c0 == c1 ? 1 : (c1 - 1) / kWarps - k0 + 2;
  }
  const int heads = at.c1 - at.c0 + 1, n = heads + tails, r = hh % kHeads;
  const float* parts = reinterpret_cast<const float*>(static_cast<const uint8_t*>(a.ws) + parts_offset());
  const size_t rows = static_cast<size_t>(a.B) * a.Hq;
  float top = -INFINITY, sum = 0.f, acc[V] = {};
  for (int i0 = 0; i0 < n; i0 += 32) {
    // lane i: the i-th part's log2 maximum, sum of weights, and values
    const int i = i0 + lane;
    float m = -INFINITY, l = 0.f;
    const float* o = nullptr;
    if (i < heads) {
      const bool whole = heads == 1;
      const int c = at.c0 + i;
      const float* part = whole ? p.whole : p.parts + (2 * static_cast<size_t>(c) + (c < at.c1 ? 1 : 0)) * paged_attn_part_floats(D);
      const size_t at_row = whole ? row : at.row;
      const float2 ml = reinterpret_cast<const float2*>(whole ? part + rows * D : part)[at_row];
      m = ml.x, l = ml.y;
      o = part + (whole ? 0 : 2 * kPagedAttnPartRows) + at_row * D;
    } else if (i < n) {
      float2 ml;
      if (c0 == c1) {
        ml = reinterpret_cast<const float2*>(a.own + rows * D)[row];
        o = a.own + static_cast<size_t>(row) * D;
      } else {
        const int k = i - heads, c = k == tails - 1 ? c1 : max(c0, (k0 + k) * kWarps);
        const float* part = parts + (2 * static_cast<size_t>(c) + (k < tails - 1)) * part_floats(D, WIDE);
        ml = reinterpret_cast<const float2*>(part)[r];
        o = part + 2 * ROWS + r * D;
      }
      m = ml.x - kShift, l = ml.y;
    }
    float up = fmaxf(top, m);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, d));
    const float g = top == -INFINITY ? 0.f : ex2(top - up), f = m == -INFINITY ? 0.f : ex2(m - up);
    l *= f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    sum = fmaf(sum, g, l);
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] *= g;
    top = up;
    const int count = min(32, n - i0);
    constexpr int kAtOnce = 8;
    for (int k0 = 0; k0 < count; k0 += kAtOnce) {
      float x[kAtOnce][V], fk[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int src = min(k0 + k, count - 1);
        const float* from = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(o), src));
        fk[k] = __shfl_sync(0xffffffffu, f, src);
        if (k0 + k < count) {
#pragma unroll
          for (int v = 0; v < V; ++v) x[k][v] = from[V * lane + v];
        }
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        if (k0 + k < count)
#pragma unroll
          for (int v = 0; v < V; ++v) acc[v] = fmaf(x[k][v], fk[k], acc[v]);
    }
  }
  const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
  float y[V];
#pragma unroll
  for (int i = 0; i < V; ++i) y[i] = E4M3 ? acc[i] * inv * a.v_scale : acc[i] * inv;
  __nv_bfloat16* out = a.out + static_cast<size_t>(row) * D + V * lane;
  if constexpr (V == 4)
    *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
  else
    *reinterpret_cast<uint32_t*>(out) = pack_bf16(y[0], y[1]);
  if (a.lse != nullptr && lane == 0) a.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

template <int D, bool E4M3, bool WIDE>
cudaError_t launch(const DecodeArgs& a, int chunks, int sms, const SharedArgs* shared, cudaStream_t stream) {
  constexpr int kSmem = kWarps * kStages * kStageBytes;
  auto kernel = shared ? paged_decode_kernel<D, E4M3, WIDE, true> : paged_decode_kernel<D, E4M3, WIDE>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  // two CTAs per SM, no more than the longest lists could give a tile to, and the last
  // ones (see the shares)
  const long long rows = a.sel != nullptr
                             ? static_cast<long long>(std::min(a.select, a.max_pages)) * a.page
                             : static_cast<long long>(a.max_pages) * a.page;
  constexpr int TK = Geo<D, E4M3>::TK;
  const long long most = static_cast<long long>(a.B) * a.Hkv * chunks * ((rows + TK - 1) / TK + kSegCost);
  const int n = std::min(sms, kMaxSms);
  const int tail = most >= 2LL * n * kWarps * kTailMin ? kTailPerSm * n : 0;
  const int grid = static_cast<int>(std::min<long long>(2 * n, most)) + tail;
  if ((e = launch_dependent(kernel, grid, kThreads, kSmem, stream, a, chunks, tail)) != cudaSuccess) return e;
  if (shared)
    return launch_dependent(paged_shared_join_kernel<D, E4M3, WIDE>, (a.B * a.Hq + 7) / 8, 256, 0, stream, a, *shared, chunks, grid, tail);
  const int segments = a.B * a.Hkv * chunks;
  if (segments <= sms / 8) {
    constexpr int kBlocks = (WIDE ? 16 : 8) / join_rows(WIDE, kJoinFew);
    return launch_dependent(paged_join_kernel<D, E4M3, WIDE, kJoinFew>, segments * kBlocks, kJoinFew, 0, stream, a, chunks,
                            grid, tail, 1, true);
  }
  const int room = 4 * sms, count = std::min((segments + room - 1) / room, kJoinMost), blocks = (segments + count - 1) / count;
  return launch_dependent(paged_join_kernel<D, E4M3, WIDE, 256>, blocks, 256, 0, stream, a, chunks, grid, tail, count,
                          a.B <= 256 && blocks <= room);
}

}  // namespace

size_t paged_decode_workspace_bytes(int D, int group) {
  return parts_offset() + 2 * kMaxCtas * kWarps * part_floats(D, group > 8) * sizeof(float);
}

cudaError_t launch_paged_decode(const DecodeArgs& a, bool e4m3, const SharedArgs* shared, cudaStream_t stream) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int group = a.Hq / a.Hkv, chunks = (group + kHeads - 1) / kHeads;
  const bool wide = group > 8;
#define MCS_DECODE_CASE(DD, EE, WW) \
  if (a.D == (DD) && e4m3 == (EE) && wide == (WW)) return launch<DD, EE, WW>(a, chunks, sms, shared, stream);
  MCS_DECODE_CASE(128, false, false)
  MCS_DECODE_CASE(128, false, true)
  MCS_DECODE_CASE(128, true, false)
  MCS_DECODE_CASE(128, true, true)
  MCS_DECODE_CASE(64, false, false)
  MCS_DECODE_CASE(64, false, true)
  MCS_DECODE_CASE(64, true, false)
  MCS_DECODE_CASE(64, true, true)
#undef MCS_DECODE_CASE
  return cudaErrorInvalidValue;
}

}  // namespace mcs
