// Attention of one token per sequence over a paged cache, split over the
// cache's length and joined.
//
// For query head i of KV head h: s_j = scale q_i . k_j, o_i = sum_j
// exp(s_j - m) v_j / l with the running maximum m and sum l, one pass over the
// keys.  Every key and value row is read once from HBM for all query heads
// that share it: 4 * group flops per 2 * element-size bytes, 8 to 64 flop/byte,
// far below the tensor cores' balance and above the FP32 pipes', so the bound
// is HBM and the products run on mma.sync m16n8k16 with the (up to 16) query
// heads of a KV head as the 16 rows.  tcgen05 would want 128 rows of queries,
// or 128 keys as rows with the softmax across TMEM lanes; at one token per
// sequence the legacy instruction needs a small part of its rate and leaves
// scores and weights in registers.
//
// Split: the keys of all (sequence, KV head) pairs, in tiles of 8 KB (K and V
// together), form one list; each of the SMs' CTAs takes an equal share, whatever the
// lengths are.  Inside a CTA each of the 8 warps takes every eighth tile and
// has a ring of its own of 3 tiles, filled by 16-byte cp.async: 192 KB per SM
// in flight, no barrier in the main loop.  At the end of a pair's part the
// warps join through shared memory; a pair that lies in one CTA is written
// at once, the parts of the others go to the workspace and a second,
// programmatically dependent launch joins them in a fixed order.
#include <cuda_fp16.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace mcs {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 3;
constexpr int kHalfStage = 4096;              // bytes of K (and of V) in a tile
constexpr int kStageBytes = 2 * kHalfStage;
constexpr int kMaxCtas = 256;                 // parts in the workspace: two per CTA
constexpr int kMinTiles = 8;                  // tiles a CTA takes at least: one per warp
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

// Workspace: exclusive sums of the sequences' tiles [B + 1], then the parts:
// (log2 maximum, sum) of 16 rows and 16 rows of D sums each.
__host__ __device__ constexpr size_t parts_offset() { return ((4096 + 1) * 8 + 255) / 256 * 256; }
__host__ __device__ constexpr size_t part_floats(int D) { return kHeads * (2 + D); }

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
__device__ __forceinline__ int tiles_of(const DecodeArgs& a, int b) {
  return (list_rows(a, a.lens[b]) + TK - 1) / TK;
}

// CTAs that share `total` tiles, and the first tile of CTA c among them.
__device__ __forceinline__ long long active_ctas(long long total, int ctas) {
  const long long want = (total + kMinTiles - 1) / kMinTiles;
  return want < 1 ? 1 : (want < ctas ? want : ctas);
}

// A walk over this CTA's tiles, segment by segment (a segment: one sequence,
// one KV head, up to 16 query heads).
struct Walk {
  int b, seg;        // sequence, segment inside it
  int tb;            // tiles of each segment of the sequence
  int t0, count;     // this CTA's tiles of the current segment: [t0, t0 + count)
  long long left;    // tiles behind the current segment
};
template <int TK>
__device__ __forceinline__ bool next_segment(Walk& w, const DecodeArgs& a, int segs) {
  if (w.left == 0) return false;
  if (++w.seg == segs) {
    w.seg = 0;
    do {
      w.tb = tiles_of<TK>(a, ++w.b);
    } while (w.tb == 0);
  }
  w.t0 = 0;
  w.count = static_cast<int>(min(static_cast<long long>(w.tb), w.left));
  w.left -= w.count;
  return true;
}

// WIDE: more than 8 query heads in a segment.
template <int D, bool E4M3, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1)
    paged_decode_kernel(const DecodeArgs a, int chunks) {
  using G = Geo<D, E4M3>;
  constexpr int RB = G::RB, TK = G::TK, NS = G::NS, CPR = G::CPR, RPI = G::RPI;
  constexpr int OS = D + 4;                     // row stride of the join buffer
  constexpr float kShift = E4M3 ? 12.f : 0.f;   // weights carry 2^12 so that f16 holds small ones
  extern __shared__ __align__(128) uint8_t smem[];
  float* s_o = reinterpret_cast<float*>(smem + kWarps * kStages * kStageBytes);
  __shared__ float s_m[kWarps][kHeads], s_l[kWarps][kHeads];
  __shared__ int s_cnt[kWarps][kStages];
  __shared__ long long s_sum[kWarps], s_off;
  __shared__ int s_b;

  const int tid = threadIdx.x, lane = lane_id(), w = warp_id();
  const int g = lane >> 2, t = lane & 3;
  const int group = a.Hq / a.Hkv, segs = a.Hkv * chunks;
  long long* prefix = static_cast<long long*>(a.ws);
  float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + parts_offset());

  // the dependent launch may be set up; it waits for this one to finish
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- this CTA's share
  long long total = 0;
  for (int b = tid; b < a.B; b += kThreads) {
    const int len = a.lens[b];
    if (blockIdx.x == 0 && len != 0 && list_rows(a, len) == 0) atomicOr(a.status, DEV_BOUNDS);
    total += tiles_of<TK>(a, b);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (lane == 0) s_sum[w] = total;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) total += s_sum[i];
  __syncthreads();
  const long long all = total * segs;
  const long long ctas = active_ctas(all, gridDim.x);
  if (blockIdx.x > 0 && (blockIdx.x >= ctas || all == 0)) return;
  const long long lo = blockIdx.x * all / ctas, hi = (blockIdx.x + 1) * all / ctas;
  long long carry = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + tid;
    const long long own = b < a.B ? tiles_of<TK>(a, b) : 0;
    long long x = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) s_sum[w] = x;
    __syncthreads();
    long long chunk = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < w) x += s_sum[i];
      chunk += s_sum[i];
    }
    const long long first = (carry + x - own) * segs, end = (carry + x) * segs;
    if (own > 0 && first <= lo && lo < end) {
      s_b = b;
      s_off = lo - first;
    }
    if (blockIdx.x == 0 && b < a.B) prefix[b] = carry + x - own;
    carry += chunk;
    __syncthreads();
  }
  if (blockIdx.x == 0 && tid == 0) prefix[a.B] = total;
  if (all == 0) return;

  Walk here;
  here.b = s_b;
  here.tb = tiles_of<TK>(a, here.b);
  here.seg = static_cast<int>(s_off / here.tb);
  here.t0 = static_cast<int>(s_off % here.tb);
  here.count = static_cast<int>(min(static_cast<long long>(here.tb - here.t0), hi - lo));
  here.left = hi - lo - here.count;

  // ---- the warp's ring: its tiles of every segment, three ahead
  uint8_t* ring = smem + w * (kStages * kStageBytes);
  const uint32_t ring_s = smem_u32(ring);
  Walk ahead = here;
  int k_next = 0;          // next tile of `ahead` to load: t0 + w + 8 k_next
  uint32_t found = 0;      // lane i: page and rows of slab i % NS of tile k0 + i / NS
  bool more = true;
  const int l_row = lane / CPR, l_chunk = lane % CPR;

  auto look_up = [&](int k) {
    const int kk = k + lane / NS;
    const long long row0 = static_cast<long long>(ahead.t0 + w + kWarps * kk) * TK + lane % NS * 16;
    found = 0;
    if (w + kWarps * kk >= ahead.count) return;
    const int len = a.lens[ahead.b];
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
    const int pid = a.table[static_cast<size_t>(ahead.b) * a.max_pages + j];
    if (pid < 0 || pid >= a.num_pages) {
      atomicOr(a.status, DEV_BOUNDS);
      return;
    }
    const int rows = min(16, max(0, len - j * a.page - inner));
    found = static_cast<uint32_t>(pid) | (static_cast<uint32_t>(rows) << kPidBits);
  };

  auto load_next = [&](int stage) {
    while (more && w + kWarps * k_next >= ahead.count) {
      more = next_segment<TK>(ahead, a, segs);
      k_next = 0;
    }
    if (more) {
      constexpr int kWindow = 32 / NS;
      if (k_next % kWindow == 0) look_up(k_next);
      const int h = ahead.seg / chunks;
      const int row0 = (ahead.t0 + w + kWarps * k_next) * TK & (a.page - 1);
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

  while (true) {
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
            const uint2 v = *reinterpret_cast<const uint2*>(p + 4 * t);
            x = bf16x2_to_f16x2(v.x);
            y = bf16x2_to_f16x2(v.y);
          } else {
            x = *reinterpret_cast<const uint32_t*>(p + 2 * t);
            y = *reinterpret_cast<const uint32_t*>(p + 8 + 2 * t);
          }
        }
        qa[i][r] = x;
        qa[i][r + 2] = y;
      }
    }
    float o[NT][4] = {};
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (int k = w; k < here.count; k += kWarps) {
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
      // weights (bf16: two parts, 2^-16 off; f16: one, 2^-11 off, the values exact)
      const float off0 = kShift - (m[0] == -INFINITY ? 0.f : m[0] * a.scale_log2);
      const float off1 = kShift - (m[1] == -INFINITY ? 0.f : m[1] * a.scale_log2);
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        uint32_t p[4], pl[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float* x = s[2 * i + j];
#pragma unroll
          for (int e = 0; e < (WIDE ? 4 : 2); ++e) {
            x[e] = ex2(fmaf(x[e], a.scale_log2, e < 2 ? off0 : off1));
            l[e >> 1] += x[e];
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            if (r == 1 && !WIDE) {
              p[2 * j + 1] = pl[2 * j + 1] = 0;
            } else if (E4M3) {
              p[2 * j + r] = pack_f16(x[2 * r], x[2 * r + 1]);
            } else {
              const uint32_t hb = pack_bf16(x[2 * r], x[2 * r + 1]);
              p[2 * j + r] = hb;
              pl[2 * j + r] = pack_bf16(x[2 * r] - __uint_as_float(hb << 16),
                                        x[2 * r + 1] - __uint_as_float(hb & 0xFFFF0000u));
            }
          }
        }
        const int r = 16 * i + (lane & 15);
#pragma unroll
        for (int c = 0; c < CPR; c += 2) {
          uint32_t f[4];
          ldm4t(vs + swz<RB>(r, c + (lane >> 4)), f);
          if (E4M3) {
            // bytes (key 2t, values 2g and 2g + 1), (key 2t + 1, the same): even
            // and odd values become two 8-column tiles
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              uint32_t a0, a1, b0, b1;
              e4m3x4_to_f16x4(f[2 * u], a0, a1);
              e4m3x4_to_f16x4(f[2 * u + 1], b0, b1);
              mma<true>(o[2 * (c + u)], p, __byte_perm(a0, a1, 0x5410), __byte_perm(b0, b1, 0x5410));
              mma<true>(o[2 * (c + u) + 1], p, __byte_perm(a0, a1, 0x7632),
                        __byte_perm(b0, b1, 0x7632));
            }
          } else {
            mma<false>(o[c], p, f[0], f[1]);
            mma<false>(o[c + 1], p, f[2], f[3]);
            mma<false>(o[c], pl, f[0], f[1]);
            mma<false>(o[c + 1], pl, f[2], f[3]);
          }
        }
      }
      __syncwarp();
      load_next(stage);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }

    // ---- join the warps
#pragma unroll
    for (int r = 0; r < (WIDE ? 2 : 1); ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      m[r] *= a.scale_log2;
      if (t == 0) {
        s_m[w][g + 8 * r] = m[r];
        s_l[w][g + 8 * r] = l[r];
      }
    }
    __syncthreads();
    const bool whole = here.t0 == 0 && here.count == here.tb;
    float* part = parts + (2 * static_cast<size_t>(blockIdx.x) + (here.t0 == 0 ? 1 : 0)) * part_floats(D);
#pragma unroll
    for (int r = 0; r < (WIDE ? 2 : 1); ++r) {
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) top = fmaxf(top, s_m[i][g + 8 * r]);
      const float f = m[r] == -INFINITY ? 0.f : ex2(m[r] - top);
      float* to = s_o + (w * 8 + g) * OS;
      if (f != 0.f) {
#pragma unroll
        for (int c = 0; c < NT; c += 2) {
          if (E4M3) {
            *reinterpret_cast<float4*>(to + 8 * c + 4 * t) =
                make_float4(o[c][2 * r] * f, o[c + 1][2 * r] * f, o[c][2 * r + 1] * f,
                            o[c + 1][2 * r + 1] * f);
          } else {
            *reinterpret_cast<float2*>(to + 8 * c + 2 * t) =
                make_float2(o[c][2 * r] * f, o[c][2 * r + 1] * f);
            *reinterpret_cast<float2*>(to + 8 * c + 8 + 2 * t) =
                make_float2(o[c + 1][2 * r] * f, o[c + 1][2 * r + 1] * f);
          }
        }
      }
      __syncthreads();
      const int row = tid / (D / 4), col = tid % (D / 4) * 4;  // 8 rows, four columns per thread
      const int head = row + 8 * r;
      if (row < 8 && head < heads) {
        float best = -INFINITY, sum = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) best = fmaxf(best, s_m[i][head]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
          const float mi = s_m[i][head];
          const float fi = mi == -INFINITY ? 0.f : ex2(mi - best);
          if (fi != 0.f) {  // a warp of no weight has written nothing
            sum += s_l[i][head] * fi;
            const float4 x = *reinterpret_cast<const float4*>(s_o + (i * 8 + row) * OS + col);
            acc.x += x.x;
            acc.y += x.y;
            acc.z += x.z;
            acc.w += x.w;
          }
        }
        if (whole) {
          const float inv = sum > 0.f || sum != sum ? a.v_scale / sum : 0.f;
          const size_t at = static_cast<size_t>(here.b) * a.Hq + h * group + q0 + head;
          *reinterpret_cast<uint2*>(a.out + at * D + col) =
              make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
          if (a.lse != nullptr && col == 0)
            a.lse[at] = sum == 0.f ? -INFINITY : (best + (log2f(sum) - kShift)) * 0.6931471805599453f;
        } else {
          if (col == 0) {
            part[2 * head] = best;
            part[2 * head + 1] = sum;
          }
          *reinterpret_cast<float4*>(part + 2 * kHeads + head * D + col) = acc;
        }
      }
      __syncthreads();
    }
    if (!next_segment<TK>(here, a, segs)) break;
  }
  cp_async_wait_group<0>();
}

// One block per query head: joins the parts of a segment that several CTAs
// share, in the order of their tiles, and writes the rows of sequences that
// hold nothing.
template <int D, int TK>
__global__ void __launch_bounds__(2 * D) paged_join_kernel(const DecodeArgs a, int chunks, int grid,
                                                           float shift) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.x / a.Hq, hq = blockIdx.x % a.Hq, group = a.Hq / a.Hkv;
  const int h = hq / group, row = hq % group % kHeads;
  const int seg = h * chunks + hq % group / kHeads, segs = a.Hkv * chunks;
  const long long* prefix = static_cast<const long long*>(a.ws);
  const float* parts =
      reinterpret_cast<const float*>(static_cast<const uint8_t*>(a.ws) + parts_offset());
  const long long p0 = prefix[b], tb = prefix[b + 1] - p0, all = prefix[a.B] * segs;
  const int col = threadIdx.x % D, side = threadIdx.x / D;
  if (tb == 0) {
    if (side == 0) a.out[static_cast<size_t>(blockIdx.x) * D + col] = __float2bfloat16(0.f);
    if (a.lse != nullptr && threadIdx.x == 0) a.lse[blockIdx.x] = -INFINITY;
    return;
  }
  const long long ctas = active_ctas(all, grid), first = p0 * segs + seg * tb;
  const int c0 = static_cast<int>(((first + 1) * ctas - 1) / all);
  const int c1 = static_cast<int>(((first + tb) * ctas - 1) / all);
  if (c0 == c1) return;
  // CTA c0 holds the segment's first tile (its second part), the others go on
  // with it (their first parts); two threads per column take every other part
  float top = -INFINITY, sum = 0.f, acc = 0.f;
  for (int c = c0; c <= c1; ++c)
    top = fmaxf(top, parts[(2 * static_cast<size_t>(c) + (c == c0)) * part_floats(D) + 2 * row]);
  for (int c = c0 + side; c <= c1; c += 2) {
    const float* part = parts + (2 * static_cast<size_t>(c) + (c == c0)) * part_floats(D);
    const float m = part[2 * row];
    if (m == -INFINITY) continue;
    const float f = ex2(m - top);
    sum += part[2 * row + 1] * f;
    acc += part[2 * kHeads + row * D + col] * f;
  }
  __shared__ float s_sum, s_acc[D];
  if (side == 1) {
    s_acc[col] = acc;
    if (col == 0) s_sum = sum;
  }
  __syncthreads();
  if (side == 0) {
    sum += s_sum;
    acc += s_acc[col];
    const float inv = sum > 0.f || sum != sum ? a.v_scale / sum : 0.f;
    a.out[static_cast<size_t>(blockIdx.x) * D + col] = __float2bfloat16(acc * inv);
    if (a.lse != nullptr && col == 0)
      a.lse[blockIdx.x] = sum == 0.f ? -INFINITY : (top + (log2f(sum) - shift)) * 0.6931471805599453f;
  }
}

template <int D, bool E4M3, bool WIDE>
cudaError_t launch(const DecodeArgs& a, int chunks, int sms, cudaStream_t stream) {
  using G = Geo<D, E4M3>;
  constexpr int kSmem = kWarps * kStages * kStageBytes + kWarps * 8 * (D + 4) * 4;
  auto kernel = paged_decode_kernel<D, E4M3, WIDE>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  // no more CTAs than the longest lists could fill
  const long long rows = a.sel != nullptr
                             ? static_cast<long long>(std::min(a.select, a.max_pages)) * a.page
                             : static_cast<long long>(a.max_pages) * a.page;
  const long long most = static_cast<long long>(a.B) * a.Hkv * chunks * ((rows + G::TK - 1) / G::TK);
  const int grid = static_cast<int>(
      std::min<long long>(std::min(sms, kMaxCtas), (most + kMinTiles - 1) / kMinTiles));
  kernel<<<grid, kThreads, kSmem, stream>>>(a, chunks);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.B * a.Hq);
  cfg.blockDim = dim3(2 * D);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<D, G::TK>, a, chunks, grid, E4M3 ? 12.f : 0.f);
}

}  // namespace

size_t paged_decode_workspace_bytes(int D) {
  return parts_offset() + 2 * kMaxCtas * part_floats(D) * sizeof(float);
}

cudaError_t launch_paged_decode(const DecodeArgs& a, bool e4m3, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  const int group = a.Hq / a.Hkv, chunks = (group + kHeads - 1) / kHeads;
  const bool wide = group > 8;
  if (a.D == 128) {
    if (e4m3) return wide ? launch<128, true, true>(a, chunks, sms, stream) : launch<128, true, false>(a, chunks, sms, stream);
    return wide ? launch<128, false, true>(a, chunks, sms, stream) : launch<128, false, false>(a, chunks, sms, stream);
  }
  if (e4m3) return wide ? launch<64, true, true>(a, chunks, sms, stream) : launch<64, true, false>(a, chunks, sms, stream);
  return wide ? launch<64, false, true>(a, chunks, sms, stream) : launch<64, false, false>(a, chunks, sms, stream);
}

}  // namespace mcs
