// RMS norm of each head of q and k and the rotation by position, one pass, and
// the gradients of both.
//
//   r = 1 / sqrt(mean(x^2) + eps), y = x r w,
//   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)
//
// D/8 threads hold a row (one head of one token), 8 values each, as four pairs
// (a, b) of the rotation: neighbours in memory when interleaved, else four
// values of each half, so that no value crosses threads and only the mean is a
// shuffle sum.  Values that are not rotated are pairs of angle 0.  The weights
// are multiplied into a token's cosines and sines once for the heads a warp
// takes (8, or 32 at D = 64; gradients 4 or 8, and 8 at D = 64): y_a' = r (x_a (w_a cos) - x_b (w_b sin)).  Pairs of values go through
// the packed fp32 instructions.
//
// Bound: HBM, 4 bytes per value (6 for the gradients), at about 45 (85)
// instructions per 512 bytes of a row pair.  The warps of a block take
// consecutive tokens, so that a head's rows of a [B, H, N, D] output are
// written next to each other.
#include <algorithm>

#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace mcs {
namespace {

constexpr int kRopeWarps = 8;
constexpr int kRopeThreads = 32 * kRopeWarps;
// Loads in flight per thread and blocks per SM, measured: forward 4 at D = 128 and 8 at
// D = 64, whose rows are half as long (75600 tokens, 64 heads of D = 64: 84 -> 90 % of
// copy bandwidth).  The gradients have two forms, 2 rows of x and dy per thread and 3 blocks, or
// 4 and 2, which takes twice the heads at a time.  At D = 128 and with heads that fill the warps, 4
// rows are faster where the tokens' positions are given and slower where they are not (why, is not
// known): 40000 tokens, 40 + 8 heads, 217 us and 236 with 2 rows, without positions 261 and 234;
// 75600 tokens, 40 + 40 heads 697 and 768, without positions 804 and 732; below 3000 tokens they are
// within 3 %.  Heads that do not fill them: 32760 tokens, 12 + 12 heads 103 us and 97.  D = 64: 75600
// tokens, 32 + 32 heads 325 and 300.  (D = 128, 2 rows and 4 blocks: spills, 40 + 8 heads 410.)
template <int D> struct Tune {
  static constexpr int STEPS = 512 / D, BLOCKS = D == 128 ? 4 : 3, FEW_BLOCKS = BLOCKS;
};
constexpr int kFewSteps = 2;  // gradients of few heads (and FEW_BLOCKS)
__host__ __device__ constexpr int grad_blocks(int steps) { return steps == 2 ? 3 : 2; }
constexpr int kGradBlocks = 2048;  // most partial sums of the weight gradients, half of them of k

// Heads of one token a warp takes.
__host__ __device__ constexpr int heads_per_warp(int D, int steps) { return steps * (256 / D); }

struct Row {  // 8 bf16 values as loaded: pairs' first and second members
  uint32_t w[4];
};

// Where a thread's values lie in a row: 8 consecutive ones (interleaved), or
// four at `a` and four at `b` (split: thread l < rot/8 holds 4l.. of both
// halves, the others 8 of the values behind the rotated ones).
struct Place {
  int a, b;
};
template <bool SPLIT>
__device__ __forceinline__ Place place_of(int rot, int l) {
  if (!SPLIT) return {8 * l, 8 * l + 4};
  const int lanes = rot / 8;
  if (l < lanes) return {4 * l, rot / 2 + 4 * l};
  return {8 * l, 8 * l + 4};
}

// Rows may be overwritten later by the thread that reads them (in-place calls).
template <bool SPLIT>
__device__ __forceinline__ Row load_row(const __nv_bfloat16* p, Place at) {
  Row r;
  if (SPLIT) {
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                 : "=r"(r.w[0]), "=r"(r.w[1]) : "l"(p + at.a) : "memory");
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                 : "=r"(r.w[2]), "=r"(r.w[3]) : "l"(p + at.b) : "memory");
  } else {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
                 : "l"(p + at.a)
                 : "memory");
  }
  return r;
}
__device__ __forceinline__ uint64_t two(uint32_t lo, uint32_t hi) {
  return f2_pack(__uint_as_float(lo), __uint_as_float(hi));
}
// a[0], a[1]: the pairs' first members, b: the second ones.
template <bool SPLIT>
__device__ __forceinline__ void unpack(const Row& r, uint64_t* a, uint64_t* b) {
  constexpr uint32_t kHi = 0xFFFF0000u;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (SPLIT) {
      a[i] = two(r.w[i] << 16, r.w[i] & kHi);
      b[i] = two(r.w[i + 2] << 16, r.w[i + 2] & kHi);
    } else {
      a[i] = two(r.w[2 * i] << 16, r.w[2 * i + 1] << 16);
      b[i] = two(r.w[2 * i] & kHi, r.w[2 * i + 1] & kHi);
    }
  }
}
template <bool SPLIT>
__device__ __forceinline__ void store_row(__nv_bfloat16* p, Place at, const uint64_t* a,
                                          const uint64_t* b) {
  float a0, a1, a2, a3, b0, b1, b2, b3;
  f2_unpack(a[0], a0, a1);
  f2_unpack(a[1], a2, a3);
  f2_unpack(b[0], b0, b1);
  f2_unpack(b[1], b2, b3);
  if (SPLIT) {
    *reinterpret_cast<uint2*>(p + at.a) = make_uint2(pack_bf16(a0, a1), pack_bf16(a2, a3));
    *reinterpret_cast<uint2*>(p + at.b) = make_uint2(pack_bf16(b0, b1), pack_bf16(b2, b3));
  } else {
    *reinterpret_cast<uint4*>(p + at.a) =
        make_uint4(pack_bf16(a0, b0), pack_bf16(a1, b1), pack_bf16(a2, b2), pack_bf16(a3, b3));
  }
}

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_neg(uint64_t a) { return a ^ 0x8000000080000000ull; }
__device__ __forceinline__ float f2_sum(uint64_t a) {
  float x, y;
  f2_unpack(a, x, y);
  return x + y;
}

// Cosines and sines of the thread's pairs (1 and 0 where nothing is rotated, and for a row that is none).
__device__ __forceinline__ void load_angles(const RopeArgs& a, int pos, int l, uint64_t* cs,
                                            uint64_t* sn) {
  float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (8 * l < a.rot && pos >= 0) {
    const size_t at = static_cast<size_t>(pos) * (a.rot / 2) + 4 * l;
    c = *reinterpret_cast<const float4*>(a.cos_table + at);
    s = *reinterpret_cast<const float4*>(a.sin_table + at);
  }
  cs[0] = f2_pack(c.x, c.y);
  cs[1] = f2_pack(c.z, c.w);
  sn[0] = f2_pack(s.x, s.y);
  sn[1] = f2_pack(s.z, s.w);
}
// The thread's weights, as the pairs' members.
template <bool SPLIT>
__device__ __forceinline__ void load_weights(const float* w, Place at, uint64_t* a, uint64_t* b) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = w ? w[at.a + i] : 1.f;
    x[i + 4] = w ? w[at.b + i] : 1.f;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    a[i] = SPLIT ? f2_pack(x[2 * i], x[2 * i + 1]) : f2_pack(x[4 * i], x[4 * i + 2]);
    b[i] = SPLIT ? f2_pack(x[4 + 2 * i], x[5 + 2 * i]) : f2_pack(x[4 * i + 1], x[4 * i + 3]);
  }
}

template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A token (below 2^31): its batch entry and place in it, and its position, or
// -1 where its rows stay as they are.
struct Token {
  int b, n, pos;
};
__device__ __forceinline__ Token token_of(const RopeArgs& a, unsigned token) {
  Token t;
  t.b = static_cast<int>(token / static_cast<unsigned>(a.N));
  t.n = static_cast<int>(token - static_cast<unsigned>(t.b) * a.N);
  t.pos = a.positions ? a.positions[token] : t.n;
  if (a.rot > 0 && t.pos >= a.table_rows) {
    atomicOr(a.status, DEV_BOUNDS);
    t.pos = -1;
  }
  return t;
}
// Head 0 of the token in the [B, H, N, D] or [B, N, H, D] tensors, and the step to the next head.
__device__ __forceinline__ size_t out_base(const RopeArgs& a, const Token& t, int H, size_t* step) {
  const bool by_token = a.layout == MCS_LAYOUT_BNHD;
  *step = by_token ? a.D : static_cast<size_t>(a.N) * a.D;
  return by_token ? (static_cast<size_t>(t.b) * a.N + t.n) * H * a.D
                  : (static_cast<size_t>(t.b) * H * a.N + t.n) * a.D;
}

template <int D, bool SPLIT>
__global__ void __launch_bounds__(kRopeThreads, Tune<D>::BLOCKS)
    norm_rope_kernel(const RopeArgs a, int chunks_q, int chunks) {
  constexpr int LANES = D / 8, ROWS = 32 / LANES, STEPS = Tune<D>::STEPS;  // ROWS: rows per load
  pdl_begin();
  const unsigned tile = blockIdx.x / static_cast<unsigned>(chunks);
  const int chunk = static_cast<int>(blockIdx.x - tile * chunks);
  const unsigned token = tile * kRopeWarps + warp_id();
  if (token >= static_cast<unsigned>(a.B) * a.N) return;
  const Token t = token_of(a, token);
  if (t.pos < 0) return;
  const bool is_q = chunk < chunks_q;
  const int H = is_q ? a.Hq : a.Hkv;
  const int l = lane_id() % LANES, h0 = (is_q ? chunk : chunk - chunks_q) * heads_per_warp(D, Tune<D>::STEPS) + lane_id() / LANES;
  const Place at = place_of<SPLIT>(a.rot, l);
  const __nv_bfloat16* src = (is_q ? a.q : a.k) + token * (is_q ? a.q_stride : a.k_stride) + h0 * D;
  Row x[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    x[i] = Row{{0, 0, 0, 0}};
    if (h0 + i * ROWS < H) x[i] = load_row<SPLIT>(src + i * ROWS * D, at);
  }
  uint64_t ac[2], as[2], bc[2], bs[2];
  {
    uint64_t cs[2], sn[2], wa[2], wb[2];
    load_angles(a, t.pos, l, cs, sn);
    load_weights<SPLIT>(is_q ? a.wq : a.wk, at, wa, wb);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ac[i] = f2_mul(wa[i], cs[i]);
      as[i] = f2_mul(wa[i], sn[i]);
      bc[i] = f2_mul(wb[i], cs[i]);
      bs[i] = f2_neg(f2_mul(wb[i], sn[i]));
    }
  }
  size_t step;
  __nv_bfloat16* dst = (is_q ? a.q_out : a.k_out) + out_base(a, t, H, &step);
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    uint64_t p[2], q[2], u[2], v[2];
    unpack<SPLIT>(x[i], p, q);
    uint64_t ss = f2_mul(p[0], p[0]);
    ss = f2_fma(p[1], p[1], ss);
    ss = f2_fma(q[0], q[0], ss);
    ss = f2_fma(q[1], q[1], ss);
    const float r = rsqrtf(row_sum<LANES>(f2_sum(ss)) * (1.f / D) + a.eps);
    const uint64_t rr = f2_pack(r, r);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      u[k] = f2_mul(f2_fma(p[k], ac[k], f2_mul(q[k], bs[k])), rr);
      v[k] = f2_mul(f2_fma(q[k], bc[k], f2_mul(p[k], as[k])), rr);
    }
    const int h = h0 + i * ROWS;
    if (h < H) store_row<SPLIT>(dst + h * step, at, u, v);
  }
}

// x / rms(x), as the pairs' members.
template <int D, bool SPLIT>
__device__ __forceinline__ void normed(const Row& x, float eps, uint64_t* u, uint64_t* v) {
  unpack<SPLIT>(x, u, v);
  uint64_t ss = f2_mul(u[0], u[0]);
  ss = f2_fma(u[1], u[1], ss);
  ss = f2_fma(v[0], v[0], ss);
  ss = f2_fma(v[1], v[1], ss);
  const float r = rsqrtf(row_sum<D / 8>(f2_sum(ss)) * (1.f / D) + eps);
  const uint64_t rr = f2_pack(r, r);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    u[k] = f2_mul(u[k], rr);
    v[k] = f2_mul(v[k], rr);
  }
}

// A tensor with at most half of the heads that a warp takes of one token (4, or 16 at D = 64;
// gradients 2 and 4): the warp takes the heads of several consecutive tokens, with angles for each row.  One
// tensor per launch.
struct One {
  int H, tokens;  // heads; tokens per warp
  long long stride;
  const __nv_bfloat16* x;
  __nv_bfloat16* out;           // q_out / k_out; backward: dq / dk
  const __nv_bfloat16* dy;      // backward
  const float* w;
  float* partial;               // backward: the blocks' sums
};
// Row r of a warp's rows: where it lies in x and in the output-shaped tensors, and its
// position (-1: none, or a row that stays as it is).
struct RowAt {
  size_t x, y;
  int pos;
};
__device__ __forceinline__ RowAt row_at(const RopeArgs& a, const One& one, unsigned warp, int r) {
  RowAt p = {0, 0, -1};
  const int k = r / one.H, h = r - k * one.H;
  const unsigned token = warp * one.tokens + k;
  if (k >= one.tokens || token >= static_cast<unsigned>(a.B) * a.N) return p;
  const Token t = token_of(a, token);
  size_t step;
  p.y = out_base(a, t, one.H, &step);
  p.y += h * step;
  p.x = token * one.stride + h * a.D;
  p.pos = t.pos;
  return p;
}

template <int D, bool SPLIT>
__global__ void __launch_bounds__(kRopeThreads, Tune<D>::BLOCKS)
    norm_rope_few_kernel(const RopeArgs a, const One one) {
  constexpr int LANES = D / 8, ROWS = 32 / LANES, STEPS = Tune<D>::STEPS;
  pdl_begin();
  const int l = lane_id() % LANES;
  const Place at = place_of<SPLIT>(a.rot, l);
  const unsigned warp = blockIdx.x * kRopeWarps + warp_id();
  RowAt p[STEPS];
  Row x[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    p[i] = row_at(a, one, warp, i * ROWS + lane_id() / LANES);
    x[i] = Row{{0, 0, 0, 0}};
    if (p[i].pos >= 0) x[i] = load_row<SPLIT>(one.x + p[i].x, at);
  }
  uint64_t wa[2], wb[2];
  load_weights<SPLIT>(one.w, at, wa, wb);
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    uint64_t cs[2], sn[2], u[2], v[2];
    load_angles(a, p[i].pos, l, cs, sn);
    normed<D, SPLIT>(x[i], a.eps, u, v);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      u[k] = f2_mul(u[k], wa[k]);
      v[k] = f2_mul(v[k], wb[k]);
      const uint64_t s = f2_mul(v[k], f2_neg(sn[k]));
      v[k] = f2_fma(v[k], cs[k], f2_mul(u[k], sn[k]));
      u[k] = f2_fma(u[k], cs[k], s);
    }
    if (p[i].pos >= 0) store_row<SPLIT>(one.out + p[i].y, at, u, v);
  }
}

// The block's sum of its threads' weight gradients.
template <int D, bool SPLIT>
__device__ __forceinline__ void block_weight_sum(const uint64_t* da, const uint64_t* db, Place at, int r0, float* out) {
  constexpr int ROWS = 256 / D;
  __shared__ float part[kRopeWarps * ROWS][D];
  float s[8];
  f2_unpack(da[0], s[0], s[1]);
  f2_unpack(da[1], s[2], s[3]);
  f2_unpack(db[0], s[4], s[5]);
  f2_unpack(db[1], s[6], s[7]);
  float* to = part[warp_id() * ROWS + r0];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    to[SPLIT ? at.a + k : at.a + 2 * k] = s[k];
    to[SPLIT ? at.b + k : at.a + 2 * k + 1] = s[4 + k];
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float sum = 0;
#pragma unroll
    for (int i = 0; i < kRopeWarps * ROWS; ++i) sum += part[i][threadIdx.x];
    out[threadIdx.x] = sum;
  }
}

// Backward: units of 8 tokens and a warp's heads as above; a block takes every
// blocks_q-th unit of q (or blocks_k-th of k) and keeps the weight gradient of
// its units in registers, one partial row per block at the end.
//   g = dy rotated back, dx = r (w g - x r^2 mean(w g x)), dw += g x r
// 16 bytes on their way to shared memory, zeros unless `live`.
__device__ __forceinline__ void copy16(uint8_t* to, const void* from, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(live ? 16 : 0) : "memory");
}
// A thread's values of a row in shared memory.
template <bool SPLIT>
__device__ __forceinline__ Row row_in(const uint8_t* p, Place at) {
  Row r;
  const __nv_bfloat16* row = reinterpret_cast<const __nv_bfloat16*>(p);
  if (SPLIT) {
    const uint2 x = *reinterpret_cast<const uint2*>(row + at.a), y = *reinterpret_cast<const uint2*>(row + at.b);
    r.w[0] = x.x, r.w[1] = x.y, r.w[2] = y.x, r.w[3] = y.y;
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(row + at.a);
    r.w[0] = x.x, r.w[1] = x.y, r.w[2] = x.z, r.w[3] = x.w;
  }
  return r;
}
__device__ __forceinline__ void angles_in(const uint8_t* cos4, const uint8_t* sin4, bool rotated, uint64_t* cs, uint64_t* sn) {
  const float4 one = make_float4(1.f, 1.f, 1.f, 1.f), zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const float4 c = rotated ? *reinterpret_cast<const float4*>(cos4) : one;
  const float4 s = rotated ? *reinterpret_cast<const float4*>(sin4) : zero;
  cs[0] = f2_pack(c.x, c.y), cs[1] = f2_pack(c.z, c.w);
  sn[0] = f2_pack(s.x, s.y), sn[1] = f2_pack(s.z, s.w);
}
// dx of a row (its pairs' members to c and d), and its part of the weight gradients added to da, db.
// A row that is not `live` (no such row, or padding) holds zeros, whose 1 / rms is infinite at
// eps = 0, and adds nothing.
template <int D, bool SPLIT>
__device__ __forceinline__ void row_gradient(const Row& x, const Row& y, bool live, float eps, const uint64_t* cs, const uint64_t* sn,
                                             const uint64_t* wa, const uint64_t* wb, uint64_t* c, uint64_t* d, uint64_t* da,
                                             uint64_t* db) {
  uint64_t p[2], q[2], g[2], f[2], ss = 0, dot = 0;
  unpack<SPLIT>(x, p, q);
  unpack<SPLIT>(y, c, d);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    ss = f2_fma(q[k], q[k], f2_fma(p[k], p[k], ss));
    g[k] = f2_fma(c[k], cs[k], f2_mul(d[k], sn[k]));
    f[k] = f2_fma(d[k], cs[k], f2_neg(f2_mul(c[k], sn[k])));
    c[k] = f2_mul(g[k], wa[k]);
    d[k] = f2_mul(f[k], wb[k]);
    dot = f2_fma(d[k], q[k], f2_fma(c[k], p[k], dot));
  }
  float s1 = f2_sum(ss), s2 = f2_sum(dot);
  s1 = row_sum<D / 8>(s1);
  s2 = row_sum<D / 8>(s2);
  const float r = live ? rsqrtf(s1 * (1.f / D) + eps) : 0.f, m = -(s2 * (1.f / D)) * r * r;
  const uint64_t rr = f2_pack(r, r), mm = f2_pack(m, m);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    da[k] = f2_fma(f2_mul(g[k], rr), p[k], da[k]);
    db[k] = f2_fma(f2_mul(f[k], rr), q[k], db[k]);
    c[k] = f2_mul(f2_fma(p[k], mm, c[k]), rr);
    d[k] = f2_mul(f2_fma(q[k], mm, d[k]), rr);
  }
}

// A warp's next unit (rows of x and dy, angles) is on its way to shared memory while it
// computes one, and the position after that to a register (with loads to registers, one unit
// after the other, 32760 tokens of 12 + 12 heads took 109 us).
__host__ __device__ constexpr int kGradStage(int steps) { return 2 * steps * 512 + 512; }  // bytes of x and dy, then the angles
constexpr int kGradStages = 2;

template <int D, bool SPLIT, int STEPS>
__global__ void __launch_bounds__(kRopeThreads, grad_blocks(STEPS))
    norm_rope_backward_kernel(const RopeArgs a, int blocks_q, int blocks_k) {
  constexpr int LANES = D / 8, ROWS = 32 / LANES, HEADS = heads_per_warp(D, STEPS);
  constexpr int STAGE = kGradStage(STEPS), ANGLES = 2 * STEPS * 512;
  extern __shared__ __align__(16) uint8_t grad_smem[];
  pdl_begin();
  const bool is_q = static_cast<int>(blockIdx.x) < blocks_q;
  const int H = is_q ? a.Hq : a.Hkv;
  const unsigned chunks = (H + HEADS - 1) / HEADS;
  const unsigned block = is_q ? blockIdx.x : blockIdx.x - blocks_q, blocks = is_q ? blocks_q : blocks_k;
  const unsigned tokens = static_cast<unsigned>(a.B) * a.N;
  const int lane = lane_id(), l = lane % LANES, r0 = lane / LANES;
  const Place at = place_of<SPLIT>(a.rot, l);
  const __nv_bfloat16* xs = is_q ? a.q : a.k;
  const __nv_bfloat16* dys = is_q ? a.dq_out : a.dk_out;
  __nv_bfloat16* dxs = is_q ? a.q_out : a.k_out;
  const long long stride = is_q ? a.q_stride : a.k_stride;
  uint8_t* ring = grad_smem + warp_id() * (kGradStages * STAGE);
  uint64_t wa[2], wb[2], da[2] = {0, 0}, db[2] = {0, 0};
  load_weights<SPLIT>(is_q ? a.wq : a.wk, at, wa, wb);

  // a warp's unit: its token and chunk of heads (pos < 0: no token, or rows that stay as they are)
  struct Unit {
    unsigned token, chunk;
    Token t;
  };
  auto find = [&](Unit& u) {
    u.t.pos = -1;
    if (u.token < tokens) u.t = token_of(a, u.token);
  };
  const unsigned tile_step = blocks / chunks, chunk_step = blocks - tile_step * chunks;
  auto after = [&](const Unit& u) {
    Unit v = u;
    v.chunk += chunk_step;
    const bool over = v.chunk >= chunks;
    if (over) v.chunk -= chunks;
    v.token += kRopeWarps * (tile_step + over);
    find(v);
    return v;
  };
  auto fetch = [&](const Unit& u, uint8_t* stage) {
    if (u.t.pos >= 0) {
      const int h0 = static_cast<int>(u.chunk) * HEADS + r0;
      size_t step;
      const size_t y0 = out_base(a, u.t, H, &step) + 8 * l;
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        // (heads past the last one: its x, so that 1 / rms is a number whatever eps is, and zeros as dy)
        const int h = h0 + i * ROWS, hc = min(h, H - 1);
        copy16(stage + i * 512 + lane * 16, xs + u.token * stride + hc * D + 8 * l, true);
        copy16(stage + (STEPS + i) * 512 + lane * 16, dys + y0 + hc * step, h < H);
      }
      if (r0 < 2 && 8 * l < a.rot) {
        const float* table = r0 == 0 ? a.cos_table : a.sin_table;
        copy16(stage + ANGLES + r0 * 256 + l * 16, table + static_cast<size_t>(u.t.pos) * (a.rot / 2) + 4 * l, true);
      }
    }
    cp_async_commit();
  };
  Unit now = {block / chunks * kRopeWarps + warp_id(), block % chunks, {}};
  find(now);
  Unit next = after(now);
  int turn = 0;
  fetch(now, ring);
  while (now.token < tokens) {
    fetch(next, ring + (turn ^ 1) * STAGE);
    const Unit later = after(next);
    cp_async_wait_group<1>();
    __syncwarp();
    if (now.t.pos >= 0) {
      const uint8_t* stage = ring + turn * STAGE;
      const int h0 = static_cast<int>(now.chunk) * HEADS + r0;
      __nv_bfloat16* dx = dxs + now.token * stride + h0 * D;
      uint64_t cs[2], sn[2];
      angles_in(stage + ANGLES + l * 16, stage + ANGLES + 256 + l * 16, 8 * l < a.rot, cs, sn);
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        uint64_t c[2], d[2];
        row_gradient<D, SPLIT>(row_in<SPLIT>(stage + i * 512 + r0 * 2 * D, at),
                               row_in<SPLIT>(stage + (STEPS + i) * 512 + r0 * 2 * D, at), true, a.eps, cs, sn, wa, wb, c, d,
                               da, db);
        if (h0 + i * ROWS < H) store_row<SPLIT>(dx + i * ROWS * D, at, c, d);
      }
    }
    __syncwarp();
    turn ^= 1;
    now = next;
    next = later;
  }
  cp_async_wait_group<0>();
  block_weight_sum<D, SPLIT>(da, db, at, r0, a.ws + static_cast<size_t>(blockIdx.x) * D);
}

// (The same ring made it slower, 39 -> 42 us for 62598 tokens of 2 + 1 heads: every row has angles of
// its own here, and the copies of those are what it spends its time on.)
template <int D, bool SPLIT>
__global__ void __launch_bounds__(kRopeThreads, Tune<D>::FEW_BLOCKS)
    norm_rope_few_backward_kernel(const RopeArgs a, const One one) {
  constexpr int LANES = D / 8, ROWS = 32 / LANES, STEPS = kFewSteps;
  pdl_begin();
  const int l = lane_id() % LANES, r0 = lane_id() / LANES;
  const Place at = place_of<SPLIT>(a.rot, l);
  const unsigned per = static_cast<unsigned>(kRopeWarps) * one.tokens;  // tokens of a block's step
  const unsigned units = (static_cast<unsigned>(a.B) * a.N + per - 1) / per;
  uint64_t wa[2], wb[2], da[2] = {0, 0}, db[2] = {0, 0};
  load_weights<SPLIT>(one.w, at, wa, wb);
  for (unsigned n = blockIdx.x; n < units; n += gridDim.x) {
    RowAt pl[STEPS];
    Row x[STEPS], y[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      pl[i] = row_at(a, one, n * kRopeWarps + warp_id(), i * ROWS + r0);
      x[i] = y[i] = Row{{0, 0, 0, 0}};
      if (pl[i].pos >= 0) {
        x[i] = load_row<SPLIT>(one.x + pl[i].x, at);
        y[i] = load_row<SPLIT>(one.dy + pl[i].y, at);
      }
    }
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      uint64_t cs[2], sn[2], c[2], d[2];
      load_angles(a, pl[i].pos, l, cs, sn);
      row_gradient<D, SPLIT>(x[i], y[i], pl[i].pos >= 0, a.eps, cs, sn, wa, wb, c, d, da, db);
      if (pl[i].pos >= 0) store_row<SPLIT>(one.out + pl[i].x, at, c, d);
    }
  }
  block_weight_sum<D, SPLIT>(da, db, at, r0, one.partial + static_cast<size_t>(blockIdx.x) * D);
}

// dw = sum of the partial rows in a fixed order, block 0 for q, 1 for k.
template <int D>
__global__ void __launch_bounds__(1024) weight_grad_kernel(const RopeArgs a, int blocks_q,
                                                           int blocks_k) {
  constexpr int COLS = D / 4, SIDES = 1024 / COLS;
  __shared__ float4 sums[SIDES][COLS];
  pdl_begin();
  const bool is_q = blockIdx.x == 0;
  float* out = is_q ? a.dwq : a.dwk;
  if (out == nullptr) return;
  const int first = is_q ? 0 : blocks_q, n = is_q ? blocks_q : blocks_k;
  const int col = threadIdx.x % COLS, side = threadIdx.x / COLS;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float4& x) {
    s.x += x.x;
    s.y += x.y;
    s.z += x.z;
    s.w += x.w;
  };
#pragma unroll 8
  for (int i = side; i < n; i += SIDES)
    add(*reinterpret_cast<const float4*>(a.ws + static_cast<size_t>(first + i) * D + 4 * col));
  sums[side][col] = s;
  __syncthreads();
  for (int half = SIDES / 2; half > 0; half /= 2) {
    if (side < half) {
      add(sums[side + half][col]);
      sums[side][col] = s;
    }
    __syncthreads();
  }
  if (side == 0) {
    out[4 * col] = s.x;
    out[4 * col + 1] = s.y;
    out[4 * col + 2] = s.z;
    out[4 * col + 3] = s.w;
  }
}

One one_of(const RopeArgs& a, bool q, int heads) {
  One o = {};
  o.H = q ? a.Hq : a.Hkv;
  o.tokens = o.H > 0 ? heads / o.H : 0;
  o.stride = q ? a.q_stride : a.k_stride;
  o.x = q ? a.q : a.k;
  o.out = q ? a.q_out : a.k_out;
  o.dy = q ? a.dq_out : a.dk_out;
  o.w = q ? a.wq : a.wk;
  return o;
}
// Whether a tensor gets a launch of its own with several tokens per warp: at most half of
// the heads a warp takes, and enough tokens to fill the SMs several times, where the
// second launch pays (62598 tokens of 2 + 1 heads, D = 128: 61 us in one, 32 in two).
bool few_heads(int H, int heads, long long tokens, int sms) {
  return H > 0 && 2 * H <= heads && tokens >= 64LL * sms;
}

template <int D>
cudaError_t forward(const RopeArgs& a, int sms, cudaStream_t stream) {
  constexpr int heads = heads_per_warp(D, Tune<D>::STEPS);
  const long long tokens = static_cast<long long>(a.B) * a.N;
  const bool few_q = few_heads(a.Hq, heads, tokens, sms), few_k = few_heads(a.Hkv, heads, tokens, sms);
  for (int t = 0; t < 2; ++t) {
    if (!(t == 0 ? few_q : few_k)) continue;
    const One one = one_of(a, t == 0, heads);
    const long long per = static_cast<long long>(kRopeWarps) * one.tokens;
    const cudaError_t e = launch_dependent(a.interleaved ? norm_rope_few_kernel<D, false> : norm_rope_few_kernel<D, true>,
                                           static_cast<unsigned>((tokens + per - 1) / per), kRopeThreads, 0, stream, a, one);
    if (e != cudaSuccess) return e;
  }
  const int cq = few_q ? 0 : (a.Hq + heads - 1) / heads, ck = few_k ? 0 : (a.Hkv + heads - 1) / heads;
  if (cq + ck == 0) return cudaSuccess;
  const long long tiles = (tokens + kRopeWarps - 1) / kRopeWarps;
  const unsigned blocks = static_cast<unsigned>(tiles * (cq + ck));
  return launch_dependent(a.interleaved ? norm_rope_kernel<D, false> : norm_rope_kernel<D, true>, blocks,
                          kRopeThreads, 0, stream, a, cq, cq + ck);
}

template <int D, int STEPS>
cudaError_t backward_rows(const RopeArgs& a, int blocks_q, int blocks_k, cudaStream_t stream) {
  constexpr int kSmem = kRopeWarps * kGradStages * kGradStage(STEPS);
  auto kernel = a.interleaved ? norm_rope_backward_kernel<D, false, STEPS> : norm_rope_backward_kernel<D, true, STEPS>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, blocks_q + blocks_k, kRopeThreads, kSmem, stream, a, blocks_q, blocks_k);
}

template <int D>
cudaError_t backward(const RopeArgs& a, int sms, cudaStream_t stream) {
  constexpr int few = heads_per_warp(D, kFewSteps);
  const long long tokens = static_cast<long long>(a.B) * a.N, tiles = (tokens + kRopeWarps - 1) / kRopeWarps;
  const bool few_q = few_heads(a.Hq, few, tokens, sms), few_k = few_heads(a.Hkv, few, tokens, sms);
  // four rows per thread at D = 128 for given positions where that leaves few lanes without a head
  const int hq = few_q ? 0 : a.Hq, hk = few_k ? 0 : a.Hkv;
  auto chunks = [](int H, int steps) { return (H + heads_per_warp(D, steps) - 1) / heads_per_warp(D, steps); };
  const bool fill = 20LL * (chunks(hq, 4) + chunks(hk, 4)) * heads_per_warp(D, 4) <= 23LL * (hq + hk);
  const int steps = D == 128 && a.positions != nullptr && fill ? 4 : 2;
  const int cq = chunks(hq, steps), ck = chunks(hk, steps);
  // the blocks that are resident at a time, shared between q and k by their work where
  // they run together
  const int most = std::min(grad_blocks(steps) * sms, kGradBlocks / 2), most_few = std::min(Tune<D>::FEW_BLOCKS * sms, kGradBlocks / 2);
  auto few_blocks = [&](int H) {
    const long long per = static_cast<long long>(kRopeWarps) * (few / H);
    return static_cast<int>(std::min<long long>((tokens + per - 1) / per, most_few));
  };
  int limit_q = most, limit_k = most;
  if (cq > 0 && ck > 0) {
    const long long share = (static_cast<long long>(most) * cq + (cq + ck) / 2) / (cq + ck);
    limit_q = static_cast<int>(std::max<long long>(1, std::min<long long>(share, most - 1)));
    limit_k = most - limit_q;
  }
  const int bq = few_q ? few_blocks(a.Hq) : static_cast<int>(std::min<long long>(tiles * cq, limit_q));
  const int bk = few_k ? few_blocks(a.Hkv) : static_cast<int>(std::min<long long>(tiles * ck, limit_k));
  cudaError_t e = cudaSuccess;
  for (int t = 0; t < 2; ++t) {
    if (!(t == 0 ? few_q : few_k)) continue;
    One one = one_of(a, t == 0, few);
    one.partial = a.ws + static_cast<size_t>(t == 0 ? 0 : bq) * D;
    e = launch_dependent(a.interleaved ? norm_rope_few_backward_kernel<D, false> : norm_rope_few_backward_kernel<D, true>,
                         t == 0 ? bq : bk, kRopeThreads, 0, stream, a, one);
    if (e != cudaSuccess) return e;
  }
  const int rest_q = few_q ? 0 : bq, rest_k = few_k ? 0 : bk;
  if (rest_q + rest_k > 0) {
    RopeArgs c = a;
    c.ws = a.ws + static_cast<size_t>(few_q ? bq : 0) * D;  // k's rows follow q's
    if constexpr (D == 128)
      e = steps == 4 ? backward_rows<D, 4>(c, rest_q, rest_k, stream) : backward_rows<D, 2>(c, rest_q, rest_k, stream);
    else
      e = backward_rows<D, 2>(c, rest_q, rest_k, stream);
    if (e != cudaSuccess) return e;
  }
  if (a.dwq == nullptr && a.dwk == nullptr) return e;
  return launch_dependent(weight_grad_kernel<D>, a.Hkv ? 2 : 1, 1024, 0, stream, a, bq, bk);
}

}  // namespace

size_t norm_rope_backward_workspace_bytes(int D) {
  return static_cast<size_t>(kGradBlocks) * D * sizeof(float);
}

cudaError_t launch_norm_rope(const RopeArgs& a, cudaStream_t stream) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  return a.D == 128 ? forward<128>(a, sms, stream) : forward<64>(a, sms, stream);
}

cudaError_t launch_norm_rope_backward(const RopeArgs& a, cudaStream_t stream) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  return a.D == 128 ? backward<128>(a, sms, stream) : backward<64>(a, sms, stream);
}

}  // namespace mcs
