// Paged key-value cache: pages and slots of new tokens, writes into the pages
// with the pages' mean keys, and the choice of pages by a cheap score.
#include <algorithm>
#include <type_traits>

#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"

namespace mcs {
namespace {

// ------------------------------------------------------------------ plan
//
// have_b = ceil(len_b / page), need_b = ceil((len_b + new_b) / page) - have_b;
// with the exclusive sums of new and need every token and every fresh page
// finds its sequence by a binary search.  Latency and nothing else, so it is
// one launch: every CTA of one cluster takes the sums over all sequences for
// itself (B <= 4096: at most four rounds of one block scan, 32 KB from L2),
// checks everything that can be wrong, and only behind the cluster barrier,
// when all have read the state, writes its share.  The state can so be updated
// in place, and a request that cannot be met takes nothing.

constexpr int kPlanMaxThreads = 1024;
constexpr int kPlanMaxCluster = 8;
constexpr int kPlanAtOnce = 4;  // tokens a thread searches side by side

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// For each x[k] the last i in [0, n) with first[i] <= x[k] (first ascending, first[0] <= x[k]).
template <int K>
__device__ __forceinline__ void owners(const int32_t* first, int n, const int (&x)[K], int (&at)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) at[k] = 0;
  for (int d = n > 1 ? 1 << (31 - __clz(n - 1)) : 0; d > 0; d >>= 1) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (at[k] + d < n && first[at[k] + d] <= x[k]) at[k] += d;
  }
}

__global__ void __launch_bounds__(kPlanMaxThreads) paged_plan_kernel(const PlanArgs a, int ctas) {
  extern __shared__ int32_t sm[];
  int32_t* s_cu = sm;                 // [B + 1] exclusive sums of new tokens
  int32_t* s_base = s_cu + a.B + 1;   // [B + 1] exclusive sums of missing pages
  int32_t* s_len = s_base + a.B + 1;  // [B]
  __shared__ long long sums[32][2];
  const int tid = threadIdx.x, lane = lane_id(), w = warp_id();
  const int threads = blockDim.x, warps = threads / 32;
  const int shift = 31 - __clz(a.page), mask = a.page - 1;
  const long long room = static_cast<long long>(a.max_pages) << shift;
  const int head = a.free_head[0];
  long long tokens = 0, pages = 0;
  bool bad = false;
  for (int b0 = 0; b0 < a.B; b0 += threads) {
    const int b = b0 + tid;
    long long nw = 0, need = 0;
    if (b < a.B) {
      const int len = a.lens[b];
      nw = a.new_lens[b];
      if (len < 0 || nw < 0 || len + nw > room) {
        bad = true;
        nw = 0;
      } else {
        need = ((len + nw + mask) >> shift) - ((static_cast<long long>(len) + mask) >> shift);
        if (nw > 0 && (len & mask) != 0) {  // continues in its last page
          const int pid = a.table[static_cast<size_t>(b) * a.max_pages + (len >> shift)];
          bad = bad || pid < 0 || pid >= a.num_pages;
        }
      }
      s_len[b] = len;
    }
    long long x = nw, y = need;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, x, d), v = __shfl_up_sync(0xffffffffu, y, d);
      if (lane >= d) x += u, y += v;
    }
    if (lane == 31) sums[w][0] = x, sums[w][1] = y;
    __syncthreads();
    long long all_x = 0, all_y = 0;
    for (int i = 0; i < warps; ++i) {
      if (i < w) x += sums[i][0], y += sums[i][1];
      all_x += sums[i][0];
      all_y += sums[i][1];
    }
    if (b < a.B) {
      // sums beyond T or n_free are refused below, before they are used
      s_cu[b] = static_cast<int32_t>(tokens + x - nw);
      s_base[b] = static_cast<int32_t>(pages + y - need);
    }
    tokens += all_x;
    pages += all_y;
    __syncthreads();
  }
  bad = bad || tokens > a.T || head < 0 || head > a.n_free || pages > a.n_free - head;
  if (!bad) {
    for (int j = tid; j < pages; j += threads) {
      const int pid = a.free_pages[head + j];
      bad = bad || pid < 0 || pid >= a.num_pages;
    }
  }
  if (tid == 0) {
    s_cu[a.B] = static_cast<int32_t>(tokens);
    s_base[a.B] = static_cast<int32_t>(pages);
  }
  bad = __syncthreads_or(bad);
  // every CTA has read what any CTA is about to write
  if (ctas > 1) cluster_sync();

  const int at = blockIdx.x * threads + tid, step = ctas * threads;
  if (bad) {
    if (at == 0) {
      atomicOr(a.status, DEV_BOUNDS);
      a.head_out[0] = head;
    }
    for (int b = at; b <= a.B; b += step) {
      if (b < a.B) a.lens_out[b] = s_len[b];
      a.cu_new[b] = 0;
    }
    for (int t = at; t < a.T; t += step) {
      a.slots[t] = -1;
      if (a.positions) a.positions[t] = -1;
    }
    return;
  }
  if (at == 0) a.head_out[0] = head + static_cast<int>(pages);
  for (int b = at; b <= a.B; b += step) {
    a.cu_new[b] = s_cu[b];
    if (b < a.B) a.lens_out[b] = s_len[b] + (s_cu[b + 1] - s_cu[b]);
  }
  for (int j = at; j < pages; j += step) {
    const int x[1] = {j};
    int b[1];
    owners(s_base, a.B, x, b);
    const int have = (s_len[b[0]] + mask) >> shift;
    a.table[static_cast<size_t>(b[0]) * a.max_pages + have + (j - s_base[b[0]])] = a.free_pages[head + j];
  }
  for (long long t0 = at; t0 < a.T; t0 += static_cast<long long>(kPlanAtOnce) * step) {
    int t[kPlanAtOnce], b[kPlanAtOnce], pid[kPlanAtOnce], pos[kPlanAtOnce];
#pragma unroll
    for (int k = 0; k < kPlanAtOnce; ++k)
      t[k] = static_cast<int>(min(t0 + static_cast<long long>(k) * step, static_cast<long long>(a.T)));
    owners(s_cu, a.B, t, b);
#pragma unroll
    for (int k = 0; k < kPlanAtOnce; ++k) {
      pos[k] = pid[k] = -1;
      if (t[k] >= tokens) continue;
      pos[k] = s_len[b[k]] + (t[k] - s_cu[b[k]]);
      // pages the sequence had (its last one, read above), or fresh ones
      const int have = (s_len[b[k]] + mask) >> shift, j = pos[k] >> shift;
      pid[k] = j < have ? a.table[static_cast<size_t>(b[k]) * a.max_pages + j]
                        : a.free_pages[head + s_base[b[k]] + (j - have)];
    }
#pragma unroll
    for (int k = 0; k < kPlanAtOnce; ++k) {
      if (t[k] >= a.T) continue;
      a.slots[t[k]] = pos[k] < 0 ? -1 : (pid[k] << shift) + (pos[k] & mask);
      if (a.positions) a.positions[t[k]] = pos[k];
    }
  }
}

// ------------------------------------------------------------------ write

// x / scale, correctly rounded, from inv = 1 / scale (itself correctly rounded): the
// product and one exact remainder (Markstein 1990).  For every mantissa of a
// bf16 x and of the scale this is the fp32 quotient (all 2^30 pairs compared);
// scales outside [2^-60, 2^60], where remainders could underflow, divide instead.
// Infinities (and what overflows) and the sign of zero are put back.
struct Scale {
  float s, inv;
  bool fast;
};
__device__ __forceinline__ uint64_t quotient2(uint32_t lo, uint32_t hi, const Scale& c) {
  const float x0 = __uint_as_float(lo), x1 = __uint_as_float(hi);
  if (!c.fast) return f2_pack(__fdiv_rn(x0, c.s), __fdiv_rn(x1, c.s));
  const uint64_t x = f2_pack(x0, x1), inv = f2_pack(c.inv, c.inv);
  const uint64_t q = f2_fma(x, inv, 0x8000000080000000ull);
  const uint64_t rem = f2_fma(q ^ 0x8000000080000000ull, f2_pack(c.s, c.s), x);
  float q0, q1, r0, r1;
  f2_unpack(q, q0, q1);
  f2_unpack(f2_fma(rem, inv, q), r0, r1);
  r0 = fabsf(q0) <= 1e30f ? copysignf(r0, x0) : q0;
  r1 = fabsf(q1) <= 1e30f ? copysignf(r1, x1) : q1;
  return f2_pack(r0, r1);
}

// 8 bf16 values (a 16-byte word) -> 8 E4M3 codes of x / scale.
__device__ __forceinline__ uint2 encode8(uint4 x, const Scale& scale) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f2_unpack(quotient2(w[i] << 16, w[i] & 0xFFFF0000u, scale), lo, hi);
    c[i] = f32x2_to_e4m3x2(lo, hi);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// sum += the stored values: 8 bf16, or scale * 8 E4M3 codes.
__device__ __forceinline__ void add8(float* sum, uint4 x, float) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sum[2 * i] += __uint_as_float(w[i] << 16);
    sum[2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void add8(float* sum, uint2 c, float scale) {
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t lo, hi;
    e4m3x4_to_f16x4(w[i], lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<__half2*>(&hi));
    sum[4 * i] += a.x * scale;
    sum[4 * i + 1] += a.y * scale;
    sum[4 * i + 2] += b.x * scale;
    sum[4 * i + 3] += b.y * scale;
  }
}

constexpr int kWriteThreads = 256;

// D/8 threads per (token, head) copy its k and v rows.  The threads of the
// first token of each page's run also take the page's mean: the rows in front
// of it from the cache, the run's own from k (now in L2), so that nothing is
// read that another thread of this launch writes; eight rows at a time, since
// one thread's loads are all that hides their latency.
template <int D, bool kE4M3Cache>
__global__ void __launch_bounds__(kWriteThreads) paged_write_kernel(const WriteArgs a, bool fast) {
  constexpr int LANES = D / 8;
  const unsigned item = blockIdx.x * (kWriteThreads / LANES) + threadIdx.x / LANES;
  const int l = threadIdx.x % LANES;
  const unsigned t = item / static_cast<unsigned>(a.Hkv), h = item - t * a.Hkv;
  if (t >= static_cast<unsigned>(a.T)) return;
  const int slot = a.slots[t];
  if (slot < 0) return;
  if (slot >= a.slots_total) {
    if (h == 0 && l == 0) atomicOr(a.status, DEV_BOUNDS);
    return;
  }
  const Scale ks = {a.k_scale, a.k_inv, fast}, vs = {a.v_scale, a.v_inv, fast};
  const int off = slot & (a.page - 1), page_id = slot >> (31 - __clz(a.page));
  const size_t page_row = (static_cast<size_t>(page_id) * a.Hkv + h) * a.page;
  const size_t src = t * a.stride + static_cast<size_t>(h) * D + 8 * l;
  const size_t dst = (page_row + off) * D + 8 * l;
  const uint4 k = ld_global_nc16(a.k + src), v = ld_global_nc16(a.v + src);
  const bool mean = a.k_mean != nullptr && (t == 0 || off == 0 || a.slots[t - 1] != slot - 1);
  if (kE4M3Cache) {
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.k_cache) + dst) = encode8(k, ks);
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.v_cache) + dst) = encode8(v, vs);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.k_cache) + dst) = k;
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.v_cache) + dst) = v;
  }
  if (!mean) return;
  // the run: how many tokens behind t continue in the page, LANES of them looked at a time
  const int lane0 = lane_id() / LANES * LANES;
  const uint32_t mates = ((1u << LANES) - 1u) << lane0;
  int run = 1;
  for (const int most = min(a.page - off, a.T - static_cast<int>(t)); run < most;) {
    const bool next = run + l < most && a.slots[t + run + l] == slot + run + l;
    const uint32_t no = ~__ballot_sync(mates, next) & mates;
    const int more = no == 0 ? LANES : __ffs(no) - 1 - lane0;
    run += more;
    if (more < LANES) break;
  }
  float sum[8] = {};
  using Word = typename std::conditional<kE4M3Cache, uint2, uint4>::type;  // 8 stored values
  const Word* old = reinterpret_cast<const Word*>(
      static_cast<const uint8_t*>(a.k_cache) + (page_row * D + 8 * l) * (kE4M3Cache ? 1 : 2));
  for (int r = 0; r < off; r += 8) {
    Word x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = Word{};
      if (r + i < off) x[i] = old[(r + i) * LANES];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) add8(sum, x[i], a.k_scale);
  }
  for (int r = 0; r < run; r += 8) {
    uint4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = make_uint4(0, 0, 0, 0);
      if (r + i < run) x[i] = ld_global_nc16(a.k + src + static_cast<size_t>(r + i) * a.stride);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (r + i >= run) break;
      if (kE4M3Cache) add8(sum, encode8(x[i], ks), a.k_scale);
      else add8(sum, x[i], 1.f);
    }
  }
  const float n = static_cast<float>(off + run);
  uint4 m;
  m.x = pack_bf16(sum[0] / n, sum[1] / n);
  m.y = pack_bf16(sum[2] / n, sum[3] / n);
  m.z = pack_bf16(sum[4] / n, sum[5] / n);
  m.w = pack_bf16(sum[6] / n, sum[7] / n);
  *reinterpret_cast<uint4*>(a.k_mean + (static_cast<size_t>(page_id) * a.Hkv + h) * D + 8 * l) = m;
}

// ------------------------------------------------------------------ select
//
// score(page) = (sum of the group's queries) . mean, and the pages of the
// largest scores.  Which page is kept must not depend on the order of a sum,
// so the products are summed in two fp32 words per sum (error-free sums and
// products of pairs: about 48 bits) and rounded to fp32 once; ties then go to
// the lower page.  fp64 would give the same but runs at 1/60 of the fp32 rate here.
// Bound: the means are read once, 2 D bytes per page and KV head.

constexpr int kScoreThreads = 256;
constexpr int kTopkKeys = 8;  // consecutive keys per thread and step

// Two independent sums (x and y halves of the pairs), each as hi + lo.
struct Sum2 {
  uint64_t hi, lo;
};
__device__ __forceinline__ uint64_t f2_sub(uint64_t a, uint64_t b) {
  return f2_fma(b, f2_pack(-1.f, -1.f), a);
}
// s + x: hi takes the rounded sum, lo what it lost (Knuth's two-sum).
__device__ __forceinline__ void two_add(Sum2& s, uint64_t x) {
  const uint64_t sum = f2_add(s.hi, x), bb = f2_sub(sum, s.hi);
  const uint64_t err = f2_add(f2_sub(s.hi, f2_sub(sum, bb)), f2_sub(x, bb));
  s.hi = sum;
  s.lo = f2_add(s.lo, err);
}
__device__ __forceinline__ void two_add(float& hi, float& lo, float x, float xl) {
  const float sum = __fadd_rn(hi, x), bb = __fsub_rn(sum, hi);
  const float err = __fadd_rn(__fsub_rn(hi, __fsub_rn(sum, bb)), __fsub_rn(x, bb));
  hi = sum;
  lo = __fadd_rn(__fadd_rn(lo, xl), err);
}

// A block takes ROWS = 256 / D KV heads of one sequence and 8 * per_warp of its
// pages.  D/8 lanes hold a head, 8 values each; a warp sums four pages at a
// time and folds them over the lanes, so that each fold halves what is left.
template <int D>
__global__ void __launch_bounds__(kScoreThreads)
    paged_score_kernel(const SelectArgs a, int head_blocks, int page_blocks, int per_warp, int stride) {
  constexpr int LANES = D / 8, ROWS = 32 / LANES;
  __shared__ float s_hi[ROWS * D], s_lo[ROWS * D];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int xp = blockIdx.x % page_blocks, hb = blockIdx.x / page_blocks % head_blocks;
  const int b = blockIdx.x / page_blocks / head_blocks;
  const int len = a.lens[b];
  if (len <= 0 || static_cast<long long>(len) > static_cast<long long>(a.max_pages) * a.page) return;
  const int n = (len - 1) / a.page + 1;
  const int j0 = (xp * (kScoreThreads / 32) + warp_id()) * per_warp;
  if (xp * (kScoreThreads / 32) * per_warp >= n) return;
  const int group = a.Hq / a.Hkv;
  {  // the group's summed query, one value per thread
    const int r = threadIdx.x / D, d = threadIdx.x % D, h = min(hb * ROWS + r, a.Hkv - 1);
    const __nv_bfloat16* q = a.q + b * a.q_stride + static_cast<size_t>(h) * group * D + d;
    float hi = 0.f, lo = 0.f;
    for (int i = 0; i < group; ++i) two_add(hi, lo, __bfloat162float(q[i * D]), 0.f);
    const float sum = __fadd_rn(hi, lo);
    s_hi[threadIdx.x] = sum;
    s_lo[threadIdx.x] = __fsub_rn(lo, __fsub_rn(sum, hi));
  }
  __syncthreads();
  const int lane = lane_id(), l = lane % LANES, h = hb * ROWS + lane / LANES;
  uint64_t qh[4], ql[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = lane / LANES * D + 8 * l + 2 * i;
    qh[i] = f2_pack(s_hi[at], s_hi[at + 1]);
    ql[i] = f2_pack(s_lo[at], s_lo[at + 1]);
  }
  const __nv_bfloat16* mean = a.k_mean + static_cast<size_t>(min(h, a.Hkv - 1)) * D + 8 * l;
  const size_t page_step = static_cast<size_t>(a.Hkv) * D;
  uint32_t* keys = a.keys + (static_cast<size_t>(b) * a.Hkv + h) * stride;
  const int j1 = min(n, j0 + per_warp);
  if (j0 >= j1) return;
  // per_warp <= 32: a page number per lane
  int pid = 0;
  bool outside = false;
  if (j0 + lane < j1) {
    pid = a.table[static_cast<size_t>(b) * a.max_pages + j0 + lane];
    outside = pid < 0 || pid >= a.num_pages;
    if (outside) {
      atomicOr(a.status, DEV_BOUNDS);
      pid = 0;
    }
  }
  const uint32_t bad = __ballot_sync(0xffffffffu, outside);
  for (int j = j0; j < j1; j += 8) {
    uint4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = ld_global_nc16(mean + __shfl_sync(0xffffffffu, pid, j - j0 + i) * page_step);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w[4] = {x[4 * half + i].x, x[4 * half + i].y, x[4 * half + i].z,
                               x[4 * half + i].w};
        Sum2 s = {0, 0};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint64_t m = f2_pack(__uint_as_float(w[c] << 16), __uint_as_float(w[c] & 0xFFFF0000u));
          const uint64_t p = f2_fma(qh[c], m, 0);
          // what the product lost, and the low word's product
          const uint64_t e = f2_fma(qh[c], m, p ^ 0x8000000080000000ull);
          two_add(s, p);
          s.lo = f2_add(s.lo, f2_fma(ql[c], m, e));
        }
        float h0, h1, l0, l1;
        f2_unpack(s.hi, h0, h1);
        f2_unpack(s.lo, l0, l1);
        two_add(h0, l0, h1, l1);
        hi[i] = h0;
        lo[i] = l0;
      }
      // fold over the lanes: the upper half of each group of lanes keeps the
      // upper half of the pages
      int o = LANES / 2;
#pragma unroll
      for (int keep = 2; keep >= 1; keep /= 2, o /= 2) {
        const bool upper = l & o;
#pragma unroll
        for (int i = 0; i < keep; ++i) {
          const float sh = upper ? hi[i] : hi[i + keep], sl = upper ? lo[i] : lo[i + keep];
          hi[i] = upper ? hi[i + keep] : hi[i];
          lo[i] = upper ? lo[i + keep] : lo[i];
          const float rh = __shfl_xor_sync(0xffffffffu, sh, o), rl = __shfl_xor_sync(0xffffffffu, sl, o);
          two_add(hi[i], lo[i], rh, rl);
        }
      }
#pragma unroll
      for (; o > 0; o /= 2) {
        const float rh = __shfl_xor_sync(0xffffffffu, hi[0], o), rl = __shfl_xor_sync(0xffffffffu, lo[0], o);
        two_add(hi[0], lo[0], rh, rl);
      }
      // lane bits LANES/2 and LANES/4 name the page
      const int mine = 4 * half + ((l & (LANES / 2)) ? 2 : 0) + ((l & (LANES / 4)) ? 1 : 0);
      const int page = j + mine;
      const int from = __shfl_sync(0xffffffffu, pid, page - j0);
      if (l % (LANES / 4) == 0 && page < j1 && h < a.Hkv) {
        float score = __fadd_rn(hi[0], lo[0]);
        if (!(fabsf(score) <= 3.0e38f)) {
          // infinities or an overflow in between, where the two-word sum does
          // not hold: in fp64
          double sum = 0;
          for (int d = 0; d < D; ++d) {
            const int at = lane / LANES * D + d;
            sum += (static_cast<double>(s_hi[at]) + static_cast<double>(s_lo[at])) *
                   static_cast<double>(__bfloat162float(a.k_mean[from * page_step + static_cast<size_t>(h) * D + d]));
          }
          score = static_cast<float>(sum);
        }
        uint32_t key = score_key_bits(__float_as_uint(score));
        if (page < a.sink || page >= n - a.recent) key = 0xFFFFFFFFu;
        if ((bad >> (page - j0)) & 1u) key = 0;  // last of all; the attention skips it too
        keys[page] = key;
      }
    }
  }
}

// One block per (sequence, KV head).  The select-th largest key by four 8-bit
// digits, counted in a histogram per warp (scores share their leading bits, and
// one histogram for all would queue every warp at a few counters); then the
// kept pages in order, each thread with 8 consecutive ones.
__global__ void __launch_bounds__(1024) paged_topk_kernel(const SelectArgs a, int stride) {
  extern __shared__ uint32_t hist[];  // [warps][256]
  __shared__ uint32_t s_prefix, s_left;
  __shared__ int s_warp[32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int bh = blockIdx.x, b = bh / a.Hkv, tid = threadIdx.x, w = warp_id(), lane = lane_id();
  const int warps = blockDim.x / 32, step = blockDim.x * kTopkKeys;
  const int len = a.lens[b];
  const bool bad = len < 0 || static_cast<long long>(len) > static_cast<long long>(a.max_pages) * a.page;
  if (bad && tid == 0) atomicOr(a.status, DEV_BOUNDS);
  const int n = bad || len == 0 ? 0 : (len - 1) / a.page + 1;
  const int keep = min(n, a.select);
  const uint32_t* keys = a.keys + static_cast<size_t>(bh) * stride;
  int32_t* sel = a.sel + static_cast<size_t>(bh) * a.select;
  for (int i = keep + tid; i < a.select; i += blockDim.x) sel[i] = -1;
  if (n <= keep) {
    for (int i = tid; i < n; i += blockDim.x) sel[i] = i;
    return;
  }
  uint32_t prefix = 0, left = keep;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < warps * 256; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    for (int j = tid * kTopkKeys; j < n; j += step) {
      uint32_t x[kTopkKeys];
      *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(keys + j);
      *reinterpret_cast<uint4*>(x + 4) = *reinterpret_cast<const uint4*>(keys + j + 4);
#pragma unroll
      for (int i = 0; i < kTopkKeys; ++i)
        if (j + i < n && (shift == 24 || (x[i] >> (shift + 8)) == prefix))
          atomicAdd(&hist[w * 256 + ((x[i] >> shift) & 255u)], 1u);
    }
    __syncthreads();
    for (int d = tid; d < 256; d += blockDim.x) {
      uint32_t c = 0;
      for (int i = 0; i < warps; ++i) c += hist[i * 256 + d];
      hist[d] = c;  // row 0; each column is one thread's
    }
    __syncthreads();
    if (w == 0) {  // lane i: digits 255 - 8 i down to 248 - 8 i
      uint32_t c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += c[i] = hist[255 - 8 * lane - i];
      uint32_t upto = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += y;
      }
      uint32_t above = upto - sum;
      if (above < left && left <= upto) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (above < left && left <= above + c[i]) {
            s_prefix = (prefix << 8) | (255 - 8 * lane - i);
            s_left = left - above;
          }
          above += c[i];
        }
      }
    }
    __syncthreads();
    prefix = s_prefix;
    left = s_left;
  }
  // keys above `prefix` are kept, and the first `left` that equal it
  int more0 = 0, same0 = 0;
  for (int base = 0; base < n; base += step) {
    const int j = base + tid * kTopkKeys;
    uint32_t x[kTopkKeys] = {};
    if (j < n) {
      *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(keys + j);
      *reinterpret_cast<uint4*>(x + 4) = *reinterpret_cast<const uint4*>(keys + j + 4);
    }
    int own = 0;  // kept above in the low half, equal in the high half
#pragma unroll
    for (int i = 0; i < kTopkKeys; ++i)
      if (j + i < n) own += x[i] > prefix ? 1 : (x[i] == prefix ? 0x10000 : 0);
    int upto = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[w] = upto;
    __syncthreads();
    int before = upto - own, all = 0;
    for (int i = 0; i < warps; ++i) {
      const int y = s_warp[i];
      if (i < w) before += y;
      all += y;
    }
    int more = more0 + (before & 0xFFFF), same = same0 + (before >> 16);
#pragma unroll
    for (int i = 0; i < kTopkKeys; ++i) {
      if (j + i >= n) break;
      if (x[i] > prefix) {
        sel[more + min(same, static_cast<int>(left))] = j + i;
        ++more;
      } else if (x[i] == prefix) {
        if (same < static_cast<int>(left)) sel[more + same] = j + i;
        ++same;
      }
    }
    more0 += all & 0xFFFF;
    same0 += all >> 16;
  }
}

}  // namespace

cudaError_t launch_paged_plan(const PlanArgs& a, cudaStream_t stream) {
  const size_t smem = (3 * static_cast<size_t>(a.B) + 2) * sizeof(int32_t);
  // a thread per item up to one CTA of 1024, then a CTA per 4096 up to one cluster
  const long long items = std::max<long long>(a.T, a.B);
  const int threads = items > 512 ? kPlanMaxThreads : items > 256 ? 512 : 256;
  int ctas = 1;
  while (ctas < kPlanMaxCluster && items > 4096LL * ctas) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&cfg, paged_plan_kernel, a, ctas);
}

cudaError_t launch_paged_write(const WriteArgs& a, bool e4m3, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  const long long items = static_cast<long long>(a.T) * a.Hkv;
  const int per_block = kWriteThreads / (a.D / 8);
  const unsigned blocks = static_cast<unsigned>((items + per_block - 1) / per_block);
  WriteArgs c = a;
  c.k_inv = e4m3 ? 1.f / a.k_scale : 1.f;
  c.v_inv = e4m3 ? 1.f / a.v_scale : 1.f;
  auto middle = [](float s) { return s >= 0x1p-60f && s <= 0x1p60f; };
  const bool fast = middle(a.k_scale) && middle(a.v_scale);
  if (a.D == 128) {
    if (e4m3) paged_write_kernel<128, true><<<blocks, kWriteThreads, 0, stream>>>(c, fast);
    else paged_write_kernel<128, false><<<blocks, kWriteThreads, 0, stream>>>(c, fast);
  } else {
    if (e4m3) paged_write_kernel<64, true><<<blocks, kWriteThreads, 0, stream>>>(c, fast);
    else paged_write_kernel<64, false><<<blocks, kWriteThreads, 0, stream>>>(c, fast);
  }
  return cudaGetLastError();
}

// Keys of a row: whole 16-byte words for every thread's eight.
static int key_stride(int max_pages) { return (max_pages + kTopkKeys - 1) / kTopkKeys * kTopkKeys; }

size_t paged_select_workspace_bytes(int B, int Hkv, int max_pages) {
  return static_cast<size_t>(B) * Hkv * key_stride(max_pages) * sizeof(uint32_t);
}

cudaError_t launch_paged_select(const SelectArgs& a, cudaStream_t stream) {
  const int rows = 256 / a.D, head_blocks = (a.Hkv + rows - 1) / rows;
  const int stride = key_stride(a.max_pages);
  // 32 pages per warp; fewer where that would leave SMs idle
  int per_warp = 32;
  while (per_warp > 8 && static_cast<long long>(a.B) * head_blocks *
                                 ((a.max_pages + 8 * per_warp - 1) / (8 * per_warp)) < 304)
    per_warp /= 2;
  const int page_blocks = (a.max_pages + 8 * per_warp - 1) / (8 * per_warp);
  const unsigned blocks = static_cast<unsigned>(static_cast<long long>(a.B) * head_blocks * page_blocks);
  if (a.D == 128)
    paged_score_kernel<128><<<blocks, kScoreThreads, 0, stream>>>(a, head_blocks, page_blocks, per_warp, stride);
  else
    paged_score_kernel<64><<<blocks, kScoreThreads, 0, stream>>>(a, head_blocks, page_blocks, per_warp, stride);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int threads = a.max_pages > 4096 ? 1024 : (a.max_pages > 1024 ? 512 : 128);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.B * a.Hkv);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = threads / 32 * 256 * sizeof(uint32_t);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_topk_kernel, a, stride);
}

}  // namespace mcs
