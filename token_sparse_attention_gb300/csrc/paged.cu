// Paged key-value cache: pages and slots of new tokens, writes into the pages
// with the pages' mean keys, and the choice of pages by a cheap score.
#include <string.h>

#include <algorithm>
#include <type_traits>

#include <cuda_fp16.h>

#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace mcs {
namespace {

// ------------------------------------------------------------------ plan
//
// have_b = ceil(len_b / page), need_b = ceil((len_b + new_b) / page) - have_b;
// with the exclusive sums of new and need every token and every fresh page
// finds its sequence by a binary search.  Latency and nothing else: one CTA
// takes the sums and checks everything that can be wrong before it writes
// anything, so the state can be updated in place and a request that cannot be
// met takes nothing.  The tokens of a small step it places itself; for many, a
// second launch (programmatically dependent) places them over all SMs from what
// the first one wrote: cu_new, lens_out and the table say everything.
// 9 sequences, 108 000 tokens: 12.3 us with all in one cluster of 8 CTAs (bound by
// their instruction issue), 6.2 us in two launches; 256 single tokens 3.9 us.

constexpr int kPlanMaxThreads = 1024;
constexpr int kPlanSums = 33;
constexpr int kPlanAtOnce = 4;      // tokens a thread searches side by side
constexpr int kPlanTokens = 8192;   // as many tokens the first launch places itself

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

// Slots and positions of the tokens at, at + step, ...: cu (shared), the
// lengths before the step and the complete table.
template <typename Len>
__device__ __forceinline__ void place_tokens(const PlanArgs& a, const int32_t* cu, Len old, int at,
                                             int step) {
  const int shift = 31 - __clz(a.page), mask = a.page - 1, tokens = cu[a.B];
  for (long long t0 = at; t0 < a.T; t0 += static_cast<long long>(kPlanAtOnce) * step) {
    int t[kPlanAtOnce], b[kPlanAtOnce], pid[kPlanAtOnce], pos[kPlanAtOnce];
#pragma unroll
    for (int k = 0; k < kPlanAtOnce; ++k)
      t[k] = static_cast<int>(min(t0 + static_cast<long long>(k) * step, static_cast<long long>(a.T)));
    owners(cu, a.B, t, b);
#pragma unroll
    for (int k = 0; k < kPlanAtOnce; ++k) {
      pos[k] = pid[k] = -1;
      if (t[k] >= tokens) continue;
      pos[k] = old(b[k]) + (t[k] - cu[b[k]]);
      pid[k] = a.table[static_cast<size_t>(b[k]) * a.max_pages + (pos[k] >> shift)];
    }
#pragma unroll
    for (int k = 0; k < kPlanAtOnce; ++k) {
      if (t[k] >= a.T) continue;
      a.slots[t[k]] = pos[k] < 0 ? -1 : (pid[k] << shift) + (pos[k] & mask);
      if (a.positions) a.positions[t[k]] = pos[k];
    }
  }
}

__global__ void __launch_bounds__(kPlanMaxThreads) paged_plan_kernel(const PlanArgs a, bool place) {
  extern __shared__ int32_t sm[];
  int32_t* s_cu = sm;                 // [B + 1] exclusive sums of new tokens
  int32_t* s_base = s_cu + a.B + 1;   // [B + 1] exclusive sums of missing pages
  int32_t* s_len = s_base + a.B + 1;  // [B]
  __shared__ long long sums[kPlanSums][2];  // of the warps in front of each; in the last the block's
  pdl_begin();
  const int tid = threadIdx.x, lane = lane_id(), w = warp_id(), threads = blockDim.x;
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
    auto scan = [&](long long& x, long long& y) {
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, x, d), v = __shfl_up_sync(0xffffffffu, y, d);
        if (lane >= d) x += u, y += v;
      }
    };
    long long x = nw, y = need;
    scan(x, y);
    if (lane == 31) sums[w][0] = x, sums[w][1] = y;
    __syncthreads();
    if (w == 0) {
      const bool in = lane < threads / 32;
      const long long p = in ? sums[lane][0] : 0, q = in ? sums[lane][1] : 0;
      long long u = p, v = q;
      scan(u, v);
      sums[lane][0] = u - p;
      sums[lane][1] = v - q;
      if (lane == 31) sums[32][0] = u, sums[32][1] = v;
    }
    __syncthreads();
    if (b < a.B) {
      // sums beyond T or n_free are refused below, before they are used
      s_cu[b] = static_cast<int32_t>(tokens + sums[w][0] + x - nw);
      s_base[b] = static_cast<int32_t>(pages + sums[w][1] + y - need);
    }
    tokens += sums[32][0];
    pages += sums[32][1];
    __syncthreads();
  }
  bad = bad || tokens > a.T || head < 0 || head > a.n_free || pages > a.n_free - head;
  if (!bad) {
    for (int j = tid; j < pages; j += threads) {
      const int pid = a.free_pages[head + j];
      bad = bad || pid < 0 || pid >= a.num_pages;
    }
  }
  bad = __syncthreads_or(bad);  // from here on everything has been read that is written below
  if (bad) {
    if (tid == 0) {
      atomicOr(a.status, DEV_BOUNDS);
      a.head_out[0] = head;
    }
    for (int b = tid; b <= a.B; b += threads) {
      if (b < a.B) a.lens_out[b] = s_len[b];
      a.cu_new[b] = 0;
      s_cu[b] = 0;
    }
  } else {
    if (tid == 0) {
      a.head_out[0] = head + static_cast<int>(pages);
      a.cu_new[a.B] = s_cu[a.B] = static_cast<int32_t>(tokens);
      s_base[a.B] = static_cast<int32_t>(pages);
    }
    __syncthreads();
    for (int b = tid; b < a.B; b += threads) {
      a.cu_new[b] = s_cu[b];
      a.lens_out[b] = s_len[b] + (s_cu[b + 1] - s_cu[b]);
    }
    for (int j = tid; j < pages; j += threads) {
      const int x[1] = {j};
      int b[1];
      owners(s_base, a.B, x, b);
      const int have = (s_len[b[0]] + mask) >> shift;
      a.table[static_cast<size_t>(b[0]) * a.max_pages + have + (j - s_base[b[0]])] = a.free_pages[head + j];
    }
  }
  if (!place) return;
  __syncthreads();  // the table's new entries, too
  place_tokens(a, s_cu, [&](int b) { return s_len[b]; }, tid, threads);
}

__global__ void __launch_bounds__(256) paged_place_kernel(const PlanArgs a) {
  extern __shared__ int32_t s_cu[];  // [B + 1]
  pdl_begin();
  for (int b = threadIdx.x; b <= a.B; b += blockDim.x) s_cu[b] = a.cu_new[b];
  __syncthreads();
  place_tokens(a, s_cu, [&](int b) { return a.lens_out[b] - (s_cu[b + 1] - s_cu[b]); },
               blockIdx.x * 256 + threadIdx.x, gridDim.x * 256);
}

// ------------------------------------------------------------------ write

// x / scale, correctly rounded, from inv = 1 / scale (itself correctly rounded): the
// product and one exact remainder (Markstein 1990).  For every mantissa of a
// bf16 x and of the scale this is the fp32 quotient (all 2^30 pairs compared).
// |x| is first limited to `most`, at least 1024 scale, which changes no code and
// keeps infinities out of the remainder; NaN stays, and so does the sign of zero.
// What is limited comes out negated (`most` is negative), as the remainder wants it.
// Scales outside [2^-60, 2^60], where remainders could underflow, divide instead.
struct Scale {
  float s, inv;
  uint32_t most;  // bf16 twice; 0: divide
};
__device__ __forceinline__ uint64_t quotient2(uint32_t w, const Scale& c) {
  if (c.most == 0)
    return f2_pack(__fdiv_rn(__uint_as_float(w << 16), c.s), __fdiv_rn(__uint_as_float(w & 0xFFFF0000u), c.s));
  uint32_t y;
  asm("min.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(w), "r"(c.most));
  const uint64_t x = f2_pack(__uint_as_float(y << 16), __uint_as_float(y & 0xFFFF0000u));  // minus the values
  const uint64_t q = f2_fma(x, f2_pack(-c.inv, -c.inv), 0x8000000080000000ull);
  const uint64_t rem = f2_fma(q, f2_pack(c.s, c.s), x);
  return f2_fma(rem, f2_pack(-c.inv, -c.inv), q);
}

// 8 bf16 values (a 16-byte word) -> 8 E4M3 codes of x / scale.
__device__ __forceinline__ uint2 encode8(uint4 x, const Scale& scale) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f2_unpack(quotient2(w[i], scale), lo, hi);
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

// Stores one row's 8 values of k and v at `dst` (elements) of the caches; what k's stand for
// afterwards is added to sum.
template <bool kE4M3Cache, bool kSum>
__device__ __forceinline__ void store8(const WriteArgs& a, const Scale& ks, const Scale& vs, size_t dst, uint4 k,
                                       uint4 v, float* sum) {
  if (kE4M3Cache) {
    const uint2 c = encode8(k, ks);
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.k_cache) + dst) = c;
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.v_cache) + dst) = encode8(v, vs);
    if (kSum) add8(sum, c, a.k_scale);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.k_cache) + dst) = k;
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.v_cache) + dst) = v;
    if (kSum) add8(sum, k, 1.f);
  }
}

// Without means.  A block takes one KV head and a window of consecutive tokens, D/8
// threads per row and ROWS rows per thread, all loaded before the first slot is needed.
// Bound: HBM (28 005 tokens of 8 heads, bf16 40 us, 94 % of a copy; E4M3 31 us, 92 %), latency for a
// step (128 tokens 1.9 us).
template <int D, bool kE4M3Cache, int ROWS>
__global__ void __launch_bounds__(kWriteThreads) paged_copy_kernel(const WriteArgs a) {
  constexpr int LANES = D / 8, GROUPS = kWriteThreads / LANES, WINDOW = GROUPS * ROWS;
  pdl_begin();
  const unsigned window = blockIdx.x / static_cast<unsigned>(a.Hkv);
  const int h = static_cast<int>(blockIdx.x - window * a.Hkv), g = threadIdx.x / LANES, l = threadIdx.x % LANES;
  const long long t0 = static_cast<long long>(window) * WINDOW + g;
  const size_t col = static_cast<size_t>(h) * D + 8 * l;
  const int shift = 31 - __clz(a.page), mask = a.page - 1;
  const Scale ks = {a.k_scale, a.k_inv, a.k_most}, vs = {a.v_scale, a.v_inv, a.v_most};
  uint4 k[ROWS], v[ROWS];
  int slot[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const long long t = t0 + i * GROUPS;
    slot[i] = -1;
    if (t < a.T) {
      k[i] = ld_global16(a.k + t * a.stride + col);
      v[i] = ld_global16(a.v + t * a.stride + col);
      slot[i] = a.slots[t];
    }
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    if (slot[i] < 0) continue;
    if (slot[i] >= a.slots_total) {
      if (h == 0 && l == 0) atomicOr(a.status, DEV_BOUNDS);
      continue;
    }
    const size_t row = ((static_cast<size_t>(slot[i] >> shift) * a.Hkv + h) << shift) + (slot[i] & mask);
    store8<kE4M3Cache, false>(a, ks, vs, row * D + 8 * l, k[i], v[i], nullptr);
  }
}

// With means.  A block takes one KV head and the runs (tokens of one page, one behind
// another) that begin in its window of tokens, wherever they end; every row is so
// read once, stored and added to its page's sum.  The rows in front of a run
// come from the cache: no block writes what another reads.  The block's threads are
// shared between its runs: all of them on one (a prompt), or D/8 on each (a decoding step).
// Bound: HBM for prompts (28 005 tokens of 8 heads, bf16: 43 us; 50 when rows were copied
// by token and each page summed afterwards, since L2 had lost a part of k by then, and
// 55 without the requests to L2 ahead), the conversions for E4M3 prompts (38 us), latency
// for a step (4.5 us).
// E4M3 prompts want more warps for their conversions, bf16 ones and steps more loads per thread
// (5 blocks of 1 row ahead against 4 of 2: 38 us and 42, bf16 43 and 42.7, steps 4.8 and 4.5).
constexpr bool write_by_warps(int D, bool e4m3, int window) { return e4m3 && window > kWriteThreads / (D / 8); }
template <int D, bool kE4M3Cache, int WINDOW>
__global__ void __launch_bounds__(kWriteThreads, write_by_warps(D, kE4M3Cache, WINDOW) ? 5 : 4)
    paged_write_kernel(const WriteArgs a) {
  constexpr int LANES = D / 8, GROUPS = kWriteThreads / LANES, AHEAD = write_by_warps(D, kE4M3Cache, WINDOW) ? 1 : 2;
  __shared__ int s_first[WINDOW], s_slot[WINDOW];
  __shared__ uint32_t s_break[kWriteThreads / 32], s_lead[kWriteThreads / 32];
  __shared__ float s_sum[GROUPS][D];
  pdl_begin();
  const unsigned window = blockIdx.x / static_cast<unsigned>(a.Hkv);
  const int h = static_cast<int>(blockIdx.x - window * a.Hkv), g = threadIdx.x / LANES, l = threadIdx.x % LANES;
  const long long start = static_cast<long long>(window) * WINDOW;
  const size_t col = static_cast<size_t>(h) * D + 8 * l;
  const int shift = 31 - __clz(a.page), mask = a.page - 1;
  // the window's rows, 128 bytes per request, set out before the first slot is known
  constexpr int LINES = D / 64;
  for (int i = g; i < WINDOW; i += GROUPS) {
    if (start + i >= a.T || l >= 2 * LINES) continue;
    const __nv_bfloat16* row = (l < LINES ? a.k : a.v) + (start + i) * a.stride + static_cast<size_t>(h) * D;
    asm volatile("prefetch.global.L2 [%0];" ::"l"(row + l % LINES * 64));
  }
  // where runs begin: a thread looks at one token of the window or of the 128
  // behind it (a run ends with its page)
  int count = 0;
  {
    static_assert(WINDOW + 128 <= kWriteThreads, "a thread per token");
    const long long t = start + threadIdx.x;
    const int mine = t < a.T ? a.slots[t] : -1, before = t > 0 && t <= a.T ? a.slots[t - 1] : -1;
    const bool begins = mine < 0 || (mine & mask) == 0 || before != mine - 1;
    const bool leads = begins && mine >= 0 && mine < a.slots_total && threadIdx.x < WINDOW;
    if (mine >= a.slots_total && threadIdx.x < WINDOW && h == 0) atomicOr(a.status, DEV_BOUNDS);
    const uint32_t bb = __ballot_sync(0xffffffffu, begins), lb = __ballot_sync(0xffffffffu, leads);
    if (lane_id() == 0) {
      s_break[warp_id()] = bb;
      s_lead[warp_id()] = lb;
    }
    __syncthreads();
    int rank = __popc(lb & ((1u << lane_id()) - 1u));
#pragma unroll
    for (int i = 0; i < kWriteThreads / 32; ++i) {
      if (i < warp_id()) rank += __popc(s_lead[i]);
      count += __popc(s_lead[i]);
    }
    if (leads) {
      s_first[rank] = static_cast<int>(threadIdx.x);
      s_slot[rank] = mine;
    }
    __syncthreads();
  }
  const Scale ks = {a.k_scale, a.k_inv, a.k_most}, vs = {a.v_scale, a.v_inv, a.v_most};
  // teams of `size` times D/8 threads, one run each
  int size = GROUPS;
  while (size > 1 && size * count > GROUPS) size /= 2;
  const int member = g % size;
  for (int n0 = 0; n0 < count; n0 += GROUPS / size) {
    const int n = n0 + g / size;
    float sum[8] = {};
    int rows = 0, page_id = 0;
    if (n < count) {
      const int at = s_first[n], first_slot = s_slot[n], off = first_slot & mask;
      page_id = first_slot >> shift;
      // the run reaches to the next beginning behind it
      int word = (at + 1) / 32;
      uint32_t bits = s_break[word] >> ((at + 1) % 32) << ((at + 1) % 32);
      while (bits == 0 && word < kWriteThreads / 32 - 1) bits = s_break[++word];
      // (slots that change under the call cannot lead out of the page)
      const int run = min(32 * word + (bits != 0 ? __ffs(bits) - 1 : 32) - at, a.page - off);
      rows = off + run;
      const size_t page_row = (static_cast<size_t>(page_id) * a.Hkv + h) << shift;
      const __nv_bfloat16* src_k = a.k + static_cast<size_t>(start + at) * a.stride + col;
      const __nv_bfloat16* src_v = a.v + static_cast<size_t>(start + at) * a.stride + col;
      using Word = typename std::conditional<kE4M3Cache, uint2, uint4>::type;  // 8 stored values
      const Word* old = reinterpret_cast<const Word*>(
          static_cast<const uint8_t*>(a.k_cache) + (page_row * D + 8 * l) * (kE4M3Cache ? 1 : 2));
      for (int r = member; r < off; r += 8 * size) {
        Word x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = Word{};
          if (r + i * size < off) x[i] = old[(r + i * size) * LANES];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) add8(sum, x[i], a.k_scale);
      }
      for (int r = member; r < run; r += AHEAD * size) {
        uint4 k[AHEAD], v[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          if (r + i * size < run) {
            k[i] = ld_global16(src_k + static_cast<size_t>(r + i * size) * a.stride);
            v[i] = ld_global16(src_v + static_cast<size_t>(r + i * size) * a.stride);
          }
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          if (r + i * size < run)
            store8<kE4M3Cache, true>(a, ks, vs, (page_row + off + r + i * size) * D + 8 * l, k[i], v[i], sum);
        }
      }
    }
    if (size > 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s_sum[g][8 * l + i] = sum[i];
      __syncthreads();
      if (member == 0)
        for (int o = 1; o < size; ++o)
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[i] += s_sum[g + o][8 * l + i];
      __syncthreads();
    }
    if (rows > 0 && member == 0) {
      const float n_rows = static_cast<float>(rows);
      uint4 m;
      m.x = pack_bf16(sum[0] / n_rows, sum[1] / n_rows);
      m.y = pack_bf16(sum[2] / n_rows, sum[3] / n_rows);
      m.z = pack_bf16(sum[4] / n_rows, sum[5] / n_rows);
      m.w = pack_bf16(sum[6] / n_rows, sum[7] / n_rows);
      *reinterpret_cast<uint4*>(a.k_mean + (static_cast<size_t>(page_id) * a.Hkv + h) * D + 8 * l) = m;
    }
  }
}

// ------------------------------------------------------------------ select
//
// score(page) = (sum of the group's queries) . mean, and the pages of the
// largest scores.  Which page is kept must not depend on the order of a sum:
// the score is the exact sum, rounded to fp32 once.  A first kernel takes plain
// fp32 sums and a bound of their error, E = 2^-20 |q| |mean| (16 half steps of
// the largest the sum can be; rounding the query, the products, 8 additions and
// the final rounding are 11).  With T the select-th largest of these, pages
// above T + 2E belong to the result and pages below T - 2E do not, whatever
// the exact scores are; where more pages than needed lie between (ties, or
// neighbours closer than 2^-19 of their size), those are computed in fp64 and
// ranked again.  Bound: the means are read once, 2 D bytes per page and KV head;
// 4725 pages of 40 heads (48 MB) take 12 us (15 before the next means were asked for
// while the last ones are summed, 20 in two-word fp32 arithmetic), and the choice 8 us,
// of which 3 are the exact scores of the lists that need some.

constexpr int kScoreThreads = 256;

// Keys of pages that are always kept, and of pages outside the cache (last of
// all; the attention skips them too).
constexpr uint32_t kKeyForced = 0xFFFFFFFFu, kKeyBad = 0u;

__device__ __forceinline__ bool bad_length(const SelectArgs& a, int len) {
  return len < 0 || static_cast<long long>(len) > static_cast<long long>(a.max_pages) * a.page;
}

// Sum of `group` bf16 values `step` apart, rounded to fp32 once (two words, Knuth's two-sum).
__device__ __forceinline__ float sum_of_group(const __nv_bfloat16* q, int group, int step) {
  float hi = 0.f, lo = 0.f;
  for (int i = 0; i < group; ++i) {
    const float x = __bfloat162float(q[static_cast<size_t>(i) * step]);
    const float sum = __fadd_rn(hi, x), bb = __fsub_rn(sum, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(sum, bb)), __fsub_rn(x, bb)));
    hi = sum;
  }
  return __fadd_rn(hi, lo);
}

// A block takes ROWS = 256 / D KV heads of one sequence and 8 * per_warp of its
// pages.  D/8 lanes hold a head, 8 values each; a warp sums four pages at a
// time and folds them over the lanes, so that each fold halves what is left.
template <int D>
__global__ void __launch_bounds__(kScoreThreads, 3)
    paged_score_kernel(const SelectArgs a, int head_blocks, int page_blocks, int per_warp, int stride) {
  constexpr int LANES = D / 8, ROWS = 32 / LANES;
  __shared__ float s_q[ROWS * D];
  pdl_begin();
  const int hb = blockIdx.x / page_blocks % head_blocks, b = blockIdx.x / page_blocks / head_blocks;
  const int len = a.lens[b];
  if (len == 0 || bad_length(a, len)) return;
  const int n = (len - 1) / a.page + 1, chunk = kScoreThreads / 32 * per_warp;
  long long j0 = static_cast<long long>(blockIdx.x % page_blocks) * chunk;
  if (j0 >= n) return;
  j0 += warp_id() * per_warp;
  // per_warp <= 32: a page number per lane, the first ones on their way while the queries are summed
  auto page_number = [&](long long j) {
    return j + lane_id() < min(static_cast<long long>(n), j + per_warp)
               ? a.table[static_cast<size_t>(b) * a.max_pages + j + lane_id()] : -1;
  };
  int first = page_number(j0);
  const int group = a.Hq / a.Hkv;
  {  // the group's summed query, one value per thread
    const int r = threadIdx.x / D, d = threadIdx.x % D, h = min(hb * ROWS + r, a.Hkv - 1);
    const __nv_bfloat16* q = a.q + b * a.q_stride + static_cast<size_t>(h) * group * D + d;
    s_q[threadIdx.x] = sum_of_group(q, group, D);
  }
  __syncthreads();
  const int lane = lane_id(), l = lane % LANES, h = hb * ROWS + lane / LANES;
  uint64_t q[4];
  float qq = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = lane / LANES * D + 8 * l + 2 * i;
    q[i] = f2_pack(s_q[at], s_q[at + 1]);
    qq = fmaf(s_q[at], s_q[at], fmaf(s_q[at + 1], s_q[at + 1], qq));
  }
#pragma unroll
  for (int o = LANES / 2; o > 0; o /= 2) qq += __shfl_xor_sync(0xffffffffu, qq, o);
  const float bound = 0x1p-20f * sqrtf(qq + 0x1p-120f);  // (squares of tiny values vanish)
  const __nv_bfloat16* mean = a.k_mean + static_cast<size_t>(min(h, a.Hkv - 1)) * D + 8 * l;
  const size_t page_step = static_cast<size_t>(a.Hkv) * D;
  uint32_t* keys = a.keys + 2 * (static_cast<size_t>(b) * a.Hkv + h) * stride;
  for (; j0 < n; j0 += static_cast<long long>(page_blocks) * chunk, first = page_number(j0)) {
    const int start = static_cast<int>(j0), j1 = static_cast<int>(min(static_cast<long long>(n), j0 + per_warp));
    const bool mine = start + lane < j1, outside = mine && (first < 0 || first >= a.num_pages);
    if (outside) atomicOr(a.status, DEV_BOUNDS);
    const int pid = outside || !mine ? 0 : first;
    const uint32_t bad = __ballot_sync(0xffffffffu, outside);
    // two sets of four means: each is asked for again as soon as its values are used
    uint4 x[2][4];
    auto fetch = [&](int set, int j) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[set][i] = ld_global16(mean + __shfl_sync(0xffffffffu, pid, j - start + i) * page_step);
    };
    fetch(0, start);
    fetch(1, start + 4);
    for (int j = start; j < j1; j += 8) {
#pragma unroll
      for (int set = 0; set < 2; ++set) {
        float dot[4], mm[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w[4] = {x[set][i].x, x[set][i].y, x[set][i].z, x[set][i].w};
          uint64_t s = 0, t = 0;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint64_t m = f2_pack(__uint_as_float(w[c] << 16), __uint_as_float(w[c] & 0xFFFF0000u));
            s = f2_fma(q[c], m, s);
            t = f2_fma(m, m, t);
          }
          float u, v;
          f2_unpack(s, u, v);
          dot[i] = u + v;
          f2_unpack(t, u, v);
          mm[i] = u + v;
        }
        if (j + 4 * set + 8 < j1) fetch(set, j + 4 * set + 8);
        // fold over the lanes: the upper half of each group of lanes keeps the
        // upper half of the pages
        int o = LANES / 2;
#pragma unroll
        for (int keep = 2; keep >= 1; keep /= 2, o /= 2) {
          const bool upper = l & o;
#pragma unroll
          for (int i = 0; i < keep; ++i) {
            const float sd = upper ? dot[i] : dot[i + keep], sm = upper ? mm[i] : mm[i + keep];
            dot[i] = (upper ? dot[i + keep] : dot[i]) + __shfl_xor_sync(0xffffffffu, sd, o);
            mm[i] = (upper ? mm[i + keep] : mm[i]) + __shfl_xor_sync(0xffffffffu, sm, o);
          }
        }
#pragma unroll
        for (; o > 0; o /= 2) {
          dot[0] += __shfl_xor_sync(0xffffffffu, dot[0], o);
          mm[0] += __shfl_xor_sync(0xffffffffu, mm[0], o);
        }
        // lane bits LANES/2 and LANES/4 name the page
        const int page = j + 4 * set + ((l & (LANES / 2)) ? 2 : 0) + ((l & (LANES / 4)) ? 1 : 0);
        if (l % (LANES / 4) == 0 && page < j1 && h < a.Hkv) {
          uint32_t key = score_key_bits(__float_as_uint(dot[0]));
          float off = bound * sqrtf(mm[0] + 0x1p-120f);
          if (page < a.sink || page >= n - a.recent) key = kKeyForced, off = 0.f;
          if ((bad >> (page - start)) & 1u) key = kKeyBad, off = 0.f;
          keys[page] = key;
          keys[stride + page] = __float_as_uint(off);
        }
      }
    }
  }
}

constexpr int kTopkKeys = 8;    // consecutive keys per thread and pass of the block
constexpr int kTopkCap = 8192;  // places of a list in shared memory; those of longer lists stay in L2
constexpr int kTopkOpen = 256;  // pages whose rank is found one by one
struct TopkShared {
  uint32_t digit, left, least;
  int warp[32], near, open, above;
  uint32_t off[32], low[32], high[32];
  uint32_t key[kTopkOpen], exact[kTopkOpen];
  int page[kTopkOpen], rank[kTopkOpen], open_page[kTopkOpen];
  double q[128];
};
// 8 consecutive words (a list's rows are padded to 16 bytes).
__device__ __forceinline__ void load8(const uint32_t* p, uint32_t* x) {
  *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(p);
  *reinterpret_cast<uint4*>(x + 4) = *reinterpret_cast<const uint4*>(p + 4);
}
// visit(page, word) for every word of a list, 8 consecutive ones per thread and pass.
template <typename F>
__device__ __forceinline__ void each(const uint32_t* at, int n, F visit) {
#pragma unroll 1
  for (int j = threadIdx.x * kTopkKeys; j < n; j += blockDim.x * kTopkKeys) {
    uint32_t x[kTopkKeys];
    load8(at + j, x);
#pragma unroll
    for (int i = 0; i < kTopkKeys; ++i)
      if (j + i < n) visit(j + i, x[i]);
  }
}
// The counter from the top that holds the `left`-th, and how many of it are among them.
template <bool CLEAR>
__device__ __forceinline__ void count_from_top(uint32_t* hist, int bins, uint32_t left, TopkShared& sh) {
  const int tid = threadIdx.x, w = warp_id(), lane = lane_id(), warps = blockDim.x / 32;
  const int top = bins - 1 - 4 * tid;  // four neighbouring ones per thread
  uint32_t c[4], own = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = 0;
    if (top < i) continue;
    c[i] = hist[top - i];
    if (CLEAR) hist[top - i] = 0;
    own += c[i];
  }
  uint32_t upto = own;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += y;
  }
  if (lane == 31) sh.warp[w] = static_cast<int>(upto);
  __syncthreads();
  uint32_t above = __reduce_add_sync(0xffffffffu, lane < w && lane < warps ? sh.warp[lane] : 0) + upto - own;
  if (above < left && left <= above + own) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (above < left && left <= above + c[i]) {
        sh.digit = static_cast<uint32_t>(top - i);
        sh.left = left - above;
      }
      above += c[i];
    }
  }
  __syncthreads();
}
// The largest key k with (number of keys >= k) >= keep, and how many of the keys
// equal to it belong to the first `keep`: by digits of log2(bins) bits, counted in hist, which is
// zero before and after.
__device__ __forceinline__ void nth_key(const uint32_t* keys, int n, int keep, int bins, uint32_t* hist, TopkShared& sh, uint32_t* key,
                                        int* equal) {
  uint32_t prefix = 0, left = keep;
  for (int rest = 32; rest > 0;) {
    const int width = min(31 - __clz(bins), rest), shift = rest - width;
    each(keys, n, [&](int, uint32_t x) {
      if (rest == 32 || x >> rest == prefix) atomicAdd(&hist[(x >> shift) & ((1u << width) - 1u)], 1u);
    });
    __syncthreads();
    count_from_top<true>(hist, bins, left, sh);
    prefix = (prefix << width) | sh.digit;
    left = sh.left;
    rest = shift;
  }
  *key = prefix;
  *equal = static_cast<int>(left);
}

__device__ __forceinline__ float key_score(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}

// Which scores lie within 2E of a key's: all of them where infinities or NaN are around.
__device__ __forceinline__ uint2 around(uint32_t key, float off) {
  const float t = key_score(key);
  if (!(fabsf(t) < INFINITY && off < INFINITY)) return make_uint2(kKeyBad + 1, kKeyForced - 1);
  return make_uint2(score_key_bits(__float_as_uint(t - 2.f * off)), score_key_bits(__float_as_uint(t + 2.f * off)));
}
__device__ __forceinline__ void is_open(TopkShared& sh, int page) {
  const int i = atomicAdd(&sh.open, 1);  // (their order says nothing about the result)
  if (i < kTopkOpen) sh.open_page[i] = page;
}
// The rare ways are functions of their own: every block fetches the kernel's instructions once,
// and with these in between a list took 0.7 us more.
//
// A lane's values of a page's mean, and the exact score from the queries summed in sh.q.
struct Mean {
  float x[4];
};
__device__ __forceinline__ Mean load_mean(const SelectArgs& a, int b, int h, int page) {
  // (the score kernel has found the page number inside the cache)
  const int pid = min(max(a.table[static_cast<size_t>(b) * a.max_pages + page], 0), a.num_pages - 1);
  const __nv_bfloat16* mean = a.k_mean + (static_cast<size_t>(pid) * a.Hkv + h) * a.D;
  Mean m;
#pragma unroll
  for (int i = 0; i < 4; ++i) m.x[i] = 32 * i < a.D ? __bfloat162float(mean[32 * i + lane_id()]) : 0.f;
  return m;
}
__device__ __forceinline__ uint32_t exact_key(const SelectArgs& a, const TopkShared& sh, const Mean& m) {
  double s = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (32 * i < a.D) s += sh.q[32 * i + lane_id()] * static_cast<double>(m.x[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return score_key_bits(__float_as_uint(static_cast<float>(s)));
}
__device__ __forceinline__ void sum_queries(const SelectArgs& a, TopkShared& sh, int b, int h) {
  const int group = a.Hq / a.Hkv;
  for (int d = threadIdx.x; d < a.D; d += blockDim.x) {
    const __nv_bfloat16* q = a.q + b * a.q_stride + static_cast<size_t>(h) * group * a.D + d;
    double s = 0;
    for (int i = 0; i < group; ++i) s += static_cast<double>(__bfloat162float(q[static_cast<size_t>(i) * a.D]));
    sh.q[d] = s;
  }
  __syncthreads();
}
// The words of the open pages become `yes` for the best `room` of them, `no` for the others.
__device__ __noinline__ void settle(const SelectArgs& a, TopkShared& sh, int b, int h, int room, uint32_t* words,
                                    uint32_t yes, uint32_t no) {
  const int open = sh.open, w = warp_id(), warps = blockDim.x / 32;
  Mean m = {};
  if (w < open) m = load_mean(a, b, h, sh.open_page[w]);
  sum_queries(a, sh, b, h);
  for (int i = w; i < open; i += warps) {
    if (i != w) m = load_mean(a, b, h, sh.open_page[i]);
    const uint32_t key = exact_key(a, sh, m);
    if (lane_id() == 0) sh.exact[i] = key;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < open; i += blockDim.x) {
    int rank = 0;
    for (int k = 0; k < open; ++k)
      rank += sh.exact[k] > sh.exact[i] || (sh.exact[k] == sh.exact[i] && sh.open_page[k] < sh.open_page[i]);
    words[sh.open_page[i]] = rank < room ? yes : no;
  }
  __syncthreads();
}
// Without steps: the threshold digit by digit.  Returned are the key above which pages are kept,
// and how many of those that equal it.
__device__ __noinline__ uint2 by_digits(const SelectArgs& a, TopkShared& sh, int b, int h, uint32_t* hist, uint32_t* keys,
                                        int n, int keep, int bins, float off) {
  uint32_t last;
  int equal;
  nth_key(keys, n, keep, bins, hist, sh, &last, &equal);
  if (last == kKeyForced || last == kKeyBad) return make_uint2(last, equal);
  const uint2 open = around(last, off);
  each(keys, n, [&](int page, uint32_t x) {
    if (x > open.y) atomicAdd(&sh.above, 1);
    if (x >= open.x && x <= open.y) is_open(sh, page);
  });
  __syncthreads();
  if (sh.open <= kTopkOpen) {
    settle(a, sh, b, h, keep - sh.above, keys, kKeyForced, kKeyBad);
    return make_uint2(open.y, 0);
  }
  // ties en masse: exact keys for all of them, forced and bad ones for the rest, and the
  // threshold again
  sum_queries(a, sh, b, h);
  const int lane = lane_id();
  for (int j0 = warp_id() * 32; j0 < n; j0 += blockDim.x) {
    uint32_t key = j0 + lane < n ? keys[j0 + lane] : kKeyBad;
    uint32_t todo = __ballot_sync(0xffffffffu, key >= open.x && key <= open.y);
    key = key > open.y ? kKeyForced : kKeyBad;
    while (todo != 0) {
      const int k = __ffs(todo) - 1;
      todo &= todo - 1;
      const uint32_t x = exact_key(a, sh, load_mean(a, b, h, j0 + k));
      if (lane == k) key = x;
    }
    if (j0 + lane < n) keys[j0 + lane] = key;
  }
  __syncthreads();
  nth_key(keys, n, keep, bins, hist, sh, &last, &equal);
  return make_uint2(last, equal);
}

// One block per (sequence, KV head).  The scores are counted in equal steps from the least to
// the largest.  Pages above the neighbours of the step that holds the select-th are kept, those
// below them are not (a step is wider than 2E); of the few in between the select-th is found by
// rank, and what lies within 2E of it is ranked by the exact scores.  Where that does not
// separate few pages (infinite scores, a range as narrow as the bound, ties en masse), the
// threshold is found digit by digit (which for all lists took 1 to 2 us more than steps).  Ties en
// masse, more than 256 pages within the bound, cost an exact score each, 0.13 us a page of a list: 4725
// pages of 40 heads take 21 us as they come, 106 us where there are 8 different means, 335 us where half
// of the means are equal and 620 us where all are.
__global__ void __launch_bounds__(1024) paged_topk_kernel(const __grid_constant__ SelectArgs a, int stride, int bins) {
  extern __shared__ __align__(16) uint32_t hist[];  // [bins], then the places of a list that fits
  __shared__ TopkShared sh;
  const int bh = blockIdx.x, b = bh / a.Hkv, h = bh % a.Hkv, tid = threadIdx.x, w = warp_id(), lane = lane_id();
  const int threads = blockDim.x, warps = threads / 32;
  for (int i = tid; i < bins; i += threads) hist[i] = 0;
  if (tid == 0) sh.near = sh.open = sh.above = 0;
  // (the score kernel neither writes the lengths nor begins before what does has ended; an L1
  // may hold older ones until the wait)
  const int len = __ldcg(a.lens + b);
  pdl_begin();
  const bool bad = bad_length(a, len);
  if (bad && tid == 0) atomicOr(a.status, DEV_BOUNDS);
  const int n = bad || len == 0 ? 0 : (len - 1) / a.page + 1;
  const int keep = min(n, a.select);
  int32_t* sel = a.sel + static_cast<size_t>(bh) * a.select;
  // (unsigned: i passes the largest int where select is near it)
  for (unsigned i = keep + tid; i < static_cast<unsigned>(a.select); i += threads) sel[i] = -1;
  if (n <= keep) {
    for (int i = tid; i < n; i += threads) sel[i] = i;
    return;
  }
  uint32_t* keys = a.keys + 2 * static_cast<size_t>(bh) * stride;
  // places: 0 for pages outside the cache, bins - 1 for pages always kept, steps of the scores between
  uint32_t* places = n <= kTopkCap ? hist + bins : keys + stride;
  const int pass = threads * kTopkKeys, mine = tid * kTopkKeys;
  // the keys, their range, and the largest error bound (bounds are >= 0: ordered as integers)
  uint32_t x[kTopkKeys], off_bits = 0, low = kKeyForced, high = kKeyBad;
  for (int j = mine; j < n; j += pass) {
    uint32_t e[kTopkKeys];
    load8(keys + j, x);
    load8(keys + stride + j, e);
#pragma unroll
    for (int i = 0; i < kTopkKeys; ++i) {
      if (j + i >= n) continue;
      off_bits = max(off_bits, e[i]);
      if (x[i] == kKeyForced || x[i] == kKeyBad) continue;
      low = min(low, x[i]);
      high = max(high, x[i]);
    }
  }
  off_bits = __reduce_max_sync(0xffffffffu, off_bits);
  low = __reduce_min_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);
  if (lane == 0) sh.off[w] = off_bits, sh.low[w] = low, sh.high[w] = high;
  __syncthreads();
  const float off = __uint_as_float(__reduce_max_sync(0xffffffffu, lane < warps ? sh.off[lane] : 0u));
  low = __reduce_min_sync(0xffffffffu, lane < warps ? sh.low[lane] : kKeyForced);
  high = __reduce_max_sync(0xffffffffu, lane < warps ? sh.high[lane] : kKeyBad);

  const float base = key_score(low), range = key_score(high) - base, per_unit = static_cast<float>(bins - 2) / range;
  bool by_step = low < high && range < INFINITY && per_unit < INFINITY && 2.f * off * per_unit < 0.9f;
  uint32_t last = 0;  // kept: pages whose place (or key) is above `last`, and the first `equal` of those at it
  int equal = 0;
  if (by_step) {
    uint32_t place[kTopkKeys];
    auto places_of = [&]() {
#pragma unroll
      for (int i = 0; i < kTopkKeys; ++i) {
        const int step = 1 + min(max(static_cast<int>((key_score(x[i]) - base) * per_unit), 0), bins - 3);
        place[i] = x[i] == kKeyForced ? bins - 1 : x[i] == kKeyBad ? 0 : step;
      }
    };
#pragma unroll 1
    for (int j = mine; j < n; j += pass) {
      if (n > pass) load8(keys + j, x);
      places_of();
#pragma unroll
      for (int i = 0; i < kTopkKeys; ++i) {
        if (j + i >= n) break;
        atomicAdd(&hist[place[i]], 1u);
        places[j + i] = place[i];
      }
    }
    __syncthreads();
    count_from_top<false>(hist, bins, keep, sh);
    const uint32_t at = sh.digit;
    last = at;
    if (at == 0 || at == static_cast<uint32_t>(bins - 1)) {
      equal = static_cast<int>(sh.left);
    } else {
      const uint32_t first = max(at - 1, 1u);
      last = min(at + 1, static_cast<uint32_t>(bins - 2));
      const int over = last > at ? static_cast<int>(hist[last]) : 0, room = static_cast<int>(sh.left) + over;
      const int near = over + static_cast<int>(hist[at]) + (first < at ? static_cast<int>(hist[first]) : 0);
      if (near <= kTopkOpen) {
#pragma unroll 1
        for (int j = mine; j < n; j += pass) {
          if (n > pass) {
            load8(keys + j, x);
            places_of();
          }
#pragma unroll
          for (int i = 0; i < kTopkKeys; ++i) {
            if (j + i >= n || place[i] < first || place[i] > last) continue;
            const int k = atomicAdd(&sh.near, 1);
            if (k >= kTopkOpen) continue;  // (as for the list below: keys that change under the call)
            sh.page[k] = j + i;
            sh.key[k] = x[i];
          }
        }
        __syncthreads();
        for (int i = tid; i < near; i += threads) {
          int rank = 0;
#pragma unroll 4
          for (int k = 0; k < near; ++k)
            rank += sh.key[k] > sh.key[i] || (sh.key[k] == sh.key[i] && sh.page[k] < sh.page[i]);
          sh.rank[i] = rank;
          if (rank == room - 1) sh.least = sh.key[i];
        }
        __syncthreads();
        const uint2 open = around(sh.least, off);
        for (int i = tid; i < near; i += threads) {
          // (kept by rank, unless the exact scores are asked below)
          places[sh.page[i]] = sh.rank[i] < room ? bins - 1 : 0;
          if (sh.key[i] > open.y) atomicAdd(&sh.above, 1);
          if (sh.key[i] >= open.x && sh.key[i] <= open.y) is_open(sh, sh.page[i]);
        }
        __syncthreads();
        if (sh.open > room - sh.above) settle(a, sh, b, h, room - sh.above, places, bins - 1, 0);
      } else {
        by_step = false;
        __syncthreads();
        for (int i = tid; i < bins; i += threads) hist[i] = 0;
        __syncthreads();
      }
    }
  }
  if (!by_step) {
    const uint2 cut = by_digits(a, sh, b, h, hist, keys, n, keep, bins, off);
    last = cut.x;
    equal = static_cast<int>(cut.y);
  }
  // in order
  const uint32_t* words = by_step ? places : keys;
  int more0 = 0, same0 = 0;
#pragma unroll 1
  for (int base_page = 0; base_page < n; base_page += pass) {
    const int j = base_page + mine;
    if (j < n) load8(words + j, x);
    int own = 0;  // kept above in the low half, equal in the high half
#pragma unroll
    for (int i = 0; i < kTopkKeys; ++i)
      if (j + i < n) own += x[i] > last ? 1 : (x[i] == last ? 0x10000 : 0);
    int upto = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += y;
    }
    __syncthreads();
    if (lane == 31) sh.warp[w] = upto;
    __syncthreads();
    const int there = lane < warps ? sh.warp[lane] : 0;
    const int before = upto - own + __reduce_add_sync(0xffffffffu, lane < w ? there : 0);
    const int all = __reduce_add_sync(0xffffffffu, there);
    int more = more0 + (before & 0xFFFF), same = same0 + (before >> 16);
#pragma unroll
    for (int i = 0; i < kTopkKeys; ++i) {
      if (j + i >= n) break;
      const bool tie = x[i] == last;
      const int to = more + min(same, equal);
      // (keys that another call overwrites cannot lead out of the list)
      if ((x[i] > last || (tie && same < equal)) && to < keep) sel[to] = j + i;
      more += x[i] > last;
      same += tie;
    }
    more0 += all & 0xFFFF;
    same0 += all >> 16;
  }
}

}  // namespace

cudaError_t launch_paged_plan(const PlanArgs& a, cudaStream_t stream) {
  const size_t smem = (3 * static_cast<size_t>(a.B) + 2) * sizeof(int32_t);
  const bool place = a.T <= kPlanTokens;
  const int items = std::max(a.B, place ? a.T : 0);
  const int threads = items > 512 || !place ? kPlanMaxThreads : items > 256 ? 512 : 256;
  // (48 KB without asking, the kernel's own sums among them: from 4052 sequences on)
  if (smem + kPlanSums * 2 * sizeof(long long) > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  cudaError_t e = launch_dependent(paged_plan_kernel, 1, threads, smem, stream, a, place);
  if (e != cudaSuccess || place) return e;
  return launch_dependent(paged_place_kernel, std::min((a.T + 256 * kPlanAtOnce - 1) / (256 * kPlanAtOnce), 1024), 256,
                          (static_cast<size_t>(a.B) + 1) * sizeof(int32_t), stream, a);
}

template <int D, bool E4M3>
static cudaError_t write_launch(const WriteArgs& a, int sms, cudaStream_t stream) {
  constexpr int GROUPS = kWriteThreads / (D / 8);
  // four rows per thread once that leaves every SM eight blocks
  const bool many = static_cast<long long>(a.T) * a.Hkv >= 8LL * sms * 4 * GROUPS;
  const int window = GROUPS * (many ? 4 : 1);
  const unsigned blocks = static_cast<unsigned>((static_cast<long long>(a.T) + window - 1) / window * a.Hkv);
  auto kernel = a.k_mean ? (many ? paged_write_kernel<D, E4M3, 4 * GROUPS> : paged_write_kernel<D, E4M3, GROUPS>)
                         : (many ? paged_copy_kernel<D, E4M3, 4> : paged_copy_kernel<D, E4M3, 1>);
  return launch_dependent(kernel, blocks, kWriteThreads, 0, stream, a);
}

cudaError_t launch_paged_write(const WriteArgs& a, bool e4m3, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  WriteArgs c = a;
  c.k_inv = e4m3 ? 1.f / a.k_scale : 1.f;
  c.v_inv = e4m3 ? 1.f / a.v_scale : 1.f;
  // -2048 scale cut to its upper half: a bf16 number, twice
  auto most = [](float s) {
    if (!(s >= 0x1p-60f && s <= 0x1p60f)) return 0u;
    const float x = -2048.f * s;
    uint32_t w;
    memcpy(&w, &x, sizeof(w));
    return (w & 0xFFFF0000u) | (w >> 16);
  };
  c.k_most = most(a.k_scale);
  c.v_most = most(a.v_scale);
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  if (a.D == 128) return e4m3 ? write_launch<128, true>(c, sms, stream) : write_launch<128, false>(c, sms, stream);
  return e4m3 ? write_launch<64, true>(c, sms, stream) : write_launch<64, false>(c, sms, stream);
}

// Keys of a row: whole 16-byte words for every thread's eight.
static int key_stride(int max_pages) { return (max_pages + kTopkKeys - 1) / kTopkKeys * kTopkKeys; }

size_t paged_select_workspace_bytes(int B, int Hkv, int max_pages) {
  return 2 * static_cast<size_t>(B) * Hkv * key_stride(max_pages) * sizeof(uint32_t);
}

cudaError_t launch_paged_select(const SelectArgs& a, cudaStream_t stream) {
  const int rows = 256 / a.D, head_blocks = (a.Hkv + rows - 1) / rows;
  const int stride = key_stride(a.max_pages);
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  // 32 pages per warp; fewer where that would leave SMs idle
  int per_warp = 32;
  while (per_warp > 8 && static_cast<long long>(a.B) * head_blocks *
                                 ((a.max_pages + 8 * per_warp - 1) / (8 * per_warp)) < 2 * sms)
    per_warp /= 2;
  // and no more blocks than a few rounds of all SMs: a table is often far longer than its sequences
  const long long pairs = static_cast<long long>(a.B) * head_blocks;
  const int page_blocks = static_cast<int>(
      std::min<long long>((a.max_pages + 8 * per_warp - 1) / (8 * per_warp), std::max<long long>(1, 16 * sms / pairs)));
  const unsigned blocks = static_cast<unsigned>(static_cast<long long>(a.B) * head_blocks * page_blocks);
  e = launch_dependent(a.D == 128 ? paged_score_kernel<128> : paged_score_kernel<64>, blocks, kScoreThreads, 0, stream, a,
                       head_blocks, page_blocks, per_warp, stride);
  if (e != cudaSuccess) return e;
  // as many threads as the longest list keeps busy; of the counters, four per thread
  const int threads = std::min((stride / kTopkKeys + 127) / 128 * 128, 1024), bins = std::min(4 * threads, 2048);
  return launch_dependent(paged_topk_kernel, a.B * a.Hkv, threads, (bins + std::min(stride, kTopkCap)) * sizeof(uint32_t),
                          stream, a, stride, bins);
}

}  // namespace mcs
