// Paged key-value cache: pages and slots of new tokens, writes into the pages
// with the pages' mean keys, and the choice of pages by a cheap score.
#include <algorithm>

#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"

namespace mcs {
namespace {

// ------------------------------------------------------------------ plan
//
// have_b = ceil(len_b / page), need_b = ceil((len_b + new_b) / page) - have_b;
// with the exclusive sums of new and need every token and every fresh page
// finds its sequence by a binary search.  A few microseconds of latency and
// nothing else, so it is one launch: every CTA of one cluster takes the sums
// over all sequences for itself (B <= 4096: at most four rounds of one block
// scan, 32 KB from L2), checks everything that can be wrong, and
// only behind the cluster barrier, when all have read the state, writes its
// share.  The state can so be updated in place and a request that cannot be
// met takes nothing.

constexpr int kPlanThreads = 1024;
constexpr int kPlanMaxCluster = 8;

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// Inclusive sum over the block of x (all threads call); `sums` holds 32 values.
__device__ __forceinline__ long long block_scan(long long x, long long* sums) {
  const int lane = lane_id(), w = warp_id();
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) sums[w] = x;
  __syncthreads();
  if (w == 0) {
    long long t = sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, t, d);
      if (lane >= d) t += y;
    }
    sums[lane] = t;
  }
  __syncthreads();
  if (w > 0) x += sums[w - 1];
  __syncthreads();
  return x;
}

// The last i in [0, n) with first[i] <= x, for ascending first with first[0] <= x.
__device__ __forceinline__ int owner(const int32_t* first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PlanArgs a, int ctas) {
  extern __shared__ int32_t sm[];
  int32_t* s_cu = sm;                // [B + 1] exclusive sums of new tokens
  int32_t* s_base = s_cu + a.B + 1;  // [B + 1] exclusive sums of missing pages
  int32_t* s_len = s_base + a.B + 1; // [B]
  __shared__ long long sums[32];
  const int tid = threadIdx.x;
  const long long room = static_cast<long long>(a.max_pages) * a.page;
  long long tokens = 0, pages = 0;
  bool bad = false;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    long long nw = 0, need = 0;
    if (b < a.B) {
      const int len = a.lens[b];
      nw = a.new_lens[b];
      if (len < 0 || nw < 0 || len + nw > room) {
        bad = true;
        nw = 0;
      } else {
        const int have = (len + a.page - 1) / a.page;
        need = (len + nw + a.page - 1) / a.page - have;
        if (nw > 0 && len % a.page != 0) {  // continues in its last page
          const int pid = a.table[static_cast<size_t>(b) * a.max_pages + len / a.page];
          bad = bad || pid < 0 || pid >= a.num_pages;
        }
      }
      s_len[b] = len;
    }
    const long long t = block_scan(nw, sums), g = block_scan(need, sums);
    if (b < a.B) {
      // sums beyond T or n_free are refused below, before they are used
      s_cu[b] = static_cast<int32_t>(tokens + t - nw);
      s_base[b] = static_cast<int32_t>(pages + g - need);
    }
    if (tid == kPlanThreads - 1) sums[0] = t, sums[1] = g;
    __syncthreads();
    tokens += sums[0];
    pages += sums[1];
    __syncthreads();
  }
  const int head = a.free_head[0];
  bad = bad || tokens > a.T || head < 0 || head > a.n_free || pages > a.n_free - head;
  bad = __syncthreads_or(bad);
  if (!bad) {
    for (int j = tid; j < pages; j += kPlanThreads) {
      const int pid = a.free_pages[head + j];
      bad = bad || pid < 0 || pid >= a.num_pages;
    }
    bad = __syncthreads_or(bad);
  }
  if (tid == 0) {
    s_cu[a.B] = static_cast<int32_t>(tokens);
    s_base[a.B] = static_cast<int32_t>(pages);
  }
  // every CTA has read what any CTA is about to write
  if (ctas > 1) cluster_sync();
  else __syncthreads();

  const int at = blockIdx.x * kPlanThreads + tid, step = ctas * kPlanThreads;
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
    const int b = owner(s_base, a.B, j);
    const int have = (s_len[b] + a.page - 1) / a.page;
    a.table[static_cast<size_t>(b) * a.max_pages + have + (j - s_base[b])] = a.free_pages[head + j];
  }
  for (int t = at; t < a.T; t += step) {
    int slot = -1, pos = -1;
    if (t < tokens) {
      const int b = owner(s_cu, a.B, t);
      pos = s_len[b] + (t - s_cu[b]);
      const int have = (s_len[b] + a.page - 1) / a.page, j = pos / a.page;
      const int pid = j < have ? a.table[static_cast<size_t>(b) * a.max_pages + j]
                               : a.free_pages[head + s_base[b] + (j - have)];
      slot = pid * a.page + pos % a.page;
    }
    a.slots[t] = slot;
    if (a.positions) a.positions[t] = pos;
  }
}

// ------------------------------------------------------------------ write

// 8 bf16 values (a 16-byte word) -> 8 E4M3 codes of x / scale.
__device__ __forceinline__ uint2 encode8(uint4 x, float scale) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = f32x2_to_e4m3x2(__fdiv_rn(__uint_as_float(w[i] << 16), scale),
                           __fdiv_rn(__uint_as_float(w[i] & 0xFFFF0000u), scale));
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// sum += the stored values: 8 bf16, or scale * 8 E4M3 codes.
__device__ __forceinline__ void add8(float* sum, uint4 x) {
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
// of it from the cache, the run's own from k, so that nothing is read that
// another thread of this launch writes.
template <bool kE4M3Cache>
__global__ void __launch_bounds__(kWriteThreads) paged_write_kernel(const WriteArgs a) {
  const int lanes = a.D / 8;
  const long long item =
      (static_cast<long long>(blockIdx.x) * kWriteThreads + threadIdx.x) / lanes;
  const int l = threadIdx.x % lanes;
  if (item >= static_cast<long long>(a.T) * a.Hkv) return;
  const int t = static_cast<int>(item / a.Hkv), h = static_cast<int>(item % a.Hkv);
  const int slot = a.slots[t];
  if (slot < 0) return;
  if (slot >= a.slots_total) {
    if (h == 0 && l == 0) atomicOr(a.status, DEV_BOUNDS);
    return;
  }
  const int page_id = slot / a.page, off = slot % a.page;
  const size_t page_row = (static_cast<size_t>(page_id) * a.Hkv + h) * a.page;
  const size_t src = static_cast<size_t>(t) * a.stride + static_cast<size_t>(h) * a.D + 8 * l;
  const size_t dst = (page_row + off) * a.D + 8 * l;
  const uint4 k = ld_global_nc16(a.k + src), v = ld_global_nc16(a.v + src);
  if (kE4M3Cache) {
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.k_cache) + dst) = encode8(k, a.k_scale);
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.v_cache) + dst) = encode8(v, a.v_scale);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.k_cache) + dst) = k;
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.v_cache) + dst) = v;
  }
  if (a.k_mean == nullptr || (t > 0 && off > 0 && a.slots[t - 1] == slot - 1)) return;
  float sum[8] = {};
  for (int r = 0; r < off; ++r) {
    const size_t row = (page_row + r) * a.D + 8 * l;
    if (kE4M3Cache)
      add8(sum, *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.k_cache) + row), a.k_scale);
    else
      add8(sum, *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.k_cache) + row));
  }
  int n = off;
  for (int u = t; u < a.T && n < a.page && a.slots[u] == slot + (u - t); ++u, ++n) {
    const uint4 x = ld_global_nc16(a.k + src + static_cast<size_t>(u - t) * a.stride);
    if (kE4M3Cache) add8(sum, encode8(x, a.k_scale), a.k_scale);
    else add8(sum, x);
  }
  const float inv = static_cast<float>(n);
  uint4 m;
  m.x = pack_bf16(sum[0] / inv, sum[1] / inv);
  m.y = pack_bf16(sum[2] / inv, sum[3] / inv);
  m.z = pack_bf16(sum[4] / inv, sum[5] / inv);
  m.w = pack_bf16(sum[6] / inv, sum[7] / inv);
  *reinterpret_cast<uint4*>(a.k_mean + (static_cast<size_t>(page_id) * a.Hkv + h) * a.D + 8 * l) = m;
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
  // one CTA per 4096 tokens or sequences, up to one cluster
  const long long items = std::max<long long>(a.T, a.B);
  int ctas = 1;
  while (ctas < kPlanMaxCluster && items > 4096LL * ctas) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaError_t e = cudaFuncSetAttribute(paged_plan_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, 49168);
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, paged_plan_kernel, a, ctas);
}

cudaError_t launch_paged_write(const WriteArgs& a, bool e4m3, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  const long long threads = static_cast<long long>(a.T) * a.Hkv * (a.D / 8);
  const unsigned blocks = static_cast<unsigned>((threads + kWriteThreads - 1) / kWriteThreads);
  if (e4m3) paged_write_kernel<true><<<blocks, kWriteThreads, 0, stream>>>(a);
  else paged_write_kernel<false><<<blocks, kWriteThreads, 0, stream>>>(a);
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
