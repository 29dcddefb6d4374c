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

constexpr int kSelectThreads = 1024;

// One warp per page: the score in 64 bits, rounded to fp32 once.
__global__ void __launch_bounds__(256) paged_score_kernel(const SelectArgs a) {
  const int bh = blockIdx.y, b = bh / a.Hkv, h = bh % a.Hkv;
  const int len = a.lens[b];
  if (len < 0 || static_cast<long long>(len) > static_cast<long long>(a.max_pages) * a.page) return;
  const int n = (len + a.page - 1) / a.page;
  const int group = a.Hq / a.Hkv, lane = lane_id();
  for (int j = blockIdx.x * 8 + warp_id(); j < n; j += gridDim.x * 8) {
    uint32_t key;
    const int pid = a.table[static_cast<size_t>(b) * a.max_pages + j];
    if (pid < 0 || pid >= a.num_pages) {
      if (lane == 0) atomicOr(a.status, DEV_BOUNDS);
      key = 0;  // last of all; the attention skips it too
    } else if (j < a.sink || j >= n - a.recent) {
      key = 0xFFFFFFFFu;
    } else {
      double s = 0;
      for (int d = lane; d < a.D; d += 32) {
        double qs = 0;
        for (int g = 0; g < group; ++g)
          qs += static_cast<double>(__bfloat162float(
              a.q[static_cast<size_t>(b) * a.q_stride + static_cast<size_t>(h * group + g) * a.D + d]));
        s += qs * static_cast<double>(
                      __bfloat162float(a.k_mean[(static_cast<size_t>(pid) * a.Hkv + h) * a.D + d]));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      key = score_key_bits(__float_as_uint(static_cast<float>(s)));
    }
    if (lane == 0) a.keys[static_cast<size_t>(bh) * a.max_pages + j] = key;
  }
}

// One block per (sequence, KV head): the select-th largest key by four 8-bit
// digits, then the kept pages in order.
__global__ void __launch_bounds__(kSelectThreads) paged_topk_kernel(const SelectArgs a) {
  const int bh = blockIdx.x, b = bh / a.Hkv, tid = threadIdx.x;
  const int len = a.lens[b];
  const bool bad = len < 0 || static_cast<long long>(len) > static_cast<long long>(a.max_pages) * a.page;
  if (bad && tid == 0) atomicOr(a.status, DEV_BOUNDS);
  const int n = bad ? 0 : (len + a.page - 1) / a.page;
  const int keep = min(n, a.select);
  const uint32_t* keys = a.keys + static_cast<size_t>(bh) * a.max_pages;
  int32_t* sel = a.sel + static_cast<size_t>(bh) * a.select;
  __shared__ uint32_t hist[256];
  __shared__ uint32_t s_digit, s_left;
  __shared__ int s_warp[2][32], s_out[2];
  uint32_t prefix = 0, left = keep;
  if (n > keep) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int j = tid; j < n; j += kSelectThreads) {
        const uint32_t key = keys[j];
        if (shift == 24 || (key >> (shift + 8)) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        uint32_t above = 0;
        int d = 255;
        while (above + hist[d] < left) above += hist[d--];
        s_digit = d;
        s_left = left - above;
      }
      __syncthreads();
      prefix = (prefix << 8) | s_digit;
      left = s_left;
      __syncthreads();
    }
  }
  // keys above `prefix` are kept, and the first `left` that equal it
  if (tid < 2) s_out[tid] = 0;
  __syncthreads();
  for (int j0 = 0; j0 < n; j0 += kSelectThreads) {
    const int j = j0 + tid;
    const uint32_t key = j < n ? keys[j] : 0;
    const bool all = n <= keep;
    const bool more = j < n && (all || key > prefix), same = j < n && !all && key == prefix;
    const uint32_t mb = __ballot_sync(0xffffffffu, more), sb = __ballot_sync(0xffffffffu, same);
    if (lane_id() == 0) {
      s_warp[0][warp_id()] = __popc(mb);
      s_warp[1][warp_id()] = __popc(sb);
    }
    __syncthreads();
    if (warp_id() < 2) {
      int x = s_warp[warp_id()][lane_id()];
      const int own = x;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane_id() >= d) x += y;
      }
      s_warp[warp_id()][lane_id()] = x - own + s_out[warp_id()];
      __syncwarp();
      if (lane_id() == 31) s_out[warp_id()] += x;
    }
    __syncthreads();
    const uint32_t below = (1u << lane_id()) - 1u;
    const int nm = s_warp[0][warp_id()] + __popc(mb & below);
    const int ns = s_warp[1][warp_id()] + __popc(sb & below);
    const int taken = min(ns, static_cast<int>(left));
    if (more || (same && ns < static_cast<int>(left))) sel[nm + (all ? 0 : taken)] = j;
    __syncthreads();
  }
  for (int i = keep + tid; i < a.select; i += kSelectThreads) sel[i] = -1;
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

size_t paged_select_workspace_bytes(int B, int Hkv, int max_pages) {
  return static_cast<size_t>(B) * Hkv * max_pages * sizeof(uint32_t);
}

cudaError_t launch_paged_select(const SelectArgs& a, cudaStream_t stream) {
  const int bh = a.B * a.Hkv;
  const unsigned x = static_cast<unsigned>(std::min((a.max_pages + 63) / 64, 256));
  // rows of the grid's y axis are limited to 65535
  for (int b0 = 0; b0 < a.B;) {
    const int nb = std::min(a.B - b0, std::max(1, 65535 / a.Hkv));
    SelectArgs c = a;
    c.q = a.q + static_cast<size_t>(b0) * a.q_stride;
    c.table = a.table + static_cast<size_t>(b0) * a.max_pages;
    c.lens = a.lens + b0;
    c.keys = a.keys + static_cast<size_t>(b0) * a.Hkv * a.max_pages;
    paged_score_kernel<<<dim3(x, nb * a.Hkv), 256, 0, stream>>>(c);
    b0 += nb;
  }
  paged_topk_kernel<<<bh, kSelectThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace mcs
