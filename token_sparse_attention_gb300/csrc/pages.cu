// Pages of the cache that several sequences hold: new sequences from old ones (forks, reordered
// beams, ended sequences), pages moved to the front of the cache, and the copies both ask for.
//
// Fork: child i of parent p holds p's pages.  A full page is held by all of them; the open
// last page stays with the first child, if nobody else holds it, and the others get a fresh page
// and a copy.  With c children of p every full page's holders change by c - 1, its open page's by
// 0 or -1; a page whose holders vanish goes back to the free list.  Compaction: with U pages in
// use, the i-th used one from the back goes to the i-th free one from the front, while that is one
// of the first U: M moves, at most as many as are asked for.  Which pages are free
// afterwards, and their order, follows from counts: of the pages in front of page p, u in use,
// max(0, p - u - M) + max(0, u - (U - M)) are free then.
//
// Both are integers and latency: a pass over the tables, one or two over an array of the
// pages, sums over it, and a decision before anything is written.  One cluster of 8 CTAs does all of
// it with its hardware barrier between the passes, in one launch; large tables are written by a
// second one (programmatically dependent) on all SMs.  Sums and maxima over pages are integer atomics,
// whose order changes nothing.
//
// Measured: 128 beams with 137 pages each, 2413 pages: 12.7 us (a launch 2, then seven passes, each a
// round trip to L2 and a cluster barrier); 120 sequences on 13 000 pages 14.6; compaction of 3780 pages
// 12.6.  Copies: 915 pages of 8 heads (472 MB read and written) 77 us, 6.1 TB/s, 90 % of a copy.
#include <algorithm>

#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace mcs {
namespace {

constexpr int kCluster = 8;
constexpr int kThreads = 1024;
constexpr int kAll = kCluster * kThreads;
constexpr int kWarps = kThreads / 32;
constexpr long long kTableHere = 1 << 16;  // entries of a table that the cluster writes itself

// What the CTAs tell each other: two words of each in everyone's shared memory.
struct Told {
  int2 of[kCluster];
};
__device__ __forceinline__ void tell(Told& told, int2 x) {
  if (threadIdx.x >= kCluster) return;
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(&told.of[blockIdx.x])), "r"(threadIdx.x));
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(x.x), "r"(x.y) : "memory");
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Exclusive sum of x over the CTA's threads, and the total.  `sums` holds 33 words; it may be used
// again after the next barrier.
__device__ __forceinline__ int block_scan(int x, int* sums, int& total) {
  int y = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, d);
    if (lane_id() >= d) y += z;
  }
  if (lane_id() == 31) sums[warp_id()] = y;
  __syncthreads();
  if (warp_id() == 0) {
    int s = sums[lane_id()];
    const int own = s;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, s, d);
      if (lane_id() >= d) s += z;
    }
    sums[lane_id()] = s - own;
    if (lane_id() == 31) sums[32] = s;
  }
  __syncthreads();
  total = sums[32];
  const int before = sums[warp_id()] + y - x;
  __syncthreads();
  return before;
}

// Calls f(row, j, page number) for the pages of all rows: the cluster's warps share the rows, or
// several of them one row where there are few.
template <typename F>
__device__ __forceinline__ void for_pages(const PagesArgs& a, F f) {
  const int shift = 31 - __clz(a.page), warps = kCluster * kWarps;
  const int w = blockIdx.x * kWarps + warp_id();
  const int ways = max(1, warps / a.B);
  for (int u = w; u < a.B * ways; u += warps) {
    const int b = u / ways, len = a.lens[b];
    const int pages = len <= 0 ? 0 : static_cast<int>(min((static_cast<long long>(len) + a.page - 1) >> shift, static_cast<long long>(a.max_pages)));
    const int32_t* row = a.table + static_cast<size_t>(b) * a.max_pages;
    for (int j0 = (u % ways) * 128; j0 < pages; j0 += ways * 128) {
      int pid[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = j0 + 32 * k + lane_id();
        pid[k] = j < pages ? row[j] : -2;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (j0 + 32 * k + lane_id() < pages) f(b, j0 + 32 * k + lane_id(), pid[k], len);
    }
  }
}

// ------------------------------------------------------------------ fork

// Rows of the new table, shared by the warps first, first + warps, ... of `warps`.
__device__ __forceinline__ void write_rows(const PagesArgs& a, const int32_t* fresh, int first, int warps) {
  const int shift = 31 - __clz(a.page), ways = max(1, warps / a.n);
  for (int u = first; u < a.n * ways; u += warps) {
    const int i = u / ways, parent = a.parents[i], len = parent < 0 ? 0 : a.lens[parent], pages = (len + a.page - 1) >> shift;
    const int own = __ldcg(fresh + i);
    const int32_t* from = a.table + static_cast<size_t>(max(parent, 0)) * a.max_pages;
    int32_t* to = a.table_out + static_cast<size_t>(i) * a.max_pages;
#pragma unroll 4
    for (int j = (u % ways) * 32 + lane_id(); j < a.max_pages; j += ways * 32)
      to[j] = j >= pages ? -1 : own >= 0 && j == pages - 1 ? own : from[j];
  }
}

// Workspace: a word for the launch behind this one, holders' changes [num_pages], the children's
// fresh pages [n] (-1: none).
constexpr int kWsHead = 4;  // words
__global__ void __cluster_dims__(kCluster) __launch_bounds__(kThreads) paged_fork_kernel(const PagesArgs a, bool here) {
  extern __shared__ int32_t sm[];
  int32_t* s_count = sm;             // [B] children
  int32_t* s_first = s_count + a.B;  // [B] the first of them
  int32_t* s_open = s_first + a.B;   // [B] the page that is not full, -1: none; -2 - it: which others hold, too
  __shared__ int s_sums[33];
  __shared__ Told s_told;
  int32_t* change = a.ws + kWsHead;
  int32_t* fresh = change + a.num_pages;
  const int tid = threadIdx.x, me = blockIdx.x * kThreads + tid;
  const int shift = 31 - __clz(a.page), mask = a.page - 1;
  const long long room = static_cast<long long>(a.max_pages) << shift;
  pdl_begin();
  const int head = a.free_head[0], parent0 = tid < a.n ? a.parents[tid] : -1;
  bool bad = false;
  for (int b = tid; b < a.B; b += kThreads) {
    const int len = a.lens[b];
    int open = -1;
    s_count[b] = 0, s_first[b] = 0x7fffffff;
    if (len < 0 || len > room) {
      bad = true;
    } else if ((len & mask) != 0) {
      open = a.table[static_cast<size_t>(b) * a.max_pages + (len >> shift)];
      if (open < 0 || open >= a.num_pages)
        bad = true;
      else if (a.extra[open] != 0)
        open = -2 - open;
    }
    s_open[b] = open;
  }
  for (int p = me; p < a.num_pages; p += kAll) change[p] = 0;
  __syncthreads();
#pragma unroll 1
  for (int i = tid; i < a.n; i += kThreads) {
    const int p = i == tid ? parent0 : a.parents[i];
    bad = bad || p < -1 || p >= a.B;
    if (p >= 0 && p < a.B) {
      atomicAdd(s_count + p, 1);
      atomicMin(s_first + p, i);
    }
  }
  cluster_sync();  // the changes are zero
  bad = __syncthreads_or(bad);
  if (!bad) {
    for_pages(a, [&](int b, int j, int pid, int len) {
      if (pid < 0 || pid >= a.num_pages) {
        bad = true;
        return;
      }
      const int c = s_count[b], d = j < (len >> shift) ? c - 1 : c > 0 && s_open[b] >= 0 ? 0 : -1;
      if (d != 0) atomicAdd(change + pid, d);
    });
  }
  // children that copy, and their places in the free list: every CTA counts, the last one writes
  int need = 0;
  bad = __syncthreads_or(bad);
  if (!bad) {
    bad = head < 0 || head > a.n_free;
#pragma unroll 1
    for (int i0 = 0; i0 < a.n; i0 += kThreads) {
      const int i = i0 + tid, p = i >= a.n ? -1 : i == tid ? parent0 : a.parents[i], open = p < 0 ? -1 : s_open[p];
      const bool copies = open < -1 || (open >= 0 && s_first[p] != i);
      const uint32_t votes = __ballot_sync(0xffffffffu, copies);
      if (lane_id() == 0) s_sums[warp_id()] = __popc(votes);
      __syncthreads();
      int at = head + need + __popc(votes & ((1u << lane_id()) - 1u)), total = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const int x = s_sums[w];
        at += w < warp_id() ? x : 0;
        total += x;
      }
      if (i < a.n && blockIdx.x == kCluster - 1) {
        int pid = -1;
        if (copies && at >= 0 && at < a.n_free) {
          pid = a.free_pages[at];
          bad = bad || pid < 0 || pid >= a.num_pages;
        }
        fresh[i] = pid;
      }
      need += total;
      __syncthreads();
    }
    bad = bad || need > a.n_free - head;
  }
  cluster_sync();  // the changes are there
  // pages without holders: each CTA looks at its part of the cache
  const int part = (a.num_pages + kCluster - 1) / kCluster;
  const int p0 = min(a.num_pages, part * static_cast<int>(blockIdx.x)), p1 = min(a.num_pages, p0 + part);
  int mine = 0;
  for (int p = p0 + tid; p < p1; p += kThreads) {
    const int d = __ldcg(change + p), extra = a.extra[p], holders = extra + 1 + d;
    bad = bad || extra < 0 || (d < 0 && holders < 0);
    mine += d < 0 && holders == 0;
  }
  bad = __syncthreads_or(bad);
  int freed_here;
  block_scan(mine, s_sums, freed_here);
  tell(s_told, make_int2(bad, freed_here));
  cluster_sync();
  int freed = 0, before = 0;
#pragma unroll
  for (int c = 0; c < kCluster; ++c) {
    const int2 x = s_told.of[c];
    bad = bad || x.x != 0;
    if (c < static_cast<int>(blockIdx.x)) before += x.y;
    freed += x.y;
  }
  const int head_out = head + need - freed;
  bad = bad || head_out < 0;
  if (me == 0) {
    a.ws[0] = bad;
    if (bad)
      atomicOr(a.status, DEV_BOUNDS);
    else
      a.head_out[0] = head_out;
  }
#pragma unroll 1
  for (int i = me; i < a.n; i += kAll) {
    const int p = bad ? -1 : a.parents[i], len = p < 0 ? 0 : a.lens[p], to = bad ? -1 : __ldcg(fresh + i);
    const int open = p < 0 ? -1 : s_open[p];
    if (!bad) a.lens_out[i] = len;
    a.moves[3 * i] = to < 0 ? -1 : open < 0 ? -2 - open : open;
    a.moves[3 * i + 1] = to;
    a.moves[3 * i + 2] = to < 0 ? 0 : len & mask;
  }
  if (bad) return;  // nothing is taken
  if (here) write_rows(a, fresh, blockIdx.x * kWarps + warp_id(), kCluster * kWarps);
  // the free list: what is freed, ascending, in front of what was free
#pragma unroll 1
  for (int q0 = p0; q0 < p1; q0 += kThreads) {
    const int p = q0 + tid;
    const int d = p < p1 ? __ldcg(change + p) : 0, extra = p < p1 ? a.extra[p] : 0;
    const bool gone = d < 0 && extra + 1 + d == 0;
    int total;
    const int at = before + block_scan(gone ? 1 : 0, s_sums, total);
    if (gone) a.free_out[head_out + at] = p;
    if (p < p1) a.extra_out[p] = gone ? 0 : extra + d;
    before += total;
  }
  if (a.free_out != a.free_pages)
    for (int f = head + need + me; f < a.n_free; f += kAll) a.free_out[f] = a.free_pages[f];
}

__global__ void __launch_bounds__(256) paged_fork_rows_kernel(const PagesArgs a) {
  pdl_begin();
  if (a.ws[0]) return;
  write_rows(a, a.ws + kWsHead + a.num_pages, blockIdx.x * 8 + warp_id(), gridDim.x * 8);
}

// ------------------------------------------------------------------ compaction

// The tables with the pages' new numbers, shared as above; entries past a sequence's end stay.
__device__ __forceinline__ void renumber_rows(const PagesArgs& a, const int32_t* to, int first, int warps) {
  const int shift = 31 - __clz(a.page), ways = max(1, warps / a.B);
  const bool in_place = a.table_out == a.table;
  for (int u = first; u < a.B * ways; u += warps) {
    const int b = u / ways, pages = (a.lens[b] + a.page - 1) >> shift, end = in_place ? pages : a.max_pages;
    const size_t row = static_cast<size_t>(b) * a.max_pages;
#pragma unroll 4
    for (int j = (u % ways) * 32 + lane_id(); j < end; j += ways * 32) {
      const int pid = a.table[row + j];
      a.table_out[row + j] = j < pages ? __ldcg(to + pid) : pid;
    }
  }
}

// Workspace: a word for the launch behind this one, tokens in each page [num_pages], the pages' new numbers [num_pages].
__global__ void __cluster_dims__(kCluster) __launch_bounds__(kThreads) paged_compact_kernel(const PagesArgs a, bool here) {
  __shared__ int s_sums[33];
  __shared__ Told s_told, s_front;
  int32_t* fill = a.ws + kWsHead;
  int32_t* to = fill + a.num_pages;
  const int tid = threadIdx.x, me = blockIdx.x * kThreads + tid;
  const long long room = static_cast<long long>(a.max_pages) * a.page;
  pdl_begin();
  for (int p = me; p < a.num_pages; p += kAll) fill[p] = 0;
  bool bad = false;
  for (int b = tid; b < a.B; b += kThreads) bad = bad || a.lens[b] < 0 || a.lens[b] > room;
  cluster_sync();
  for_pages(a, [&](int, int j, int pid, int len) {
    if (pid < 0 || pid >= a.num_pages)
      bad = true;
    else
      atomicMax(fill + pid, min(a.page, len - j * a.page));
  });
  bad = __syncthreads_or(bad);
  cluster_sync();
  const int part = (a.num_pages + kCluster - 1) / kCluster;
  const int p0 = min(a.num_pages, part * static_cast<int>(blockIdx.x)), p1 = min(a.num_pages, p0 + part);
  // pages in use in this CTA's part in front of page `end`
  auto count = [&](int end) {
    int mine = 0, total;
    for (int p = p0 + tid; p < min(p1, end); p += kThreads) mine += __ldcg(fill + p) > 0;
    block_scan(mine, s_sums, total);
    return total;
  };
  const int own = count(a.num_pages);
  tell(s_told, make_int2(bad, own));
  cluster_sync();
  int used = 0, before = 0;  // U, and of these in front of this CTA's part
#pragma unroll
  for (int c = 0; c < kCluster; ++c) {
    const int2 x = s_told.of[c];
    bad = bad || x.x != 0;
    if (c < static_cast<int>(blockIdx.x)) before += x.y;
    used += x.y;
  }
  const int head_out = a.n_free - (a.num_pages - used);
  bad = bad || head_out < 0;
  tell(s_front, make_int2(0, count(used)));
  cluster_sync();
  int moves = used;  // M: the free pages among the first U
#pragma unroll
  for (int c = 0; c < kCluster; ++c) moves -= s_front.of[c].y;
  moves = bad ? 0 : min(moves, a.n);
  if (me == 0) {
    a.ws[0] = bad;
    if (bad)
      atomicOr(a.status, DEV_BOUNDS);
    else
      a.head_out[0] = head_out;
  }
  for (int i = moves + me; i < a.n; i += kAll) a.moves[3 * i] = a.moves[3 * i + 1] = -1, a.moves[3 * i + 2] = 0;
  if (!bad) {
    for (int q0 = p0; q0 < p1; q0 += kThreads) {
      const int p = q0 + tid, rows = p < p1 ? __ldcg(fill + p) : 0;
      int total;
      const int u = before + block_scan(rows > 0 ? 1 : 0, s_sums, total);  // in use in front of p
      before += total;
      if (p >= p1) continue;
      const int above = used - 1 - u, below = p - u;
      const bool moves_off = rows > 0 && above < moves, taken = rows == 0 && below < moves;
      if (moves_off) a.moves[3 * above] = p, a.moves[3 * above + 2] = rows;
      if (taken) a.moves[3 * below + 1] = p;
      if (moves_off || (rows == 0 && !taken)) a.free_out[head_out + max(0, below - moves) + max(0, u - (used - moves))] = p;
      to[p] = moves_off ? above : rows > 0 ? -1 : taken ? -2 : -3;
    }
  }
  cluster_sync();
  if (!bad) {
    for (int p = p0 + tid; p < p1; p += kThreads) {
      const int m = to[p];
      if (m == -2) continue;  // what moves here writes it
      const int extra = m == -3 ? 0 : a.extra[p], at = m >= 0 ? __ldcg(a.moves + 3 * m + 1) : p;
      a.extra_out[at] = extra;
      if (at != p) a.extra_out[p] = 0;
      to[p] = at;
    }
  }
  cluster_sync();
  if (!bad && here) renumber_rows(a, to, blockIdx.x * kWarps + warp_id(), kCluster * kWarps);
}

__global__ void __launch_bounds__(256) paged_renumber_kernel(const PagesArgs a) {
  pdl_begin();
  if (a.ws[0]) return;
  renumber_rows(a, a.ws + kWsHead + a.num_pages, blockIdx.x * 8 + warp_id(), gridDim.x * 8);
}

// ------------------------------------------------------------------ copies

// A unit is one KV head's rows of one of the two caches (and, with the first, its mean), which lie one
// behind another: at most 32 KB.  A warp per unit, the next one's entry on its way; every warp by
// itself, so that one's first loads cover the other's last stores.  Bound: HBM.
constexpr int kCopyWarps = 8;
__global__ void __launch_bounds__(32 * kCopyWarps) paged_page_copy_kernel(const CopyArgs a) {
  pdl_begin();
  const int lane = lane_id();
  // unit: entry * per + which; from one of a warp's units to its next
  const int per = 2 * a.Hkv, step = gridDim.x * kCopyWarps, step_entry = step / per, step_which = step - step_entry * per;
  const int first = blockIdx.x * kCopyWarps + warp_id();
  int at = first / per, next_which = first - at * per;
  auto entry = [&](int k) { return at < a.n ? a.moves[3 * static_cast<size_t>(at) + k] : -1; };
  int from = entry(0), to = entry(1), rows = entry(2);
  while (at < a.n) {
    const int src_page = from, dst_page = to, n = rows, which = next_which, h = which >= a.Hkv ? which - a.Hkv : which;
    at += step_entry;
    next_which += step_which;
    if (next_which >= per) next_which -= per, ++at;
    from = entry(0), to = entry(1), rows = entry(2);
    if (src_page < 0) continue;
    if (src_page >= a.num_pages || dst_page < 0 || dst_page >= a.num_pages || n < 0 || n > a.page) {
      if (lane == 0) atomicOr(a.status, DEV_BOUNDS);
      continue;
    }
    if (src_page == dst_page) continue;
    const int words = n * a.row_words;
    const size_t pitch = static_cast<size_t>(a.page) * a.row_words;
    uint4* base = static_cast<uint4*>(which >= a.Hkv ? a.v : a.k);
    const uint4* src = base + (static_cast<size_t>(src_page) * a.Hkv + h) * pitch;
    uint4* dst = base + (static_cast<size_t>(dst_page) * a.Hkv + h) * pitch;
    if (a.mean != nullptr && which < a.Hkv && lane < a.mean_words) {
      uint4* mean = static_cast<uint4*>(a.mean) + static_cast<size_t>(h) * a.mean_words + lane;
      mean[static_cast<size_t>(dst_page) * a.Hkv * a.mean_words] = ld_global16(mean + static_cast<size_t>(src_page) * a.Hkv * a.mean_words);
    }
    constexpr int kAtOnce = 16;
    for (int w = lane; w < words; w += 32 * kAtOnce) {
      uint4 x[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        if (w + 32 * i < words) x[i] = ld_global16(src + w + 32 * i);
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        if (w + 32 * i < words) dst[w + 32 * i] = x[i];
    }
  }
}

}  // namespace

size_t paged_fork_workspace_bytes(int num_pages) {
  return (kWsHead + static_cast<size_t>(num_pages) + 4096) * sizeof(int32_t);
}
size_t paged_compact_workspace_bytes(int num_pages) {
  return (kWsHead + 2 * static_cast<size_t>(num_pages)) * sizeof(int32_t);
}

cudaError_t launch_paged_fork(const PagesArgs& a, cudaStream_t stream) {
  const bool here = static_cast<long long>(a.n) * a.max_pages <= kTableHere;
  constexpr int kMost = 3 * 4096 * sizeof(int32_t);
  cudaError_t e = cudaFuncSetAttribute(paged_fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
  if (e != cudaSuccess) return e;
  e = launch_dependent(paged_fork_kernel, kCluster, kThreads, 3 * a.B * sizeof(int32_t), stream, a, here);
  if (e != cudaSuccess || here) return e;
  int sms = 0;
  if ((e = sm_count(&sms)) != cudaSuccess) return e;
  return launch_dependent(paged_fork_rows_kernel, 4 * sms, 256, 0, stream, a);
}

cudaError_t launch_paged_compact(const PagesArgs& a, cudaStream_t stream) {
  const bool here = static_cast<long long>(a.B) * a.max_pages <= kTableHere;
  cudaError_t e = launch_dependent(paged_compact_kernel, kCluster, kThreads, 0, stream, a, here);
  if (e != cudaSuccess || here) return e;
  int sms = 0;
  if ((e = sm_count(&sms)) != cudaSuccess) return e;
  return launch_dependent(paged_renumber_kernel, 4 * sms, 256, 0, stream, a);
}

cudaError_t launch_paged_copy(const CopyArgs& a, cudaStream_t stream) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const long long blocks = (2LL * a.Hkv * a.n + kCopyWarps - 1) / kCopyWarps;
  return launch_dependent(paged_page_copy_kernel, static_cast<unsigned>(std::min<long long>(blocks, 8LL * sms)), 32 * kCopyWarps, 0, stream, a);
}

}  // namespace mcs
