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

// What one CTA tells the others, in the workspace.
struct Told {
  int bad, a, b, c;
};

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

// Workspace: Told [kCluster], holders' changes [num_pages], the children's fresh pages [n] (-1: none).
__global__ void __cluster_dims__(kCluster) __launch_bounds__(kThreads) paged_fork_kernel(const PagesArgs a, bool here) {
  extern __shared__ int32_t sm[];
  int32_t* s_count = sm;             // [B] children
  int32_t* s_first = s_count + a.B;  // [B] the first of them
  __shared__ int s_sums[33];
  Told* told = reinterpret_cast<Told*>(a.ws);
  int32_t* change = a.ws + sizeof(Told) * kCluster / 4;
  int32_t* fresh = change + a.num_pages;
  const int tid = threadIdx.x, me = blockIdx.x * kThreads + tid;
  const int shift = 31 - __clz(a.page), mask = a.page - 1;
  const long long room = static_cast<long long>(a.max_pages) << shift;
  pdl_begin();
  for (int b = tid; b < a.B; b += kThreads) s_count[b] = 0, s_first[b] = 0x7fffffff;
  for (int p = me; p < a.num_pages; p += kAll) change[p] = 0;
  __syncthreads();
  bool bad = false;
  for (int i = tid; i < a.n; i += kThreads) {
    const int p = a.parents[i];
    bad = bad || p < -1 || p >= a.B;
    if (p >= 0 && p < a.B) {
      atomicAdd(s_count + p, 1);
      atomicMin(s_first + p, i);
    }
  }
  for (int b = tid; b < a.B; b += kThreads) bad = bad || a.lens[b] < 0 || a.lens[b] > room;
  bad = __syncthreads_or(bad);
  const int head = a.free_head[0];
  int need = 0;
  if (!bad) {  // every CTA for itself: the children that copy, and their places in the free list
    for (int i0 = 0; i0 < a.n; i0 += kThreads) {
      const int i = i0 + tid, p = i < a.n ? a.parents[i] : -1, len = p < 0 ? 0 : a.lens[p];
      bool copies = false;
      if ((len & mask) != 0) {
        const int pid = a.table[static_cast<size_t>(p) * a.max_pages + (len >> shift)];
        if (pid < 0 || pid >= a.num_pages)
          bad = true;
        else
          copies = s_first[p] != i || a.extra[pid] != 0;
      }
      int total;
      const int at = head + need + block_scan(copies ? 1 : 0, s_sums, total);
      if (i < a.n && blockIdx.x == 0) {
        int pid = -1;
        if (copies && at >= 0 && at < a.n_free) {
          pid = a.free_pages[at];
          bad = bad || pid < 0 || pid >= a.num_pages;
        }
        fresh[i] = pid;
      }
      need += total;
    }
    bad = __syncthreads_or(bad) || head < 0 || head > a.n_free || need > a.n_free - head;
  }
  cluster_sync();  // the changes are zero
  if (!bad) {
    for_pages(a, [&](int b, int j, int pid, int len) {
      if (pid < 0 || pid >= a.num_pages) {
        bad = true;
        return;
      }
      const int c = s_count[b], d = j < (len >> shift) ? c - 1 : c > 0 && a.extra[pid] == 0 ? 0 : -1;
      if (d != 0) atomicAdd(change + pid, d);
    });
  }
  bad = __syncthreads_or(bad);
  cluster_sync();
  // pages without holders: each CTA looks at its part of the cache
  const int part = (a.num_pages + kCluster - 1) / kCluster;
  const int p0 = min(a.num_pages, part * static_cast<int>(blockIdx.x)), p1 = min(a.num_pages, p0 + part);
  int mine = 0;
  for (int p = p0 + tid; p < p1; p += kThreads) {
    const int d = __ldcg(change + p), holders = a.extra[p] + 1 + d;
    bad = bad || (d < 0 && holders < 0);
    mine += d < 0 && holders == 0;
  }
  bad = __syncthreads_or(bad);
  int freed_here;
  block_scan(mine, s_sums, freed_here);
  if (tid == 0) told[blockIdx.x] = {bad ? 1 : 0, freed_here, 0, 0};
  cluster_sync();
  int freed = 0, before = 0;
#pragma unroll
  for (int c = 0; c < kCluster; ++c) {
    const int x = __ldcg(&told[c].a);
    bad = bad || __ldcg(&told[c].bad) != 0;
    if (c < static_cast<int>(blockIdx.x)) before += x;
    freed += x;
  }
  const int head_out = head + need - freed;
  bad = bad || head_out < 0;
  if (me == 0) {
    told[0].b = bad;  // for the launch behind this one
    if (bad)
      atomicOr(a.status, DEV_BOUNDS);
    else
      a.head_out[0] = head_out;
  }
  for (int i = me; i < a.n; i += kAll) {
    const int p = bad ? -1 : a.parents[i], len = p < 0 ? 0 : a.lens[p], to = bad ? -1 : __ldcg(fresh + i);
    if (!bad) a.lens_out[i] = len;
    a.moves[3 * i] = to < 0 ? -1 : a.table[static_cast<size_t>(p) * a.max_pages + (len >> shift)];
    a.moves[3 * i + 1] = to;
    a.moves[3 * i + 2] = to < 0 ? 0 : len & mask;
  }
  if (bad) return;  // nothing is taken
  if (here) write_rows(a, fresh, blockIdx.x * kWarps + warp_id(), kCluster * kWarps);
  // the free list: what is freed, ascending, in front of what was free
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
  if (reinterpret_cast<const Told*>(a.ws)[0].b) return;
  write_rows(a, a.ws + sizeof(Told) * kCluster / 4 + a.num_pages, blockIdx.x * 8 + warp_id(), gridDim.x * 8);
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

// Workspace: Told [kCluster], tokens in each page [num_pages], the pages' new numbers [num_pages].
__global__ void __cluster_dims__(kCluster) __launch_bounds__(kThreads) paged_compact_kernel(const PagesArgs a, bool here) {
  __shared__ int s_sums[33];
  Told* told = reinterpret_cast<Told*>(a.ws);
  int32_t* fill = a.ws + sizeof(Told) * kCluster / 4;
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
  if (tid == 0) told[blockIdx.x] = {bad ? 1 : 0, own, 0, 0};
  cluster_sync();
  int used = 0, before = 0;  // U, and of these in front of this CTA's part
#pragma unroll
  for (int c = 0; c < kCluster; ++c) {
    const int x = __ldcg(&told[c].a);
    bad = bad || __ldcg(&told[c].bad) != 0;
    if (c < static_cast<int>(blockIdx.x)) before += x;
    used += x;
  }
  const int head_out = a.n_free - (a.num_pages - used);
  bad = bad || head_out < 0;
  const int in_front = count(used);
  if (tid == 0) told[blockIdx.x].b = in_front;
  cluster_sync();
  int moves = used;  // M: the free pages among the first U
#pragma unroll
  for (int c = 0; c < kCluster; ++c) moves -= __ldcg(&told[c].b);
  moves = bad ? 0 : min(moves, a.n);
  if (me == 0) {
    told[0].c = bad;  // for the launch behind this one
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
  if (reinterpret_cast<const Told*>(a.ws)[0].c) return;
  renumber_rows(a, a.ws + sizeof(Told) * kCluster / 4 + a.num_pages, blockIdx.x * 8 + warp_id(), gridDim.x * 8);
}

// ------------------------------------------------------------------ copies

// A unit is one of the two caches of a move (and its page's mean, with the first); a block looks
// kCopyThreads of its units over at once, since most moves of a call may be none.  Bound: HBM.
constexpr int kCopyThreads = 256;
__global__ void __launch_bounds__(kCopyThreads) paged_page_copy_kernel(const CopyArgs a) {
  __shared__ int s_todo[kCopyThreads];
  __shared__ int s_count;
  pdl_begin();
  const int tid = threadIdx.x;
  const long long units = 2LL * a.parts * a.n;
  for (long long u0 = blockIdx.x; u0 < units; u0 += static_cast<long long>(kCopyThreads) * gridDim.x) {
    __syncthreads();
    if (tid == 0) s_count = 0;
    __syncthreads();
    const long long mine = u0 + static_cast<long long>(tid) * gridDim.x;
    if (mine < units) {
      const int32_t* m = a.moves + 3 * (mine / (2 * a.parts));
      if (m[0] >= 0) s_todo[atomicAdd(&s_count, 1)] = tid;
    }
    __syncthreads();
    for (int k = 0; k < s_count; ++k) {
      const long long unit = u0 + static_cast<long long>(s_todo[k]) * gridDim.x;
      const int32_t* m = a.moves + 3 * (unit / (2 * a.parts));
      const int which = static_cast<int>(unit % (2 * a.parts)), cache = which / a.parts, piece = which % a.parts;
      const int from = m[0], to = m[1], rows = m[2];
      if (from >= a.num_pages || to < 0 || to >= a.num_pages || rows < 0 || rows > a.page) {
        if (tid == 0) atomicOr(a.status, DEV_BOUNDS);
        continue;
      }
      if (from == to) continue;
      // words of 16 bytes: a head's rows one behind another, heads page * row apart
      const int h0 = static_cast<int>(static_cast<long long>(a.Hkv) * piece / a.parts);
      const int h1 = static_cast<int>(static_cast<long long>(a.Hkv) * (piece + 1) / a.parts);
      const int row = a.row_words, run = rows * row, words = (h1 - h0) * run;
      uint4* base = static_cast<uint4*>(cache ? a.v : a.k);
      const size_t pitch = static_cast<size_t>(a.page) * row;
      const uint4* src = base + (static_cast<size_t>(from) * a.Hkv + h0) * pitch;
      uint4* dst = base + (static_cast<size_t>(to) * a.Hkv + h0) * pitch;
      constexpr int kAtOnce = 8;
      for (int w0 = tid; w0 < words; w0 += kAtOnce * kCopyThreads) {
        uint4 x[kAtOnce];
        int at[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          const int w = w0 + i * kCopyThreads, h = run == static_cast<int>(pitch) ? 0 : w / max(run, 1);
          at[i] = w + h * (static_cast<int>(pitch) - run);
          if (w < words) x[i] = ld_global16(src + at[i]);
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
          if (w0 + i * kCopyThreads < words) dst[at[i]] = x[i];
      }
      if (a.mean != nullptr && which == 0) {
        const int n = a.Hkv * a.mean_words;
        uint4* mean = static_cast<uint4*>(a.mean);
        for (int w = tid; w < n; w += kCopyThreads) mean[static_cast<size_t>(to) * n + w] = ld_global16(mean + static_cast<size_t>(from) * n + w);
      }
    }
  }
}

}  // namespace

size_t paged_fork_workspace_bytes(int num_pages) {
  return sizeof(Told) * kCluster + (static_cast<size_t>(num_pages) + 4096) * sizeof(int32_t);
}
size_t paged_compact_workspace_bytes(int num_pages) {
  return sizeof(Told) * kCluster + 2 * static_cast<size_t>(num_pages) * sizeof(int32_t);
}

cudaError_t launch_paged_fork(const PagesArgs& a, cudaStream_t stream) {
  const bool here = static_cast<long long>(a.n) * a.max_pages <= kTableHere;
  cudaError_t e = launch_dependent(paged_fork_kernel, kCluster, kThreads, 2 * a.B * sizeof(int32_t), stream, a, here);
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

cudaError_t launch_paged_copy(CopyArgs a, cudaStream_t stream) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  // pieces of at most about 16 KB, whole heads
  const long long bytes = 16LL * a.Hkv * a.page * a.row_words;
  a.parts = static_cast<int>(std::max(1LL, std::min<long long>(a.Hkv, bytes >> 14)));
  const long long units = 2LL * a.parts * a.n;
  return launch_dependent(paged_page_copy_kernel, static_cast<unsigned>(std::min<long long>(units, 6LL * sms)), kCopyThreads, 0, stream, a);
}

}  // namespace mcs
