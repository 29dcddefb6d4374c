// Attention of one token per sequence over a paged cache.
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"

namespace mcs {
namespace {

constexpr int kDecThreads = 256;

__device__ __forceinline__ float load_value(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load_value(const uint8_t* p) {
  uint32_t lo, hi;
  e4m3x4_to_f16x4(*p, lo, hi);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(lo & 0xFFFFu)));
}

// One CTA per query head: each warp runs over every eighth key with a running
// maximum and sum, then the warps join.
template <int D, typename T>
__global__ void __launch_bounds__(kDecThreads) paged_decode_kernel(const DecodeArgs a) {
  constexpr int V = D / 32;
  const int b = blockIdx.x / a.Hq, hq = blockIdx.x % a.Hq, group = a.Hq / a.Hkv, h = hq / group;
  const int lane = lane_id(), w = warp_id();
  int len = a.lens[b];
  if (len < 0 || static_cast<long long>(len) > static_cast<long long>(a.max_pages) * a.page) {
    if (threadIdx.x == 0) atomicOr(a.status, DEV_BOUNDS);
    len = 0;
  }
  const int n = (len + a.page - 1) / a.page;
  const int pages = a.sel ? min(n, a.select) : n;
  float q[V], o[V] = {}, m = -INFINITY, l = 0;
  for (int i = 0; i < V; ++i) {
    q[i] = __bfloat162float(a.q[static_cast<size_t>(b) * a.q_stride + hq * D + lane * V + i]);
    if (sizeof(T) == 1) q[i] = fminf(fmaxf(q[i], -65504.f), 65504.f);
  }
  for (long long r = w; r < static_cast<long long>(pages) * a.page; r += kDecThreads / 32) {
    int j = static_cast<int>(r / a.page);
    if (a.sel) {
      j = a.sel[(static_cast<size_t>(b) * a.Hkv + h) * a.select + j];
      if (j == -1) continue;
      if (j < -1 || j >= n) {
        if (lane == 0) atomicOr(a.status, DEV_BOUNDS);
        continue;
      }
    }
    const int off = static_cast<int>(r % a.page);
    if (static_cast<long long>(j) * a.page + off >= len) continue;
    const int pid = a.table[static_cast<size_t>(b) * a.max_pages + j];
    if (pid < 0 || pid >= a.num_pages) {
      if (lane == 0) atomicOr(a.status, DEV_BOUNDS);
      continue;
    }
    const size_t row = ((static_cast<size_t>(pid) * a.Hkv + h) * a.page + off) * D + lane * V;
    float s = 0;
    for (int i = 0; i < V; ++i) s += q[i] * load_value(static_cast<const T*>(a.k) + row + i);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= a.scale_log2;
    const float mn = fmaxf(m, s), c = exp2f(m - mn), p = exp2f(s - mn);
    l = l * c + p;
    for (int i = 0; i < V; ++i)
      o[i] = o[i] * c + p * load_value(static_cast<const T*>(a.v) + row + i);
    m = mn;
  }
  __shared__ float s_m[8], s_l[8], s_o[8][D];
  if (lane == 0) s_m[w] = m, s_l[w] = l;
  for (int i = 0; i < V; ++i) s_o[w][lane * V + i] = o[i];
  __syncthreads();
  if (threadIdx.x < D) {
    float top = -INFINITY, sum = 0, acc = 0;
    for (int i = 0; i < 8; ++i) top = fmaxf(top, s_m[i]);
    for (int i = 0; i < 8; ++i) {
      const float c = s_m[i] == -INFINITY ? 0.f : exp2f(s_m[i] - top);
      sum += s_l[i] * c;
      acc += s_o[i][threadIdx.x] * c;
    }
    a.out[static_cast<size_t>(blockIdx.x) * D + threadIdx.x] =
        __float2bfloat16(sum > 0 ? acc * a.v_scale / sum : 0.f);
    if (a.lse && threadIdx.x == 0)
      a.lse[blockIdx.x] = sum > 0 ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
  }
}

}  // namespace

size_t paged_decode_workspace_bytes(int) { return 256; }

cudaError_t launch_paged_decode(const DecodeArgs& a, bool e4m3, cudaStream_t stream) {
  const int grid = a.B * a.Hq;
  if (a.D == 128) {
    if (e4m3) paged_decode_kernel<128, uint8_t><<<grid, kDecThreads, 0, stream>>>(a);
    else paged_decode_kernel<128, __nv_bfloat16><<<grid, kDecThreads, 0, stream>>>(a);
  } else {
    if (e4m3) paged_decode_kernel<64, uint8_t><<<grid, kDecThreads, 0, stream>>>(a);
    else paged_decode_kernel<64, __nv_bfloat16><<<grid, kDecThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace mcs
