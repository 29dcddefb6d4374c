// RMS norm of each head of q and k and the rotation by position, one pass, and
// the gradients of both.
//
//   r = 1 / sqrt(mean(x^2) + eps), y = x r w,
//   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)
//
// D/8 threads hold a row (one head of one token), 8 values each: the mean is a
// shuffle sum over them, the rotation's partner is in the same thread
// (interleaved pairs) or rot/16 threads away (split pairs).  A warp keeps one
// token, so that its angles are loaded once for a chunk of heads, and the warps
// of a block take consecutive tokens, so that a head's rows of a
// [B, H, N, D] output are written next to each other.
#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace mcs {
namespace {

constexpr int kRopeWarps = 8;
constexpr int kRopeThreads = 32 * kRopeWarps;
constexpr int kRopeHeads = 8;   // heads of one token a warp takes
constexpr int kGradBlocks = 1024;  // partial sums of the weight gradients

// 16 bytes that may be overwritten later by this thread (in-place calls).
__device__ __forceinline__ uint4 ld_row16(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ void unpack8(uint4 x, float* f) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                    pack_bf16(f[6], f[7]));
}

// A thread's angles: cs[i], sn[i] for its values 8l + i (split pairs), or
// for its pairs i < 4 (interleaved).
struct Angles {
  float cs[8], sn[8];
};

__device__ __forceinline__ void load_angles(Angles& g, const RopeArgs& a, int pos, int l) {
  if (8 * l >= a.rot) return;
  const size_t row = static_cast<size_t>(pos) * (a.rot / 2);
  if (a.interleaved) {
    *reinterpret_cast<float4*>(g.cs) = *reinterpret_cast<const float4*>(a.cos_table + row + 4 * l);
    *reinterpret_cast<float4*>(g.sn) = *reinterpret_cast<const float4*>(a.sin_table + row + 4 * l);
  } else {
    const int i = 8 * l < a.rot / 2 ? 8 * l : 8 * l - a.rot / 2;
#pragma unroll
    for (int k = 0; k < 8; k += 4) {
      *reinterpret_cast<float4*>(g.cs + k) =
          *reinterpret_cast<const float4*>(a.cos_table + row + i + k);
      *reinterpret_cast<float4*>(g.sn + k) =
          *reinterpret_cast<const float4*>(a.sin_table + row + i + k);
    }
  }
}

// Rotates the row's values (sign = 1) or rotates them back (sign = -1).  All
// lanes of the warp call.
template <int LANES>
__device__ __forceinline__ void rotate(float* y, const Angles& g, const RopeArgs& a, int l,
                                       float sign) {
  if (a.rot == 0) return;
  if (a.interleaved) {
    if (8 * l < a.rot) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = y[2 * i], q = y[2 * i + 1], s = sign * g.sn[i];
        y[2 * i] = p * g.cs[i] - q * s;
        y[2 * i + 1] = q * g.cs[i] + p * s;
      }
    }
    return;
  }
  const int half = a.rot / 16;  // threads that hold the first halves
  const bool first = l < half;
  const int from = l < half ? l + half : (l < 2 * half ? l - half : l);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float other = __shfl_sync(0xffffffffu, y[i], from, LANES);
    if (8 * l < a.rot) {
      const float s = sign * g.sn[i];
      y[i] = y[i] * g.cs[i] + (first ? -other : other) * s;
    }
  }
}

template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The token's position, or -1 where its rows stay as they are.
__device__ __forceinline__ int position_of(const RopeArgs& a, long long token) {
  const int pos = a.positions ? a.positions[token] : static_cast<int>(token % a.N);
  if (a.rot > 0 && pos >= a.table_rows) {
    atomicOr(a.status, DEV_BOUNDS);
    return -1;
  }
  return pos;
}

// Offset of (token, head h of H) in the [B, H, N, D] or [B, N, H, D] tensors.
__device__ __forceinline__ size_t out_row(const RopeArgs& a, long long token, int h, int H) {
  if (a.layout == MCS_LAYOUT_BNHD) return (static_cast<size_t>(token) * H + h) * a.D;
  const long long b = token / a.N, n = token % a.N;
  return ((static_cast<size_t>(b) * H + h) * a.N + n) * a.D;
}

template <int D>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(const RopeArgs a, int chunks_q,
                                                                 int chunks) {
  constexpr int LANES = D / 8, ROWS = 32 / LANES;  // rows a warp holds at a time
  const int chunk = blockIdx.x % chunks;
  const long long token =
      static_cast<long long>(blockIdx.x / chunks) * kRopeWarps + warp_id();
  if (token >= static_cast<long long>(a.B) * a.N) return;
  const int pos = position_of(a, token);
  if (pos < 0) return;
  const bool is_q = chunk < chunks_q;
  const int H = is_q ? a.Hq : a.Hkv, h0 = (is_q ? chunk : chunk - chunks_q) * kRopeHeads;
  const int l = lane_id() % LANES, r = lane_id() / LANES;
  const __nv_bfloat16* src = (is_q ? a.q : a.k) + token * (is_q ? a.q_stride : a.k_stride);
  __nv_bfloat16* dst = is_q ? a.q_out : a.k_out;
  const float* wp = is_q ? a.wq : a.wk;
  uint4 x[kRopeHeads / ROWS];
#pragma unroll
  for (int i = 0; i < kRopeHeads / ROWS; ++i) {
    const int h = h0 + i * ROWS + r;
    x[i] = h < H ? ld_row16(src + h * D + 8 * l) : make_uint4(0, 0, 0, 0);
  }
  Angles g;
  load_angles(g, a, pos, l);
  float w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = wp ? wp[8 * l + i] : 1.f;
#pragma unroll
  for (int i = 0; i < kRopeHeads / ROWS; ++i) {
    float y[8], ss = 0;
    unpack8(x[i], y);
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = fmaf(y[k], y[k], ss);
    const float rr = rsqrtf(row_sum<LANES>(ss) * (1.f / D) + a.eps);
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = y[k] * rr * w[k];
    rotate<LANES>(y, g, a, l, 1.f);
    const int h = h0 + i * ROWS + r;
    if (h < H) *reinterpret_cast<uint4*>(dst + out_row(a, token, h, H) + 8 * l) = pack8(y);
  }
}

// Backward: units of (8 tokens, 8 heads) as above; a block takes every
// gridDim-th unit of q (blocks below blocks_q) or of k and keeps the weight
// gradient of its units in registers, one partial row per block at the end.
template <int D>
__global__ void __launch_bounds__(kRopeThreads)
    norm_rope_backward_kernel(const RopeArgs a, int blocks_q, int blocks_k) {
  constexpr int LANES = D / 8, ROWS = 32 / LANES;
  const bool is_q = static_cast<int>(blockIdx.x) < blocks_q;
  const int H = is_q ? a.Hq : a.Hkv, chunks = (H + kRopeHeads - 1) / kRopeHeads;
  const int block = is_q ? blockIdx.x : blockIdx.x - blocks_q, blocks = is_q ? blocks_q : blocks_k;
  const long long tokens = static_cast<long long>(a.B) * a.N;
  const long long units = (tokens + kRopeWarps - 1) / kRopeWarps * chunks;
  const int l = lane_id() % LANES, r = lane_id() / LANES;
  const __nv_bfloat16* xs = is_q ? a.q : a.k;
  const __nv_bfloat16* dys = is_q ? a.dq_out : a.dk_out;
  __nv_bfloat16* dxs = is_q ? a.q_out : a.k_out;
  const long long stride = is_q ? a.q_stride : a.k_stride;
  const float* wp = is_q ? a.wq : a.wk;
  float w[8], dw[8] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = wp ? wp[8 * l + i] : 1.f;
  for (long long u = block; u < units; u += blocks) {
    const long long token = u / chunks * kRopeWarps + warp_id();
    const int h0 = static_cast<int>(u % chunks) * kRopeHeads;
    if (token >= tokens) continue;  // whole warps
    const int pos = position_of(a, token);
    if (pos < 0) continue;
    uint4 x[kRopeHeads / ROWS], dy[kRopeHeads / ROWS];
#pragma unroll
    for (int i = 0; i < kRopeHeads / ROWS; ++i) {
      const int h = h0 + i * ROWS + r;
      x[i] = h < H ? ld_row16(xs + token * stride + h * D + 8 * l) : make_uint4(0, 0, 0, 0);
      dy[i] = h < H ? ld_row16(dys + out_row(a, token, h, H) + 8 * l) : make_uint4(0, 0, 0, 0);
    }
    Angles ang;
    load_angles(ang, a, pos, l);
#pragma unroll
    for (int i = 0; i < kRopeHeads / ROWS; ++i) {
      float xh[8], g[8], ss = 0, dot = 0;
      unpack8(x[i], xh);
      unpack8(dy[i], g);
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(xh[k], xh[k], ss);
      const float rr = rsqrtf(row_sum<LANES>(ss) * (1.f / D) + a.eps);
      rotate<LANES>(g, ang, a, l, -1.f);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        xh[k] *= rr;
        dw[k] = fmaf(g[k], xh[k], dw[k]);
        g[k] *= w[k];
        dot = fmaf(g[k], xh[k], dot);
      }
      dot = row_sum<LANES>(dot) * (1.f / D);
#pragma unroll
      for (int k = 0; k < 8; ++k) g[k] = rr * (g[k] - xh[k] * dot);
      const int h = h0 + i * ROWS + r;
      if (h < H) *reinterpret_cast<uint4*>(dxs + token * stride + h * D + 8 * l) = pack8(g);
    }
  }
  __shared__ float part[kRopeWarps * ROWS][D];
#pragma unroll
  for (int k = 0; k < 8; ++k) part[warp_id() * ROWS + r][8 * l + k] = dw[k];
  __syncthreads();
  if (threadIdx.x < D) {
    float s = 0;
    for (int i = 0; i < kRopeWarps * ROWS; ++i) s += part[i][threadIdx.x];
    a.ws[static_cast<size_t>(blockIdx.x) * D + threadIdx.x] = s;
  }
}

// dw = sum of the partial rows [first, first + n), block 0 for q, 1 for k.
template <int D>
__global__ void __launch_bounds__(1024) weight_grad_kernel(const RopeArgs a, int blocks_q,
                                                           int blocks_k) {
  const bool is_q = blockIdx.x == 0;
  float* out = is_q ? a.dwq : a.dwk;
  if (out == nullptr) return;
  const int first = is_q ? 0 : blocks_q, n = is_q ? blocks_q : blocks_k;
  const int d = threadIdx.x % D, part = threadIdx.x / D, parts = 1024 / D;
  float s = 0;
  for (int i = part; i < n; i += parts) s += a.ws[static_cast<size_t>(first + i) * D + d];
  __shared__ float sums[1024];
  sums[threadIdx.x] = s;
  __syncthreads();
  if (part == 0) {
    for (int i = 1; i < parts; ++i) s += sums[i * D + d];
    out[d] = s;
  }
}

}  // namespace

size_t norm_rope_backward_workspace_bytes(int D) {
  return static_cast<size_t>(kGradBlocks) * D * sizeof(float);
}

cudaError_t launch_norm_rope(const RopeArgs& a, cudaStream_t stream) {
  const int cq = (a.Hq + kRopeHeads - 1) / kRopeHeads, ck = (a.Hkv + kRopeHeads - 1) / kRopeHeads;
  const long long tiles = (static_cast<long long>(a.B) * a.N + kRopeWarps - 1) / kRopeWarps;
  const unsigned blocks = static_cast<unsigned>(tiles * (cq + ck));
  if (a.D == 128) norm_rope_kernel<128><<<blocks, kRopeThreads, 0, stream>>>(a, cq, cq + ck);
  else norm_rope_kernel<64><<<blocks, kRopeThreads, 0, stream>>>(a, cq, cq + ck);
  return cudaGetLastError();
}

cudaError_t launch_norm_rope_backward(const RopeArgs& a, cudaStream_t stream) {
  const int cq = (a.Hq + kRopeHeads - 1) / kRopeHeads, ck = (a.Hkv + kRopeHeads - 1) / kRopeHeads;
  const long long tiles = (static_cast<long long>(a.B) * a.N + kRopeWarps - 1) / kRopeWarps;
  // the partial rows are shared between q and k by their work
  const long long share = static_cast<long long>(kGradBlocks) * cq / (cq + ck);
  const int limit_q = static_cast<int>(std::max<long long>(1, ck ? std::min<long long>(share, kGradBlocks - 1) : kGradBlocks));
  const int bq = static_cast<int>(std::min<long long>(tiles * cq, limit_q));
  const int bk = static_cast<int>(std::min<long long>(tiles * ck, kGradBlocks - limit_q));
  if (a.D == 128) norm_rope_backward_kernel<128><<<bq + bk, kRopeThreads, 0, stream>>>(a, bq, bk);
  else norm_rope_backward_kernel<64><<<bq + bk, kRopeThreads, 0, stream>>>(a, bq, bk);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (a.dwq == nullptr && a.dwk == nullptr)) return e;
  if (a.D == 128) weight_grad_kernel<128><<<a.Hkv ? 2 : 1, 1024, 0, stream>>>(a, bq, bk);
  else weight_grad_kernel<64><<<a.Hkv ? 2 : 1, 1024, 0, stream>>>(a, bq, bk);
  return cudaGetLastError();
}

}  // namespace mcs
