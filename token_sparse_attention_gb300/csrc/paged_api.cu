// C-ABI entry points of the paged cache and of the norm with rotation:
// argument checks and dispatch.  Declarations and per-call documentation live
// in include/mcs.h.
#include <math.h>

#include "internal.h"
#include "mcs.h"

namespace {

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool good(const void* p) { return p != nullptr && aligned(p, 16); }
bool good_ints(const void* p) { return p != nullptr && aligned(p, 4); }
bool good_scale(float s) { return s > 0.f && isfinite(s); }

// A token stride: 0 (rows next to each other) or at least a row, whole 16-byte words.
bool good_stride(int s, long long row) { return s == 0 || (s >= row && s % 8 == 0); }

constexpr long long kIntMax = 0x7fffffffLL;
constexpr float kLog2e = 1.4426950408889634f;

// What a product of stored q and k is multiplied by, for powers of two.  Scales whose product
// vanishes stay above zero: the kernels multiply the -inf of masked scores by it, and with the
// smallest float any weight is within 2^-21 of 1.
float scale_log2_of(const mcs_paged* p) {
  const float scale = p->scale > 0.f ? p->scale : 1.0f / sqrtf(static_cast<float>(p->D));
  return fmaxf(scale * (p->kv == MCS_KV_E4M3 ? p->k_scale : 1.f) * kLog2e, 0x1p-149f);
}

mcs_status check_paged(const mcs_paged* p) {
  if (p == nullptr) return MCS_ERR_INVALID_ARG;
  if (p->B < 1 || p->Hkv < 1 || p->Hq < 1 || p->Hq % p->Hkv != 0 || p->num_pages < 1 ||
      p->max_pages < 1)
    return MCS_ERR_INVALID_ARG;
  if (p->D != 64 && p->D != 128) return MCS_ERR_UNSUPPORTED;
  if (p->page != 16 && p->page != 32 && p->page != 64 && p->page != 128) return MCS_ERR_UNSUPPORTED;
  if (p->B > 4096 || static_cast<long long>(p->B) * p->Hq > (1 << 20)) return MCS_ERR_UNSUPPORTED;
  if (static_cast<long long>(p->num_pages) * p->page > kIntMax / p->Hkv) return MCS_ERR_UNSUPPORTED;
  if (static_cast<long long>(p->max_pages) * p->page > kIntMax - 128) return MCS_ERR_UNSUPPORTED;
  if (p->kv != MCS_KV_BF16 && p->kv != MCS_KV_E4M3) return MCS_ERR_INVALID_ARG;
  if (p->kv == MCS_KV_E4M3 && (!good_scale(p->k_scale) || !good_scale(p->v_scale)))
    return MCS_ERR_INVALID_ARG;
  if (!(p->scale >= 0.f) || !isfinite(p->scale) || !isfinite(scale_log2_of(p)))
    return MCS_ERR_INVALID_ARG;
  if (!good_stride(p->q_stride, static_cast<long long>(p->Hq) * p->D) ||
      !good_stride(p->kv_stride, static_cast<long long>(p->Hkv) * p->D))
    return MCS_ERR_INVALID_ARG;
  return MCS_OK;
}

long long q_stride_of(const mcs_paged* p) {
  return p->q_stride ? p->q_stride : static_cast<long long>(p->Hq) * p->D;
}

mcs_status status_word(unsigned** out) {
  const cudaError_t e = mcs::device_status_word(out);
  return e == cudaSuccess ? MCS_OK : mcs::record_cuda_error(e, "cudaGetSymbolAddress(status)");
}

mcs_status finish(cudaError_t e, const char* what) {
  return e == cudaSuccess ? MCS_OK : mcs::record_cuda_error(e, what);
}

mcs_status run_decode(const mcs_paged* p, const void* q, const void* k_cache, const void* v_cache,
                      const int32_t* table, const int32_t* lens, const int32_t* sel, int select,
                      void* out, float* lse, void* ws, size_t ws_bytes, cudaStream_t stream,
                      const char* what) {
  if (!good(q) || !good(k_cache) || !good(v_cache) || !good(out) || !good_ints(table) ||
      !good_ints(lens) || !aligned(lse, 4))
    return MCS_ERR_INVALID_ARG;
  if (!good(ws) || ws_bytes < mcs_paged_decode_workspace(p)) return MCS_ERR_WORKSPACE;
  const bool e4m3 = p->kv == MCS_KV_E4M3;
  mcs::DecodeArgs a{};
  a.B = p->B;
  a.Hq = p->Hq;
  a.Hkv = p->Hkv;
  a.D = p->D;
  a.page = p->page;
  a.num_pages = p->num_pages;
  a.max_pages = p->max_pages;
  a.q_stride = q_stride_of(p);
  a.scale_log2 = scale_log2_of(p);
  a.v_scale = e4m3 ? p->v_scale : 1.f;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = k_cache;
  a.v = v_cache;
  a.table = table;
  a.lens = lens;
  a.sel = sel;
  a.select = select;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.ws = ws;
  mcs_status s = status_word(&a.status);
  if (s != MCS_OK) return s;
  return finish(mcs::launch_paged_decode(a, e4m3, stream), what);
}

mcs_status check_rope(const mcs_rope* p) {
  if (p == nullptr) return MCS_ERR_INVALID_ARG;
  if (p->B < 1 || p->N < 1 || p->Hq < 1 || p->Hkv < 0 || p->table_rows < 0) return MCS_ERR_INVALID_ARG;
  if (p->D != 64 && p->D != 128) return MCS_ERR_UNSUPPORTED;
  if (p->rot < 0 || p->rot > p->D || p->rot % 16 != 0) return MCS_ERR_UNSUPPORTED;
  if ((p->interleaved != 0 && p->interleaved != 1) || !(p->eps >= 0.f) || !isfinite(p->eps))
    return MCS_ERR_INVALID_ARG;
  if (p->layout != MCS_LAYOUT_BHND && p->layout != MCS_LAYOUT_BNHD) return MCS_ERR_INVALID_ARG;
  const long long tokens = static_cast<long long>(p->B) * p->N;
  const long long heads = static_cast<long long>(p->Hq) + p->Hkv;
  if (tokens > kIntMax || heads > kIntMax / tokens || heads > kIntMax / p->D)
    return MCS_ERR_UNSUPPORTED;
  if (!good_stride(p->q_stride, static_cast<long long>(p->Hq) * p->D) ||
      !good_stride(p->k_stride, static_cast<long long>(p->Hkv) * p->D))
    return MCS_ERR_INVALID_ARG;
  return MCS_OK;
}

// The arguments both directions share.
mcs_status rope_args(const mcs_rope* p, const void* q, const void* k, const float* wq,
                     const float* wk, const float* cos_table, const float* sin_table,
                     const int32_t* positions, mcs::RopeArgs* a) {
  if (!good(q) || (p->Hkv > 0 && !good(k)) || !aligned(wq, 4) || !aligned(wk, 4) ||
      !aligned(positions, 4))
    return MCS_ERR_INVALID_ARG;
  if (p->rot > 0) {
    if (!good(cos_table) || !good(sin_table)) return MCS_ERR_INVALID_ARG;
    if (p->table_rows < 1 || (!positions && p->N > p->table_rows)) return MCS_ERR_INVALID_ARG;
  }
  a->B = p->B;
  a->N = p->N;
  a->Hq = p->Hq;
  a->Hkv = p->Hkv;
  a->D = p->D;
  a->rot = p->rot;
  a->interleaved = p->interleaved;
  a->table_rows = p->table_rows;
  a->layout = p->layout;
  a->eps = p->eps;
  a->q_stride = p->q_stride ? p->q_stride : static_cast<long long>(p->Hq) * p->D;
  a->k_stride = p->k_stride ? p->k_stride : static_cast<long long>(p->Hkv) * p->D;
  a->q = static_cast<const __nv_bfloat16*>(q);
  a->k = static_cast<const __nv_bfloat16*>(k);
  a->wq = wq;
  a->wk = wk;
  a->cos_table = cos_table;
  a->sin_table = sin_table;
  a->positions = positions;
  return status_word(&a->status);
}

}  // namespace

extern "C" {

mcs_status mcs_paged_plan(const mcs_paged* p, const int32_t* new_lens, const int32_t* lens,
                          const int32_t* free_pages, int n_free, const int32_t* free_head,
                          int32_t* block_table, int32_t* lens_out, int32_t* head_out,
                          int32_t* cu_new, int32_t* slots, int32_t* positions, int T,
                          cudaStream_t stream) {
  mcs_status s = check_paged(p);
  if (s != MCS_OK) return s;
  if (T < 0 || n_free < 0) return MCS_ERR_INVALID_ARG;
  if (T > (1 << 30) || n_free > (1 << 30)) return MCS_ERR_UNSUPPORTED;
  if (!good_ints(new_lens) || !good_ints(lens) || (n_free > 0 && !good_ints(free_pages)) ||
      !good_ints(free_head) || !good_ints(block_table) || !good_ints(lens_out) ||
      !good_ints(head_out) || !good_ints(cu_new) || (T > 0 && !good_ints(slots)) ||
      !aligned(positions, 4))
    return MCS_ERR_INVALID_ARG;
  mcs::PlanArgs a{};
  a.B = p->B;
  a.page = p->page;
  a.num_pages = p->num_pages;
  a.max_pages = p->max_pages;
  a.n_free = n_free;
  a.T = T;
  a.new_lens = new_lens;
  a.lens = lens;
  a.free_pages = free_pages;
  a.free_head = free_head;
  a.table = block_table;
  a.lens_out = lens_out;
  a.head_out = head_out;
  a.cu_new = cu_new;
  a.slots = slots;
  a.positions = positions;
  if ((s = status_word(&a.status)) != MCS_OK) return s;
  return finish(mcs::launch_paged_plan(a, stream), "paged plan launch");
}

mcs_status mcs_paged_write(const mcs_paged* p, int T, const void* k, const void* v,
                           const int32_t* slots, void* k_cache, void* v_cache, void* k_mean,
                           cudaStream_t stream) {
  mcs_status s = check_paged(p);
  if (s != MCS_OK) return s;
  if (T < 0) return MCS_ERR_INVALID_ARG;
  if (static_cast<long long>(T) > kIntMax / p->Hkv) return MCS_ERR_UNSUPPORTED;
  if (T == 0) return MCS_OK;
  if (!good(k) || !good(v) || !good_ints(slots) || !good(k_cache) || !good(v_cache) ||
      !aligned(k_mean, 16))
    return MCS_ERR_INVALID_ARG;
  mcs::WriteArgs a{};
  a.T = T;
  a.Hkv = p->Hkv;
  a.D = p->D;
  a.page = p->page;
  a.slots_total = static_cast<long long>(p->num_pages) * p->page;
  a.stride = p->kv_stride ? p->kv_stride : static_cast<long long>(p->Hkv) * p->D;
  a.k_scale = p->k_scale;
  a.v_scale = p->v_scale;
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.slots = slots;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_mean = static_cast<__nv_bfloat16*>(k_mean);
  if ((s = status_word(&a.status)) != MCS_OK) return s;
  return finish(mcs::launch_paged_write(a, p->kv == MCS_KV_E4M3, stream), "paged write launch");
}

size_t mcs_paged_decode_workspace(const mcs_paged* p) {
  return check_paged(p) == MCS_OK ? mcs::paged_decode_workspace_bytes(p->D, p->Hq / p->Hkv) : 0;
}

mcs_status mcs_paged_decode(const mcs_paged* p, const void* q, const void* k_cache,
                            const void* v_cache, const int32_t* block_table, const int32_t* lens,
                            void* out, float* lse, void* ws, size_t ws_bytes,
                            cudaStream_t stream) {
  const mcs_status s = check_paged(p);
  if (s != MCS_OK) return s;
  return run_decode(p, q, k_cache, v_cache, block_table, lens, nullptr, 0, out, lse, ws, ws_bytes,
                    stream, "paged decode launch");
}

size_t mcs_paged_select_workspace(const mcs_paged* p) {
  return check_paged(p) == MCS_OK
             ? mcs::paged_select_workspace_bytes(p->B, p->Hkv, p->max_pages)
             : 0;
}

mcs_status mcs_paged_select(const mcs_paged* p, const void* q, const void* k_mean,
                            const int32_t* block_table, const int32_t* lens, int select, int sink,
                            int recent, int32_t* sel, void* ws, size_t ws_bytes,
                            cudaStream_t stream) {
  mcs_status s = check_paged(p);
  if (s != MCS_OK) return s;
  if (select < 1 || sink < 0 || recent < 0 || static_cast<long long>(sink) + recent > select)
    return MCS_ERR_INVALID_ARG;
  if (!good(q) || !good(k_mean) || !good_ints(block_table) || !good_ints(lens) || !good_ints(sel))
    return MCS_ERR_INVALID_ARG;
  if (!good(ws) || ws_bytes < mcs_paged_select_workspace(p)) return MCS_ERR_WORKSPACE;
  mcs::SelectArgs a{};
  a.B = p->B;
  a.Hq = p->Hq;
  a.Hkv = p->Hkv;
  a.D = p->D;
  a.page = p->page;
  a.num_pages = p->num_pages;
  a.max_pages = p->max_pages;
  a.select = select;
  a.sink = sink;
  a.recent = recent;
  a.q_stride = q_stride_of(p);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k_mean = static_cast<const __nv_bfloat16*>(k_mean);
  a.table = block_table;
  a.lens = lens;
  a.sel = sel;
  a.keys = static_cast<uint32_t*>(ws);
  if ((s = status_word(&a.status)) != MCS_OK) return s;
  return finish(mcs::launch_paged_select(a, stream), "paged select launch");
}

mcs_status mcs_paged_decode_sparse(const mcs_paged* p, const void* q, const void* k_cache,
                                   const void* v_cache, const int32_t* block_table,
                                   const int32_t* lens, const int32_t* sel, int select, void* out,
                                   float* lse, void* ws, size_t ws_bytes, cudaStream_t stream) {
  const mcs_status s = check_paged(p);
  if (s != MCS_OK) return s;
  if (select < 1 || !good_ints(sel)) return MCS_ERR_INVALID_ARG;
  return run_decode(p, q, k_cache, v_cache, block_table, lens, sel, select, out, lse, ws, ws_bytes,
                    stream, "paged sparse decode launch");
}

mcs_status mcs_qk_norm_rope(const mcs_rope* p, const void* q, const void* k, const float* wq,
                            const float* wk, const float* cos_table, const float* sin_table,
                            const int32_t* positions, void* q_out, void* k_out,
                            cudaStream_t stream) {
  mcs_status s = check_rope(p);
  if (s != MCS_OK) return s;
  if (!good(q_out) || (p->Hkv > 0 && !good(k_out))) return MCS_ERR_INVALID_ARG;
  mcs::RopeArgs a{};
  if ((s = rope_args(p, q, k, wq, wk, cos_table, sin_table, positions, &a)) != MCS_OK) return s;
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  return finish(mcs::launch_norm_rope(a, stream), "norm and rotation launch");
}

size_t mcs_qk_norm_rope_backward_workspace(const mcs_rope* p) {
  return check_rope(p) == MCS_OK ? mcs::norm_rope_backward_workspace_bytes(p->D) : 0;
}

mcs_status mcs_qk_norm_rope_backward(const mcs_rope* p, const void* dq_out, const void* dk_out,
                                     const void* q, const void* k, const float* wq,
                                     const float* wk, const float* cos_table,
                                     const float* sin_table, const int32_t* positions, void* dq,
                                     void* dk, float* dwq, float* dwk, void* ws, size_t ws_bytes,
                                     cudaStream_t stream) {
  mcs_status s = check_rope(p);
  if (s != MCS_OK) return s;
  if (!good(dq_out) || !good(dq) || (p->Hkv > 0 && (!good(dk_out) || !good(dk))) ||
      !aligned(dwq, 4) || !aligned(dwk, 4))
    return MCS_ERR_INVALID_ARG;
  if (!good(ws) || ws_bytes < mcs_qk_norm_rope_backward_workspace(p)) return MCS_ERR_WORKSPACE;
  mcs::RopeArgs a{};
  if ((s = rope_args(p, q, k, wq, wk, cos_table, sin_table, positions, &a)) != MCS_OK) return s;
  a.q_out = static_cast<__nv_bfloat16*>(dq);
  a.k_out = static_cast<__nv_bfloat16*>(dk);
  a.dq_out = static_cast<const __nv_bfloat16*>(dq_out);
  a.dk_out = static_cast<const __nv_bfloat16*>(dk_out);
  a.dwq = dwq;
  a.dwk = p->Hkv > 0 ? dwk : nullptr;
  a.ws = static_cast<float*>(ws);
  return finish(mcs::launch_norm_rope_backward(a, stream), "norm and rotation backward launch");
}

}  // extern "C"
