// C ABI of the paged latent cache (declared in include/mla.h): validation and dispatch.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "handle.cuh"
#include "mla.h"
#include "paged.cuh"
#include "tc_paged.cuh"

namespace mla {
static std::atomic<bool> g_paged_stall{false};
bool take_paged_stall() { return g_paged_stall.exchange(false, std::memory_order_relaxed); }
}  // namespace mla

namespace {

using mla::aligned16;
using mla::cuda_status;
using mla::DeviceGuard;
using mla::elem_size;
using mla::ensure_device;
using mla::PagedView;
using mla::tc_dims;

constexpr int64_t kMaxRows = INT32_MAX;
constexpr int64_t kMaxLen = 1 << 30;         // rows of a sequence: 32-bit key numbers with room for a step
constexpr int64_t kMaxSelectTokens = 65535;  // a grid's second dimension
constexpr int64_t kMaxSeqs = 1 << 20;
constexpr int32_t kMinPage = 16;

// The host checks that every paged call shares; on MLA_OK *v describes the batch.
mla_status_t view_of(const mla_handle_t* h, const mla_paged_t* b, PagedView* v) {
  if (!h || !b) return MLA_ERR_INVALID_ARG;
  if (h->opts.cache_fp8) return MLA_ERR_UNSUPPORTED;
  if (!b->cache || !b->block_table || !b->cu_q || !b->kv_lens || b->B <= 0 || b->total_q <= 0 || b->num_pages <= 0 ||
      b->max_pages <= 0 || b->table_stride < b->max_pages || b->page_size <= 0 || b->page_size % kMinPage != 0)
    return MLA_ERR_INVALID_ARG;
  if (b->num_pages > kMaxRows / b->page_size || b->max_pages > kMaxLen / b->page_size || b->B > kMaxSeqs ||
      b->total_q > kMaxRows / h->dims.n_h)
    return MLA_ERR_INVALID_ARG;
  if (!aligned16(b->cache) || !aligned16(b->block_table) || !aligned16(b->cu_q) || !aligned16(b->kv_lens))
    return MLA_ERR_ALIGNMENT;
  v->cache = b->cache;
  v->table = b->block_table;
  v->cu_q = b->cu_q;
  v->kv_lens = b->kv_lens;
  v->num_pages = b->num_pages;
  v->max_pages = b->max_pages;
  v->stride = b->table_stride;
  v->B = b->B;
  v->total_q = b->total_q;
  v->page = b->page_size;
  v->n_h = h->dims.n_h;
  v->d_c = h->dims.d_c;
  v->d_r = h->dims.d_r;
  return MLA_OK;
}

mla_status_t attention(mla_handle_t* h, const mla_paged_t* batch, const void* q_abs, const void* q_rope,
                       const int32_t* blocks, int32_t top_k, void* o_lat, float* lse, void* ws, size_t ws_bytes,
                       mla_stream_t stream) {
  PagedView v;
  mla_status_t s = view_of(h, batch, &v);
  if (s != MLA_OK) return s;
  if (!q_abs || !q_rope || !o_lat || !lse) return MLA_ERR_INVALID_ARG;
  if (!aligned16(q_abs) || !aligned16(q_rope) || !aligned16(o_lat) || !aligned16(lse) || (ws && !aligned16(ws)))
    return MLA_ERR_ALIGNMENT;
  size_t need = 0;
  s = mla_attn_paged_workspace(h, v.B, v.total_q, &need);
  if (s != MLA_OK) return s;
  if (ws_bytes < need || (need > 0 && !ws)) return MLA_ERR_WORKSPACE;
  DeviceGuard g(h->device);
  if (!g.ok) return MLA_ERR_CUDA;
  if ((s = ensure_device(h)) != MLA_OK) return s;
  const float scale = (float)(1.0 / sqrt((double)(h->dims.d_h + h->dims.d_r)));
  if (tc_dims(h))
    return cuda_status(mla::tc_paged_attention(v, q_abs, q_rope, blocks, top_k, scale, o_lat, lse, ws, h->num_sms,
                                               h->d_err, (cudaStream_t)stream));
  return cuda_status(
      mla::paged_attention_simt(v, q_abs, q_rope, blocks, top_k, scale, o_lat, lse, h->d_err, (cudaStream_t)stream));
}

}  // namespace

extern "C" {

mla_status_t mla_paged_summary_bytes(const mla_handle_t* h, size_t* bytes) {
  if (!h || !bytes) return MLA_ERR_INVALID_ARG;
  if ((h->dims.d_c + h->dims.d_r) % 4) return MLA_ERR_UNSUPPORTED;
  *bytes = mla::summary_pitch(h->dims.d_c, h->dims.d_r);
  return MLA_OK;
}

mla_status_t mla_paged_append(mla_handle_t* h, const mla_paged_t* batch, const void* kv, int64_t kv_stride,
                              const void* q_rope, void* q_out, void* summaries, mla_stream_t stream) {
  PagedView v;
  mla_status_t s = view_of(h, batch, &v);
  if (s != MLA_OK) return s;
  if (!kv || kv_stride < v.d_c + v.d_r || (tc_dims(h) && kv_stride % 8) || (!q_rope) != (!q_out))
    return MLA_ERR_INVALID_ARG;
  if (summaries && (v.d_c + v.d_r) % 4) return MLA_ERR_UNSUPPORTED;
  if (!aligned16(kv) || (q_rope && !aligned16(q_rope)) || (q_out && !aligned16(q_out)) ||
      (summaries && !aligned16(summaries)))
    return MLA_ERR_ALIGNMENT;
  DeviceGuard g(h->device);
  if (!g.ok) return MLA_ERR_CUDA;
  if ((s = ensure_device(h)) != MLA_OK) return s;
  return cuda_status(mla::paged_append(v, tc_dims(h), kv, kv_stride, q_rope, q_out, summaries, h->opts, h->theta,
                                       h->d_err, (cudaStream_t)stream));
}

mla_status_t mla_attn_paged_workspace(const mla_handle_t* h, int64_t B, int64_t total_q, size_t* bytes) {
  if (!h || !bytes || B <= 0 || B > kMaxSeqs || total_q <= 0 || total_q > kMaxRows / h->dims.n_h) return MLA_ERR_INVALID_ARG;
  *bytes = tc_dims(h) ? mla::tc_paged_attention_bytes(total_q) : 0;
  return MLA_OK;
}

mla_status_t mla_attn_paged(mla_handle_t* h, const mla_paged_t* batch, const void* q_abs, const void* q_rope,
                            void* o_lat, float* lse, void* ws, size_t ws_bytes, mla_stream_t stream) {
  return attention(h, batch, q_abs, q_rope, nullptr, 0, o_lat, lse, ws, ws_bytes, stream);
}

mla_status_t mla_attn_paged_sparse(mla_handle_t* h, const mla_paged_t* batch, const void* q_abs, const void* q_rope,
                                   const int32_t* blocks, int32_t top_k, void* o_lat, float* lse, void* ws,
                                   size_t ws_bytes, mla_stream_t stream) {
  if (!blocks || top_k <= 0 || top_k > (1 << 20)) return MLA_ERR_INVALID_ARG;
  if (!aligned16(blocks)) return MLA_ERR_ALIGNMENT;
  return attention(h, batch, q_abs, q_rope, blocks, top_k, o_lat, lse, ws, ws_bytes, stream);
}

mla_status_t mla_paged_select_workspace(const mla_handle_t* h, int64_t total_q, int64_t max_pages, size_t* bytes) {
  if (!h || !bytes || total_q <= 0 || total_q > kMaxSelectTokens || max_pages <= 0 || max_pages > kMaxLen / kMinPage)
    return MLA_ERR_INVALID_ARG;
  *bytes = mla::paged_select_bytes(tc_dims(h), h->dims.n_h, h->dims.d_c, h->dims.d_r, total_q, max_pages);
  return MLA_OK;
}

mla_status_t mla_paged_select(mla_handle_t* h, const mla_paged_t* batch, const void* q_abs, const void* q_rope,
                              const void* summaries, int32_t top_k, int32_t n_first, int32_t n_last, int32_t* blocks,
                              void* ws, size_t ws_bytes, mla_stream_t stream) {
  PagedView v;
  mla_status_t s = view_of(h, batch, &v);
  if (s != MLA_OK) return s;
  if (!q_abs || !q_rope || !summaries || !blocks || !ws || top_k <= 0 || top_k > (1 << 20) || n_first < 0 ||
      n_last < 1 || n_first > top_k - n_last || v.total_q > kMaxSelectTokens)
    return MLA_ERR_INVALID_ARG;
  if ((v.d_c + v.d_r) % 4) return MLA_ERR_UNSUPPORTED;
  if (!aligned16(q_abs) || !aligned16(q_rope) || !aligned16(summaries) || !aligned16(blocks) || !aligned16(ws))
    return MLA_ERR_ALIGNMENT;
  size_t need = 0;
  if ((s = mla_paged_select_workspace(h, v.total_q, v.max_pages, &need)) != MLA_OK) return s;
  if (ws_bytes < need) return MLA_ERR_WORKSPACE;
  DeviceGuard g(h->device);
  if (!g.ok) return MLA_ERR_CUDA;
  if ((s = ensure_device(h)) != MLA_OK) return s;
  return cuda_status(mla::paged_select(v, tc_dims(h), q_abs, q_rope, summaries, top_k, n_first, n_last, blocks, ws,
                                       h->num_sms, h->d_err, (cudaStream_t)stream));
}

void mla_test_arm_paged_stall(void) { mla::g_paged_stall.store(true, std::memory_order_relaxed); }

}  // extern "C"
