// The paged latent cache: what a batch of new tokens looks like to a kernel, and the launchers of the kernels
// that work on it (paged.cu: append, summaries, selection, and the generic attention).
#pragma once

#include <stdint.h>

#include "common.cuh"
#include "mla.h"

namespace mla {

// mla_paged_t by value, with the row widths.
struct PagedView {
  void* cache;              // [num_pages][page][d_c + d_r]
  const int32_t* table;     // row b at b * stride, max_pages entries
  const int64_t* cu_q;      // [B + 1]
  const int64_t* kv_lens;   // [B]
  int64_t num_pages, max_pages, stride, B, total_q;
  int32_t page;
  int32_t n_h, d_c, d_r;
};

// A new token's sequence and position. seq < 0: a row behind the last sequence (left as it was);
// pos < 0: a token of a sequence that fails the checks (an empty row).
struct PagedToken {
  int32_t seq;
  int64_t pos;
};

// (Called by whole warps with one t: the lanes look at 32 entries of cu_q at a time, one trip to L2 where a bisection
// takes log2(B) one after the other; it only narrows long lists down.)
__device__ __forceinline__ PagedToken paged_token(const PagedView& v, int64_t t) {
  PagedToken r;
  r.seq = -1;
  r.pos = -1;
  const int lane = threadIdx.x & 31;
  int64_t lo = 0, hi = v.B;           // the last entry <= t is in [lo, hi]
  while (hi - lo >= 256) {
    const int64_t mid = (lo + hi) >> 1;
    if (v.cu_q[mid] <= t) lo = mid; else hi = mid;
  }
  const int64_t end = v.cu_q[v.B];
  int64_t b = lo;
#pragma unroll 4
  for (int64_t i = lo; i <= hi; i += 32) {
    const bool in = i + lane <= hi && v.cu_q[min(i + lane, hi)] <= t;
    const uint32_t m = __ballot_sync(0xffffffffu, in);
    if (m) b = i + 31 - __clz(m);
  }
  if (t >= end) return r;
  b = min(b, v.B - 1);
  const int64_t q0 = v.cu_q[b], n = v.cu_q[b + 1] - q0, len = v.kv_lens[b];
  r.seq = (int32_t)b;
  if (t >= q0 && t - q0 < n && n <= len && len <= v.max_pages * v.page) r.pos = len - n + (t - q0);
  return r;
}

// Page of block g of sequence b, or -1 (flagged) when the table names none of the pool.
__device__ __forceinline__ int64_t paged_page(const PagedView& v, int64_t b, int64_t g, uint32_t* err) {
  const int32_t p = v.table[b * v.stride + g];
  if (p < 0 || p >= v.num_pages) {
    flag_error(err, DEVERR_PAGE);
    return -1;
  }
  return p;
}

// The checks of a batch's sequences, by the threads of one block.
__device__ inline void paged_check(const PagedView& v, uint32_t* err) {
  for (int64_t b = threadIdx.x; b < v.B; b += blockDim.x) {
    const int64_t q0 = v.cu_q[b], q1 = v.cu_q[b + 1], len = v.kv_lens[b];
    if ((b == 0 && q0 != 0) || q1 < q0) flag_error(err, DEVERR_CU_SEQLENS);
    if (len < 0 || q1 - q0 > len) flag_error(err, DEVERR_SHORT_SEQ);
    if (q1 > q0 && len > v.max_pages * v.page) flag_error(err, DEVERR_PAGE);
  }
  if (threadIdx.x == 0 && v.cu_q[v.B] > v.total_q) flag_error(err, DEVERR_TOTAL);
}

// A token's list of chosen blocks: its entries before the first -1. Every thread of the block calls this;
// n rows of the concatenated blocks are at or before pos (only the token's own block, the last one if it is
// chosen, can be partly behind it). A list that does not ascend or passes the own block is flagged: n = 0.
// scratch: 2 ints of shared memory.
__device__ inline int64_t paged_list_rows(const int32_t* list, int32_t top_k, int64_t pos, int32_t page, int* scratch,
                                          uint32_t* err) {
  if (threadIdx.x == 0) {
    scratch[0] = top_k;   // first -1
    scratch[1] = 0;       // faults
  }
  __syncthreads();
  for (int i = threadIdx.x; i < top_k; i += blockDim.x)
    if (list[i] < 0) atomicMin(&scratch[0], i);
  __syncthreads();
  const int n = scratch[0];
  for (int i = threadIdx.x; i < n; i += blockDim.x)
    if (list[i] > pos / page || (i > 0 && list[i] <= list[i - 1])) atomicOr(&scratch[1], 1);
  __syncthreads();
  const bool bad = scratch[1] != 0;
  const int last = n > 0 ? list[n - 1] : -1;
  __syncthreads();
  if (bad) {
    if (threadIdx.x == 0) flag_error(err, DEVERR_BLOCKS);
    return 0;
  }
  if (n == 0) return 0;
  return (int64_t)(n - 1) * page + (last == pos / page ? pos % page + 1 : page);
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// Programmatic dependent launch: the next kernel of the chain may start its prologue; this one waits for the kernel
// before it (and with it all earlier ones) to be complete and visible.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launches a kernel of the chain behind the one before it: its blocks may start early and wait in
// wait_for_previous(), so that launch latency and prologue overlap the kernel before.
template <typename... Params, typename... Args>
cudaError_t launch_next(void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  note_launch();
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

size_t summary_pitch(int32_t d_c, int32_t d_r);   // bytes of a summary row

cudaError_t paged_append(const PagedView& v, bool bf16, const void* kv, int64_t kv_stride, const void* q_rope,
                         void* q_out, void* summaries, const LayerOpts& o, const RopeTable& rope, uint32_t* err,
                         cudaStream_t st);

// o_lat and lse of the new tokens in fp32 by CUDA cores, over all rows (blocks == nullptr) or the listed blocks.
cudaError_t paged_attention_simt(const PagedView& v, const void* q_abs, const void* q_rope,
                                 const int32_t* blocks, int32_t top_k, float scale, void* o_lat, float* lse,
                                 uint32_t* err, cudaStream_t st);

size_t paged_select_bytes(bool bf16, int32_t n_h, int32_t d_c, int32_t d_r, int64_t total_q, int64_t max_pages);
cudaError_t paged_select(const PagedView& v, bool bf16, const void* q_abs, const void* q_rope, const void* summaries,
                         int32_t top_k, int32_t n_first, int32_t n_last, int32_t* blocks, void* ws, int num_sms,
                         uint32_t* err, cudaStream_t st);

}  // namespace mla
