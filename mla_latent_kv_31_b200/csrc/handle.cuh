// The handle behind the C ABI and the host helpers that its entry points share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "common.cuh"
#include "mla.h"

struct mla_handle {
  mla_dims_t dims;
  mla_dtype_t dtype;
  int device;
  mla_weights_t w;
  bool has_weights;
  uint32_t* d_err;         // device error word (sticky until mla_sync_status)
  uint32_t last_err_bits;  // last word read by mla_sync_status
  int num_sms;
  mla::LayerOpts opts;     // RMSNorm gains and the RoPE (plain or YaRN)
  mla::RopeTable theta;    // the RoPE's frequencies and factor, for the calls that rotate on their own
};

namespace mla {

// The handle's RoPE frequencies, computed once on the host (kRopeTablePairs covers d_r <= 128; wider
// blocks compute them on the device).
inline void fill_theta(mla_handle* h) {
  for (int m = 0; m < kRopeTablePairs && m < h->dims.d_r / 2; ++m)
    h->theta.theta[m] = rope_theta(h->opts.rope, m, h->dims.d_r);
  h->theta.mul = rope_mul(h->opts.rope);
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t elem_size(const mla_handle* h) { return h->dtype == MLA_BF16 ? 2 : 4; }

// BF16 handles run on the tcgen05/TMA kernels; FP32 handles on the generic CUDA-core kernels.
inline bool tc_dims(const mla_handle* h) { return h->dtype == MLA_BF16; }

// Makes the handle's device current for the life of the guard and restores the caller's device
// afterwards, so that no entry point changes the calling thread's current device.
struct DeviceGuard {
  int prev = -1;
  bool ok = false;
  explicit DeviceGuard(int device) {
    if (cudaGetDevice(&prev) != cudaSuccess) return;
    ok = prev == device || cudaSetDevice(device) == cudaSuccess;
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
  }
};

inline mla_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA; }

#define MLA_TRY(expr)                              \
  do {                                             \
    cudaError_t _e = (expr);                       \
    if (_e != cudaSuccess) return MLA_ERR_CUDA;    \
  } while (0)

// Makes the handle ready for launches on first use: the error word, zeroed and waited for (on a stream of its own, which
// waits for no other work), and the SM count, published together. Calls of several threads may be the first ones; a
// failure leaves the handle as it was. The caller holds a DeviceGuard for h->device.
inline mla_status_t ensure_device(mla_handle* h) {
  static std::mutex mu;
  std::lock_guard<std::mutex> lock(mu);
  if (h->d_err) return MLA_OK;
  int sms = 0;
  MLA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, h->device));
  uint32_t* word = nullptr;
  MLA_TRY(cudaMalloc(&word, sizeof(uint32_t)));
  cudaStream_t st = nullptr;
  cudaError_t e = cudaStreamCreateWithFlags(&st, cudaStreamNonBlocking);
  if (e == cudaSuccess) {
    e = cudaMemsetAsync(word, 0, sizeof(uint32_t), st);
    const cudaError_t s = cudaStreamSynchronize(st);
    if (e == cudaSuccess) e = s;
    cudaStreamDestroy(st);
  }
  if (e != cudaSuccess) {
    cudaFree(word);
    return MLA_ERR_CUDA;
  }
  h->num_sms = sms;
  h->d_err = word;
  return MLA_OK;
}

// Waits for the stream, then reads and clears the error word. The clearing is waited for too (cudaMemset is asynchronous):
// a launch on any stream after it finds the word at zero, and what it flags stays.
inline cudaError_t take_error_bits(mla_handle* h, cudaStream_t stream, uint32_t* bits) {
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e == cudaSuccess) e = cudaMemcpy(bits, h->d_err, sizeof(uint32_t), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaMemset(h->d_err, 0, sizeof(uint32_t));
  if (e == cudaSuccess) e = cudaStreamSynchronize(cudaStreamLegacy);
  return e;
}

}  // namespace mla
