// The first call of a handle (ensure_device, csrc/handle.cuh) over a stand-in for the CUDA runtime: no GPU and no
// cudart, host code only. Threads that make it at once all find the handle ready, a failure of any runtime call leaves
// nothing behind, and the next call tries again; reading the error word clears it for good. "ok" and exit status 0 on success. Built and run by
// tests/test_paged_host.py.
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <atomic>
#include <chrono>
#include <thread>
#include <vector>

#include "handle.cuh"

static std::atomic<int> g_words{0}, g_streams{0}, g_mallocs{0}, g_calls{0};
static int g_fail_at = -1;              // the runtime call that fails, counted from the start of a scenario
static std::atomic<void*> g_pending{nullptr};

#ifndef __CUDA_ARCH__                   // (the device pass has definitions of its own)
// A runtime call: slow, so that threads meet inside it; whether it works.
static bool works() {
  std::this_thread::sleep_for(std::chrono::milliseconds(2));
  return g_calls.fetch_add(1) != g_fail_at;
}

#define CALL extern "C" cudaError_t CUDARTAPI
CALL cudaMalloc(void** p, size_t n) {
  if (!works()) return cudaErrorMemoryAllocation;
  ++g_words;
  ++g_mallocs;
  *p = malloc(n);
  memset(*p, 0xa5, n);
  return cudaSuccess;
}
CALL cudaFree(void* p) {
  if (p) --g_words;
  free(p);
  return cudaSuccess;
}
// A memset is asynchronous: the word is zero once its stream has been waited for.
CALL cudaMemset(void* p, int, size_t) {
  if (!works()) return cudaErrorUnknown;
  g_pending = p;
  return cudaSuccess;
}
CALL cudaMemsetAsync(void* p, int, size_t, cudaStream_t) {
  if (!works()) return cudaErrorUnknown;
  g_pending = p;
  return cudaSuccess;
}
CALL cudaStreamCreateWithFlags(cudaStream_t* s, unsigned) {
  if (!works()) return cudaErrorUnknown;
  ++g_streams;
  *s = (cudaStream_t)malloc(1);
  return cudaSuccess;
}
CALL cudaStreamSynchronize(cudaStream_t) {
  if (!works()) return cudaErrorUnknown;
  if (void* p = g_pending.exchange(nullptr)) memset(p, 0, sizeof(uint32_t));
  return cudaSuccess;
}
CALL cudaStreamDestroy(cudaStream_t s) {
  --g_streams;
  free(s);
  return cudaSuccess;
}
CALL cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) {
  if (!works()) return cudaErrorUnknown;
  *v = 148;
  return cudaSuccess;
}
CALL cudaMemcpy(void* to, const void* from, size_t n, cudaMemcpyKind) {
  if (!works()) return cudaErrorUnknown;
  memcpy(to, from, n);
  return cudaSuccess;
}
CALL cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
CALL cudaSetDevice(int) { return cudaSuccess; }
// What the compiler's start-up code calls for a program with device code; this one launches none.
extern "C" void** __cudaRegisterFatBinary(void*) { return nullptr; }
extern "C" void __cudaRegisterFatBinaryEnd(void**) {}
extern "C" void __cudaUnregisterFatBinary(void**) {}
#endif

#define CHECK(n, cond)                              \
  do {                                              \
    if (!(cond)) {                                  \
      fprintf(stderr, "check %d failed\n", (n));    \
      exit(n);                                      \
    }                                               \
  } while (0)

static bool ready(const mla_handle& h) { return h.d_err && *h.d_err == 0 && h.num_sms == 148; }

int main() {
  // threads that are first at once
  for (int round = 0; round < 10; ++round) {
    mla_handle h;
    memset(&h, 0, sizeof(h));
    g_mallocs = 0;
    std::atomic<int> go{0}, wrong{0};
    std::vector<std::thread> threads;
    for (int t = 0; t < 8; ++t)
      threads.emplace_back([&] {
        ++go;
        while (go < 8) {}
        if (mla::ensure_device(&h) != MLA_OK || !ready(h)) ++wrong;
      });
    for (auto& t : threads) t.join();
    CHECK(1, wrong == 0);
    CHECK(2, g_mallocs == 1);
    cudaFree(h.d_err);
  }
  // reading the error word leaves it at zero, with no clearing on its way behind the call
  {
    mla_handle h;
    memset(&h, 0, sizeof(h));
    CHECK(8, mla::ensure_device(&h) == MLA_OK);
    *h.d_err = 5;
    uint32_t bits = 0;
    CHECK(9, mla::take_error_bits(&h, nullptr, &bits) == cudaSuccess && bits == 5);
    CHECK(10, *h.d_err == 0 && !g_pending);
    cudaFree(h.d_err);
  }
  // each runtime call fails once
  int failures = 0;
  for (int k = 0;; ++k) {
    mla_handle h;
    memset(&h, 0, sizeof(h));
    g_calls = 0;
    g_fail_at = k;
    const mla_status_t s = mla::ensure_device(&h);
    g_fail_at = -1;
    if (s == MLA_OK) {                  // there is no k-th call
      CHECK(3, ready(h));
      cudaFree(h.d_err);
      break;
    }
    ++failures;
    CHECK(4, s == MLA_ERR_CUDA && !h.d_err && h.num_sms == 0);
    CHECK(5, g_words == 0 && g_streams == 0);
    CHECK(6, mla::ensure_device(&h) == MLA_OK && ready(h));
    cudaFree(h.d_err);
  }
  CHECK(7, failures >= 3 && g_words == 0 && g_streams == 0);
  puts("ok");
  return 0;
}
