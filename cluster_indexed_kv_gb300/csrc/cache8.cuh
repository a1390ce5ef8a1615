// cache8.cuh -- shared by the calls that have no context: rotary positions
// and the 8-bit cache (rope.cu, cache8.cu, move8.cu, attend8.cu).
#pragma once

#include <cuda_fp16.h>

#include <atomic>
#include <cstdio>
#include <type_traits>

#include "../../include/lkv.h"
#include "lkv_internal.cuh"

namespace lkv {

constexpr int kBlock = LKV_CACHE8_BLOCK;  // tokens that share a scale

// Anomalies of a cache, kept in ticket[batch] until lkv_cache8_status.
enum : int32_t {
  kAnomRange = 1,      // a write's start or count is not one the cache can take, or what a take or keep names is not there
  kAnomCapacity = 2,   // a write, take or keep past the capacity
  kAnomNotFinite = 4,  // a NaN or an infinity was written
  kAnomTimeout = 8,    // a bounded wait in an attention, take or keep gave up
};

inline lkv_status refuse(const char *msg) {
  set_unbound_error(msg);
  return LKV_EINVAL;
}

inline lkv_status refuse_in(const char *where, const char *why) {
  char buf[192];
  std::snprintf(buf, sizeof buf, "%s: %s", where, why);
  return refuse(buf);
}

inline lkv_status cuda_refuse(const char *where, cudaError_t e) {
  char buf[256];
  std::snprintf(buf, sizeof buf, "%s: %s", where, cudaGetErrorString(e));
  set_unbound_error(buf);
  return LKV_ECUDA;
}

inline bool aligned(const void *p, uintptr_t to) { return (uintptr_t)p % to == 0; }

inline bool overlap(const void *a, int64_t an, const void *b, int64_t bn) {
  if (!a || !b || an <= 0 || bn <= 0) return false;
  return (uintptr_t)a < (uintptr_t)b + (uintptr_t)bn && (uintptr_t)b < (uintptr_t)a + (uintptr_t)an;
}

// Multiprocessors of the current device.
inline cudaError_t sm_count(int *sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

// The sizes and pointers of a cache, checked; null if they are fine.
const char *check_cache8(const lkv_cache8 *c);
// Whether [p, p + bytes) lies in one of the cache's arrays.
bool overlaps_cache8(const lkv_cache8 *c, const void *p, int64_t bytes);
// Whether two of the cache's own arrays share memory, and one of a's with one of b's.
bool cache8_arrays_overlap(const lkv_cache8 *c);
bool caches_overlap(const lkv_cache8 *a, const lkv_cache8 *b);

// Programmatic dependent launch: the stream's next kernel may start; and:
// everything the previous kernel wrote is visible, and it has ended. Every
// kernel of these calls is launched that way and waits before its first access
// to memory, so that its launch overlaps the end of the kernel before. Rotating
// and writing let the next kernel start once their own wait is over; reading
// and attention (but for their own merge) do not, as its waiting blocks cost
// them more (16 rows read back 5.7 against 4.8 us, 8 x 8K tokens attended 41
// against 39 us a step). A step (rotate, write, attend) of 8 sequences, from
// call to call: at 8K 47.0 -> 39.7 us, at 32K 102.1 -> 93.6.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_prerequisites() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Whether a kernel has been allowed its largest dynamic shared memory on a
// device: once a process (two such calls for each attention behind prefixes took
// 3 of its 17 us from Python). The runtime keeps that for the device, in every
// context and past a reset of the primary one.
struct SmemAllowed {
  std::atomic<bool> on[64]{};
  cudaError_t allow(const void *fn, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && on[dev].load(std::memory_order_acquire))) return e;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) on[dev].store(true, std::memory_order_release);
    return e;
  }
};

template <class... Args>
inline cudaError_t launch_next(void (*fn)(Args...), dim3 grid, int block, size_t smem, cudaStream_t st, const std::common_type_t<Args> &...args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 w = __floats2bfloat162_rn(lo, hi);
  return *(const uint32_t *)&w;
}

// Four codes as values.
template <int CODE>
__device__ __forceinline__ void decode4(uint32_t w, float (&x)[4]) {
  if constexpr (CODE == LKV_CODE_INT8) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = (float)(int8_t)(w >> (8 * e));
  } else {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
    const float2 a = __half22float2(*(__half2 *)&lo), b = __half22float2(*(__half2 *)&hi);
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  }
}

}  // namespace lkv
