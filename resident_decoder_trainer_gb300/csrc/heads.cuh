// What the per-head norm with rotation and the attention over spans share:
// the checks of a [tokens, heads, head_dim] tensor and launches that overlap.
#pragma once

#include <cuda_fp16.h>

#include <atomic>

#include "../../include/rdt.h"
#include "common.cuh"
#include "internal.h"

namespace rdt {

// Each kernel of these files may be launched while the one before it in the
// stream still runs, and waits here for its end before it touches memory
// (programmatic launch). Nothing is read through the read-only path (__ldg,
// const __restrict__): that is for memory nobody writes while the kernel is
// there, and this one may be there while the kernel before it writes.
__device__ __forceinline__ void after_previous_kernel() {
  asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
}

// Launches `kernel` so that it may start while the stream's previous one ends.
template <typename... P, typename... A>
cudaError_t launch_overlapping(void (*kernel)(P...), int64_t grid, int threads, size_t smem,
                               cudaStream_t s, A... args) {
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  note_launch();
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// Lets a kernel have `smem` bytes of dynamic shared memory on the current device;
// asked for once on each of the first 64 devices.
template <auto kernel>
cudaError_t allow_smem(size_t smem) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem));
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

inline rdt_status refuse(const char* msg) {
  set_last_error(msg);
  return RDT_EINVAL;
}
inline rdt_status launched(cudaError_t e) {
  if (e == cudaSuccess) return RDT_OK;
  cudaGetLastError();  // not left for the next call to find
  set_last_error(cudaGetErrorString(e));
  return RDT_ECUDA;
}

inline bool dtype_ok(int dtype) {
  return dtype == RDT_F32 || dtype == RDT_BF16 || dtype == RDT_F16;
}
inline int dtype_bytes(int dtype) { return dtype == RDT_F32 ? 4 : 2; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

// What is wrong with x as a [tokens, heads, d] tensor; null if nothing is. A
// stride along an axis of one element is not looked at.
inline const char* heads_problem(const rdt_heads* x, int64_t tokens, int64_t heads, int64_t d,
                                 int bytes, bool written) {
  if (!x || !x->data) return "null pointer";
  const int64_t ts = x->token_stride, hs = x->head_stride;
  if (reinterpret_cast<uintptr_t>(x->data) & 15) return "tensors must be 16-byte aligned";
  const int64_t most = (int64_t{1} << 39) / bytes;
  if ((tokens > 1 && (ts < d || ts > most)) || (heads > 1 && (hs < d || hs > most)))
    return "strides must be at least head_dim and below 2^39 bytes";
  if ((tokens > 1 && ts * bytes % 16) || (heads > 1 && hs * bytes % 16))
    return "strides must be multiples of 16 bytes";
  if (written && tokens > 1 && heads > 1) {
    const bool apart = ts >= hs ? ts >= (heads - 1) * hs + d : hs >= (tokens - 1) * ts + d;
    if (!apart) return "a written tensor overlaps itself";
  }
  return nullptr;
}

}  // namespace rdt
