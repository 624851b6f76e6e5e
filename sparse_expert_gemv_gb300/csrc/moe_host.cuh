// What the host sides of the operators share: launches, tensor maps, and a
// handle's device error word.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <mutex>

#include "moe_decode.h"

namespace moe {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A tensor's bytes; null is none.
struct Span {
  const void* at;
  size_t bytes;
};
inline bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  return x && y && x < y + b.bytes && y < x + a.bytes;
}

template <typename... KArgs, typename... Args>
moe_status_t launch(void (*kernel)(KArgs...), unsigned grid, dim3 block, size_t smem, void* stream,
                    unsigned cluster, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

inline bool encode(CUtensorMap* tm, CUtensorMapDataType type, int rank, const void* base,
                   const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
  const cuuint32_t es[5] = {1, 1, 1, 1, 1};
  return fn && fn(tm, type, rank, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// err[1] = the error word err[0], which is cleared.
static __global__ void moe_take_error(uint32_t* err) { err[1] = atomicExch(err, 0u); }

struct Handle {
  int device;         // where the handle was created
  uint32_t* d_err;    // device error word, and where a read of it leaves its value
  // as the decode layer's handle has them: completion of the latest run outside
  // a capture, which the reads of the error word wait for, and their own
  // non-blocking stream; reads take turns
  cudaEvent_t done_ev;
  std::atomic<bool> done_recorded;
  cudaStream_t aux;
  std::mutex read_mu;

  // The error word cleared on s, the event and the stream; release() in any case.
  bool acquire(cudaStream_t s) {
    return cudaMalloc(&d_err, 8) == cudaSuccess && cudaMemsetAsync(d_err, 0, 8, s) == cudaSuccess &&
           cudaEventCreateWithFlags(&done_ev, cudaEventDisableTiming) == cudaSuccess &&
           cudaStreamCreateWithFlags(&aux, cudaStreamNonBlocking) == cudaSuccess;
  }
  void release() {
    if (done_ev) cudaEventDestroy(done_ev);
    if (aux) cudaStreamDestroy(aux);
    cudaFree(d_err);
  }

  // After a run has been enqueued on s: record its completion, unless s is being
  // captured into a graph (the event would stand for a graph node then).
  void mark_done(cudaStream_t s) {
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &cs) != cudaSuccess) {
      (void)cudaGetLastError();
      return;
    }
    if (cs != cudaStreamCaptureStatusNone) return;
    if (cudaEventRecord(done_ev, s) == cudaSuccess) done_recorded = true;
  }

  // Reads and clears the error word in one step, so that no bit set meanwhile is
  // lost, once the latest run outside a capture is over.
  moe_status_t read_error(uint32_t* device_flags) {
    if (done_recorded && cudaEventSynchronize(done_ev) != cudaSuccess) return MOE_ERR_CUDA;
    const std::lock_guard<std::mutex> turn(read_mu);
    int current = 0;
    if (cudaGetDevice(&current) != cudaSuccess || cudaSetDevice(device) != cudaSuccess)
      return MOE_ERR_CUDA;
    moe_take_error<<<1, 1, 0, aux>>>(d_err);
    uint32_t v = 0;
    const bool ok =
        cudaGetLastError() == cudaSuccess &&
        cudaMemcpyAsync(&v, d_err + 1, 4, cudaMemcpyDeviceToHost, aux) == cudaSuccess &&
        cudaStreamSynchronize(aux) == cudaSuccess;
    if (cudaSetDevice(current) != cudaSuccess || !ok) return MOE_ERR_CUDA;
    *device_flags = v;
    return v ? MOE_ERR_DEVICE_FAULT : MOE_OK;
  }
};

}  // namespace moe
