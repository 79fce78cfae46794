// Launch helpers shared by the kernel translation units.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace af {

// Raises a kernel's dynamic shared-memory limit once per device (the
// attribute stays set for the life of the context); `force` sets it again
// (after a context was torn down and recreated).
template <auto KERN>
cudaError_t set_smem_once(int bytes, bool force = false) {
  static std::atomic<uint64_t> done{0};   // one per kernel
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
  if (!force && bit != 0ull && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && bit != 0ull) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

// Launches `launch()`; if that fails, sets the kernel's shared-memory limit
// again and retries once.
template <auto KERN, class F>
cudaError_t launch_with_smem(int bytes, F launch) {
  cudaError_t e = set_smem_once<KERN>(bytes);
  if (e != cudaSuccess) return e;
  e = launch();
  if (e == cudaSuccess) return e;
  if ((e = set_smem_once<KERN>(bytes, true)) != cudaSuccess) return e;
  return launch();
}

// Launches `kern(p)` as a programmatic dependent of the kernel before it on
// the stream: its blocks may start while that kernel's last ones finish, and
// wait for it (griddepcontrol.wait) before their first global access.
template <class K, class P>
cudaError_t launch_dependent(K kern, const P& p, dim3 grid, int threads, int smem_bytes, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem_bytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace af
