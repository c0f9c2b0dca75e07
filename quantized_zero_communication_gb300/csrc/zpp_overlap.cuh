// zpp_overlap.cuh -- launches whose CTAs may be placed while the kernel before them in the
// stream is still ending (programmatic stream serialization): the launch itself, some 1 to 2
// us, is then hidden. Such a kernel calls grid_wait() before it touches global memory.
#pragma once

#include <cuda_runtime.h>

#include "zpp_device.cuh"

namespace zpp {

// Returns once the kernels before this one in the stream have ended and their writes are
// visible (at once if this kernel was launched without overlap).
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Lets the next kernel's CTAs be placed from now on.
__device__ __forceinline__ void grid_release() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Loads of what the kernel before may have written: ordinary ones, which the compiler leaves
// behind grid_wait(). The read-only path (ld.global.nc) is for data that does not change while
// a kernel runs, and an overlapped kernel begins to run before its predecessor's last store.
__device__ __forceinline__ uint4 ld_after_v4(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}
// The same through L1, for data that several warps read.
__device__ __forceinline__ uint4 ld_after_shared_v4(const void* p) {
  uint4 r;
  asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}
// Predicated, without a branch: r keeps its value where not `on`.
__device__ __forceinline__ void ld_after_shared_v4_if(bool on, const void* p, uint4& r) {
  asm volatile(
      "{.reg .pred q; setp.ne.b32 q, %5, 0; @q ld.global.v4.b32 {%0,%1,%2,%3}, [%4];}"
      : "+r"(r.x), "+r"(r.y), "+r"(r.z), "+r"(r.w)
      : "l"(p), "r"(static_cast<int>(on))
      : "memory");
}
__device__ __forceinline__ void ld_after_shared_v2_if(bool on, const void* p, uint4& r) {
  asm volatile("{.reg .pred q; setp.ne.b32 q, %3, 0; @q ld.global.v2.b32 {%0,%1}, [%2];}"
               : "+r"(r.x), "+r"(r.y)
               : "l"(p), "r"(static_cast<int>(on))
               : "memory");
}
__device__ __forceinline__ float ld_after_f32(const float* p) {
  float r;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(r) : "l"(p) : "memory");
  return r;
}
__device__ __forceinline__ double ld_after_f64(const double* p) {
  double r;
  asm volatile("ld.global.f64 %0, [%1];" : "=d"(r) : "l"(p) : "memory");
  return r;
}
__device__ __forceinline__ uint16_t ld_after_u16(const uint16_t* p) {
  uint16_t r;
  asm volatile("ld.global.u16 %0, [%1];" : "=h"(r) : "l"(p) : "memory");
  return r;
}
template <bool V8>
__device__ __forceinline__ U8x32 ld_after_vec32(const void* p) {
  U8x32 r;
  if constexpr (V8) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]),
                   "=r"(r.w[5]), "=r"(r.w[6]), "=r"(r.w[7])
                 : "l"(p)
                 : "memory");
  } else {
    const uint4 a = ld_after_v4(p), b = ld_after_v4(static_cast<const uint8_t*>(p) + 16);
    r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
    r.w[4] = b.x, r.w[5] = b.y, r.w[6] = b.z, r.w[7] = b.w;
  }
  return r;
}

// smem: dynamic shared memory; cluster: CTAs of a cluster (along x).
template <typename... Params, typename... Args>
inline cudaError_t launch_overlapped_cluster(void (*kern)(Params...), dim3 grid, int cluster, int threads,
                                             int smem, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}
template <typename... Params, typename... Args>
inline cudaError_t launch_overlapped_smem(void (*kern)(Params...), dim3 grid, int threads, int smem,
                                          cudaStream_t s, const Args&... args) {
  return launch_overlapped_cluster(kern, grid, 1, threads, smem, s, args...);
}
template <typename... Params, typename... Args>
inline cudaError_t launch_overlapped(void (*kern)(Params...), int grid, int threads, cudaStream_t s,
                                     const Args&... args) {
  return launch_overlapped_smem(kern, dim3(static_cast<unsigned>(grid)), threads, 0, s, args...);
}

}  // namespace zpp
