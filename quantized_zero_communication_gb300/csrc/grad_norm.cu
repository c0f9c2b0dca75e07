// grad_norm.cu -- K7: the global gradient norm over a list of tensors, and the factor that
// clips it, left on the device for the optimiser step.
//
//   norm = |pre| sqrt(sum g^2),  coef = pre * min(1, max_norm / norm), NaN if the norm is not
//   finite.
//
// One pass over the gradients; each CTA sums one chunk of one tensor in fp32 and writes a
// partial, a single CTA adds the partials (in fp64) in a fixed order, so that the norm is the
// same in every run. Bound by DRAM: 536,870,912 bf16 elements 163 us, 6.6 TB/s; 32 registers
// leave room for 8 CTAs per SM, whose loads are all in flight at once. A short list is bound by
// its two launches: one of 1024 elements 4.1 us on the device.
#include "zpp_device.cuh"
#include "zpp_launch.h"
#include "zpp_overlap.cuh"
#include "zpp_step_count.cuh"

namespace zpp {

__device__ __forceinline__ float load_as_f32(const void* p, int64_t i, int kind) {
  if (kind == 2) return static_cast<const float*>(p)[i];
  const uint16_t b = static_cast<const uint16_t*>(p)[i];
  return kind == 0 ? bits16_to_float(b, F16()) : bits16_to_float(b, BF16());
}

template <typename T>
__device__ __forceinline__ T block_sum(T v) {  // valid in thread 0; blockDim.x <= 1024
  __shared__ T part[32];
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  const int warps = blockDim.x >> 5;
  v = threadIdx.x < warps ? part[threadIdx.x] : T(0);
  if (threadIdx.x < 32)
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// One chunk per CTA. A full chunk is kNormChunk / kThreads = 64 elements per thread, all of
// whose 32-byte vectors are loaded before the first product (no loop, so the most loads in
// flight); a tensor's last, shorter chunk is read element by element.
template <int KIND, bool V8, int CAP>
__global__ void __launch_bounds__(kThreads)
    k_norm_partial(const __grid_constant__ NormTableOf<CAP> tab, float* __restrict__ partial) {
  grid_wait();
  grid_release();
  const int lo = tensor_of(tab.hints, tab.first, static_cast<int>(blockIdx.x));
  const int64_t begin = static_cast<int64_t>(blockIdx.x - tab.first[lo]) * kNormChunk;
  const int64_t left = tab.n[lo] - begin;
  float sum = 0.0f;
  if (left >= kNormChunk) {
    constexpr int PER = KIND == 2 ? 8 : 16;  // elements in 32 bytes
    constexpr int VECS = kNormChunk / kThreads / PER;
    constexpr int BYTES = 32 / PER;
    const char* p = static_cast<const char*>(tab.ptr[lo]) + begin * BYTES + threadIdx.x * 32;
    U8x32 w[VECS];
#pragma unroll
    for (int u = 0; u < VECS; ++u) w[u] = ld_after_vec32<V8>(p + u * kThreads * 32);
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < VECS; ++u)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr (KIND == 2) {
          const float g = __uint_as_float(w[u].w[k]);
          acc[k & 3] = __fmaf_rn(g, g, acc[k & 3]);
        } else {
          const float2 g = KIND == 0 ? unpack2(w[u].w[k], F16()) : unpack2(w[u].w[k], BF16());
          acc[(2 * k) & 3] = __fmaf_rn(g.x, g.x, acc[(2 * k) & 3]);
          acc[(2 * k + 1) & 3] = __fmaf_rn(g.y, g.y, acc[(2 * k + 1) & 3]);
        }
      }
    sum = (acc[0] + acc[1]) + (acc[2] + acc[3]);
  } else {  // whole vectors first, all loaded ahead too, then the last few elements
    constexpr int PER = KIND == 2 ? 8 : 16;
    constexpr int VECS = kNormChunk / kThreads / PER;
    const int vecs = static_cast<int>(left) / PER;
    const char* p = static_cast<const char*>(tab.ptr[lo]) + begin * (32 / PER);
    U8x32 w[VECS];
#pragma unroll
    for (int u = 0; u < VECS; ++u) {
      const int at = u * kThreads + threadIdx.x;
#pragma unroll
      for (int k = 0; k < 8; ++k) w[u].w[k] = 0u;
      if (at < vecs) w[u] = ld_after_vec32<V8>(p + static_cast<int64_t>(at) * 32);
    }
    const int64_t i = begin + vecs * PER + threadIdx.x;
    if (i < begin + left) {  // fewer than PER elements
      const float g = load_as_f32(tab.ptr[lo], i, KIND);
      sum = __fmul_rn(g, g);
    }
#pragma unroll
    for (int u = 0; u < VECS; ++u)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr (KIND == 2) {
          const float g = __uint_as_float(w[u].w[k]);
          sum = __fmaf_rn(g, g, sum);
        } else {
          const float2 g = KIND == 0 ? unpack2(w[u].w[k], F16()) : unpack2(w[u].w[k], BF16());
          sum = __fmaf_rn(g.x, g.x, sum);
          sum = __fmaf_rn(g.y, g.y, sum);
        }
      }
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// COUNTED: also the record of the optimiser step by this factor, by the last warp, which makes the
// step's factors while the others wait for their partials.
template <bool COUNTED>
__global__ void __launch_bounds__(1024) k_norm_finish(const float* __restrict__ partial, int count,
                                                      float pre_scale, float max_norm,
                                                      float* __restrict__ out, const StepCount c) {
  grid_wait();
  grid_release();
  const int lane = static_cast<int>(threadIdx.x) - (1024 - 32);
  StepFactor f{};
  if constexpr (COUNTED)
    if (lane == 0 || lane == 1) f = step_factor(c, lane);
  __shared__ float taken_by;
  double sum = 0.0;
  for (int i = threadIdx.x; i < count; i += 1024)
    sum += static_cast<double>(*static_cast<const volatile float*>(partial + i));
  sum = block_sum(sum);
  if (threadIdx.x == 0) {
    const float norm = static_cast<float>(sqrt(sum)) * fabsf(pre_scale);
    out[0] = norm;
    const float factor = !isfinite(norm) ? __int_as_float(0x7fc00000)
                                         : pre_scale * (norm > max_norm ? max_norm / norm : 1.0f);
    out[1] = factor;
    if constexpr (COUNTED) taken_by = factor;
  }
  if constexpr (COUNTED) {
    __syncthreads();
    const float inv_root_bc2 = __shfl_sync(~0u, f.made, 1);
    if (lane == 0 || lane == 1) write_record(c, f, lane, taken_by, inv_root_bc2);
  }
}

template <int CAP>
static cudaError_t run_partial(NormTableOf<CAP>& tab, int g_kind, bool v8, float* workspace,
                               cudaStream_t s) {
  auto kern = g_kind == 2   ? (v8 ? k_norm_partial<2, true, CAP> : k_norm_partial<2, false, CAP>)
              : g_kind == 1 ? (v8 ? k_norm_partial<1, true, CAP> : k_norm_partial<1, false, CAP>)
                            : (v8 ? k_norm_partial<0, true, CAP> : k_norm_partial<0, false, CAP>);
  tab.hints.fill(tab.first, tab.count);
  return launch_overlapped(kern, tab.first[tab.count], kThreads, s, tab, workspace);
}

cudaError_t launch_grad_norm(NormTable& tab, int g_kind, float pre_scale, float max_norm,
                             float* workspace, float* out, const StepCount& count, cudaStream_t s) {
  const int chunks = tab.first[tab.count];
  if (chunks > 0) {
    uintptr_t bits = 0;
    for (int i = 0; i < tab.count; ++i)
      if (tab.n[i] > 0) bits |= reinterpret_cast<uintptr_t>(tab.ptr[i]);
    const bool v8 = (bits & 31) == 0;
    cudaError_t e;
    if (tab.count > kFewTensors) {
      e = run_partial(tab, g_kind, v8, workspace, s);
    } else {
      NormTableOf<kFewTensors> few;
      for (int i = 0; i < tab.count; ++i) {
        few.ptr[i] = tab.ptr[i];
        few.n[i] = tab.n[i];
        few.first[i] = tab.first[i];
      }
      few.first[tab.count] = chunks;
      few.count = tab.count;
      e = run_partial(few, g_kind, v8, workspace, s);
    }
    if (e != cudaSuccess) return e;
  }
  return launch_overlapped(count.record ? k_norm_finish<true> : k_norm_finish<false>, 1, 1024, s,
                           static_cast<const float*>(workspace), chunks, pre_scale, max_norm, out, count);
}

}  // namespace zpp
