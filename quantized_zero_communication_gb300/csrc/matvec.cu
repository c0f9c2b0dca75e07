// matvec.cu -- K9: y = x W^T (+ bias) straight from block-quantised codes.
//
//   y[j][r] = sum_c q[r][c] scale[(r cols + c) / block] x[j][c] + bias[r]
//
// One warp per row and vector: lanes stride over the row's codes, fp32 sums joined by shuffles.
#include "zpp_device.cuh"
#include "zpp_launch.h"

namespace zpp {

__device__ __forceinline__ void store_y(void* y, int64_t i, float v, int kind) {
  if (kind == 2) static_cast<float*>(y)[i] = v;
  else if (kind == 0) static_cast<__half*>(y)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(y)[i] = __float2bfloat16_rn(v);
}

template <typename TT>
__global__ void __launch_bounds__(kThreads) k_matvec(const MatvecArgs a, int log2b) {
  const int lane = threadIdx.x & 31;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (r >= a.rows) return;
  for (int64_t j = blockIdx.y; j < a.vecs; j += gridDim.y) {
    const uint16_t* x = a.x + j * a.x_stride;
    float sum = 0.0f;
    for (int64_t c = lane; c < a.cols; c += 32) {
      const int64_t e = r * a.cols + c;
      const int q = a.bits == 8 ? static_cast<int>(static_cast<int8_t>(__ldg(a.codes + e)))
                                : code_int4(__ldg(a.codes + (e >> 1)), static_cast<int>(e & 1));
      const float w = __fmul_rn(static_cast<float>(q), __ldg(a.scales + (e >> log2b)));
      sum = __fmaf_rn(w, bits16_to_float(__ldg(x + c), TT()), sum);
    }
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane == 0) {
      if (a.bias) sum += bits16_to_float(__ldg(a.bias + r), TT());
      store_y(a.y, j * a.y_stride + r, sum, a.y_kind);
    }
  }
}

cudaError_t launch_matvec(const MatvecArgs& a, cudaStream_t s) {
  const int log2b = __builtin_ctz(static_cast<unsigned>(a.block));
  const dim3 grid(tile_grid(a.rows, kWarps), static_cast<unsigned>(a.vecs));
  if (a.x_bf16) k_matvec<BF16><<<grid, kThreads, 0, s>>>(a, log2b);
  else k_matvec<F16><<<grid, kThreads, 0, s>>>(a, log2b);
  return cudaGetLastError();
}

}  // namespace zpp
