// adamw.cu -- K8: one AdamW step over a list of tensors, fp32 master weights, states in
// fp32 or as e4m3 codes with a scale per 256 elements.
//
//   g = c grad;  m = b1 m + (1-b1) g;  v = b2 v + (1-b2) g^2
//   p = p - (lr wd p + lr/(1-b1^t) m / (sqrt(v)/sqrt(1-b2^t) + eps))
//
// Elementwise and memory-bound: every byte of p, m, v and g is read once and p, m, v (and
// the 16-bit weight) written once. A warp owns 256 consecutive elements of one tensor, which
// is one state block, so the block maximum of an 8-bit state is a warp reduction.
#include <cuda_fp8.h>

#include "zpp_device.cuh"
#include "zpp_launch.h"

namespace zpp {

constexpr int kVec = kStateBlock / 32;  // elements per lane
static_assert(kAdamwChunk == kWarps * kStateBlock, "one state block per warp");

__device__ __forceinline__ float grad_at(const void* p, int64_t i, int kind) {
  if (kind == 2) return static_cast<const float*>(p)[i];
  const uint16_t b = static_cast<const uint16_t*>(p)[i];
  return kind == 0 ? bits16_to_float(b, F16()) : bits16_to_float(b, BF16());
}

__device__ __forceinline__ float e4m3_to_f32(uint8_t b) {
  __nv_fp8_e4m3 v;
  v.__x = b;
  return static_cast<float>(v);
}

// 32 bits for element number i: low 16 round m, high 16 round sqrt(v). Two multiply-xorshift
// rounds over a Weyl sequence; the odd constants are fractional bits of the golden ratio and of
// the square roots of 3, 7 and 13.
__device__ __forceinline__ uint32_t round_bits(uint64_t i, uint32_t key) {
  uint32_t x = static_cast<uint32_t>(i) * 0x9E3779B9u +
               static_cast<uint32_t>(i >> 32) * 0xA54FF53Bu + key;
  x = (x ^ (x >> 16)) * 0xBB67AE85u + key;
  x = (x ^ (x >> 15)) * 0x9B05688Du;
  return x ^ (x >> 16);
}

// e4m3 code of x * inv, rounded by floor(|x inv| / h + (k + 1/2) / 65536): adding the random
// bits below the third mantissa bit and cutting there. Below 2^-6 the grid is uniform (2^-9),
// which is the spacing of [2^-6, 2^-5): the value is shifted there and back. A non-finite x
// becomes NaN. KEEP: x > 0 gives at least the smallest code.
template <bool KEEP>
__device__ __forceinline__ uint8_t e4m3_round(float x, float inv, uint32_t k16) {
  const float a = fabsf(x);
  const float s = __fmul_rn(a, inv);
  const bool low = s < 0.015625f;
  uint32_t b = __float_as_uint(low ? __fadd_rn(s, 0.015625f) : s);
  b = (b + (k16 * 16u + 8u)) & 0xFFF00000u;
  float r = __uint_as_float(b);
  if (low) r = __fadd_rn(r, -0.015625f);
  if (KEEP && a > 0.0f && inv > 0.0f) r = fmaxf(r, 0.001953125f);
  if (!(a <= 3.402823466e38f)) r = __int_as_float(0x7fc00000);
  return __nv_fp8_e4m3(copysignf(r, x)).__x;
}

// Scale of a state block from its largest finite magnitude, and its inverse, each by one
// correctly rounded reciprocal and a product; zero when the inverse would not be finite.
__device__ __forceinline__ void state_scale(float amax, float& scale, float& inv) {
  inv = __fmul_rn(448.0f, __frcp_rn(amax));
  scale = __fmul_rn(amax, 1.0f / 448.0f);
  if (!isfinite(inv)) inv = scale = 0.0f;
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.0f;
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads) k_adamw(const __grid_constant__ AdamwTable tab) {
  const AdamwArgs& a = tab.a;
  const float c = a.grad_scale ? __ldg(a.grad_scale) : 1.0f;
  if (!isfinite(c)) return;  // overflowed gradients: the step is skipped
  int lo = 0, hi = tab.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tab.first[mid] <= static_cast<int>(blockIdx.x)) lo = mid;
    else hi = mid;
  }
  const AdamwTensor& t = tab.t[lo];
  const int lane = threadIdx.x & 31;
  const int64_t block =
      static_cast<int64_t>(blockIdx.x - tab.first[lo]) * kWarps + (threadIdx.x >> 5);
  if (block * kStateBlock >= t.n) return;
  const int valid = static_cast<int>(min(static_cast<int64_t>(kStateBlock), t.n - block * kStateBlock));

  float ms = 1.0f, vs = 1.0f;
  if (FP8) {
    ms = t.m_scale[block];
    vs = t.v_scale[block];
  }
  float m[kVec], r[kVec], amax_m = 0.0f, amax_r = 0.0f;
#pragma unroll
  for (int k = 0; k < kVec; ++k) {
    const int o = k * 32 + lane;
    const int64_t i = block * kStateBlock + o;
    m[k] = r[k] = 0.0f;
    if (o >= valid) continue;
    const float g = __fmul_rn(grad_at(t.grad, i, a.g_kind), c);
    float m0, v0;
    if (FP8) {
      m0 = __fmul_rn(e4m3_to_f32(static_cast<uint8_t*>(t.m)[i]), ms);
      const float r0 = __fmul_rn(e4m3_to_f32(static_cast<uint8_t*>(t.v)[i]), vs);
      v0 = __fmul_rn(r0, r0);
    } else {
      m0 = static_cast<float*>(t.m)[i];
      v0 = static_cast<float*>(t.v)[i];
    }
    // States: every operation rounded by itself, so that the codes can be reproduced bit for
    // bit by elementary fp32 arithmetic.
    m0 = __fadd_rn(__fmul_rn(a.beta1, m0), __fmul_rn(a.one_minus_beta1, g));
    v0 = __fadd_rn(__fmul_rn(a.beta2, v0), __fmul_rn(a.one_minus_beta2, __fmul_rn(g, g)));
    const float root = __fsqrt_rn(v0);
    const float p0 = t.param[i];
    const float step = __fmul_rn(a.step_size, __fdiv_rn(m0, __fmaf_rn(root, a.inv_root_bc2, a.eps)));
    const float p = __fadd_rn(p0, -__fmaf_rn(a.decay, p0, step));
    t.param[i] = p;
    if (t.weight) {
      if (a.w_kind == 0) static_cast<__half*>(t.weight)[i] = __float2half_rn(p);
      else static_cast<__nv_bfloat16*>(t.weight)[i] = __float2bfloat16_rn(p);
    }
    if (FP8) {
      m[k] = m0;
      r[k] = root;
      amax_m = fmaxf(amax_m, finite_abs(m0));
      amax_r = fmaxf(amax_r, finite_abs(root));
    } else {
      static_cast<float*>(t.m)[i] = m0;
      static_cast<float*>(t.v)[i] = v0;
    }
  }
  if (FP8) {
    float inv_m, inv_r;
    state_scale(warp_max(amax_m, 32), ms, inv_m);
    state_scale(warp_max(amax_r, 32), vs, inv_r);
    // element number in the list: the blocks of earlier tensors (whole chunks are not
    // blocks, so they are counted tensor by tensor) come first
    int64_t before = tab.first_block;
    for (int j = 0; j < lo; ++j) before += (tab.t[j].n + kStateBlock - 1) / kStateBlock;
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      const int o = k * 32 + lane;
      if (o >= valid) continue;
      const uint32_t bits = round_bits(static_cast<uint64_t>((before + block) * kStateBlock + o), a.key);
      const int64_t i = block * kStateBlock + o;
      static_cast<uint8_t*>(t.m)[i] = e4m3_round<false>(m[k], inv_m, bits & 0xffffu);
      static_cast<uint8_t*>(t.v)[i] = e4m3_round<true>(r[k], inv_r, bits >> 16);
    }
    if (lane == 0) {
      t.m_scale[block] = ms;
      t.v_scale[block] = vs;
    }
  }
}

cudaError_t launch_adamw(const AdamwTable& tab, int state_bits, cudaStream_t s) {
  const int grid = tab.first[tab.count];
  if (state_bits == 8) k_adamw<true><<<grid, kThreads, 0, s>>>(tab);
  else k_adamw<false><<<grid, kThreads, 0, s>>>(tab);
  return cudaGetLastError();
}

}  // namespace zpp
