// adamw.cu -- K8: one AdamW step over a list of tensors, fp32 master weights, states in
// fp32 or as e4m3 codes with a scale per 256 elements.
//
//   g = c grad;  m = b1 m + (1-b1) g;  v = b2 v + (1-b2) g^2
//   p = p - (lr wd p + lr/(1-b1^t) m / (sqrt(v)/sqrt(1-b2^t) + eps))
//
// Elementwise and memory-bound: every byte of p, m, v and g is read once and p, m, v (and
// the 16-bit weight) written once. A warp owns 256 consecutive elements of one tensor, which
// is one state block, so the block maximum of an 8-bit state is a warp reduction and the
// states never leave registers between decoding and encoding. A lane holds 8 consecutive
// elements: 32 bytes of p, one 256-bit access where the buffers allow it.
//
// fp32 states are bound by DRAM: 201,326,592 elements with bf16 gradients and weights 801 us, 7.04
// TB/s over 28 bytes each. 8-bit states (16.06 bytes) are bound by instruction issue, some 80 per
// element: 268,435,456 elements 680 us, 6.34 TB/s, issue slots 79 % busy; a warp takes two blocks
// there so that the loads of one cover the arithmetic of the other. A short list is bound by the
// call: 1024 elements 5.6 us, 1.8 of them on the device.
#include <cuda_fp8.h>

#include "zpp_device.cuh"
#include "zpp_launch.h"
#include "zpp_overlap.cuh"
#include "zpp_step_count.cuh"

namespace zpp {

constexpr int kVec = kStateBlock / 32;  // elements per lane
static_assert(kVec == 8, "the vector accesses below hold 8 elements");
static_assert(adamw_chunk(32) == kWarps * kStateBlock, "one state block per warp");
constexpr float kFltMax = 3.402823466e38f;

template <bool V8>
__device__ __forceinline__ void ld_f32x8(const float* p, float f[kVec]) {
  const U8x32 w = ld_after_vec32<V8>(p);
#pragma unroll
  for (int k = 0; k < kVec; ++k) f[k] = __uint_as_float(w.w[k]);
}
__device__ __forceinline__ uint2 ld_b32x2(const void* p) {
  uint2 r;
  asm volatile("ld.global.L1::no_allocate.v2.b32 {%0,%1}, [%2];"
               : "=r"(r.x), "=r"(r.y)
               : "l"(p)
               : "memory");
  return r;
}
template <bool V8>
__device__ __forceinline__ void st_f32x8(float* p, const float f[kVec]) {
  U8x32 w;
#pragma unroll
  for (int k = 0; k < kVec; ++k) w.w[k] = __float_as_uint(f[k]);
  st_vec32<V8>(p, w);
}

// Gradients of a lane's 8 elements: raw words first (so that every load of the block is in
// flight before the first conversion), floats later.
template <bool V8>
__device__ __forceinline__ U8x32 ld_grad(const void* g, int64_t i, int kind) {
  if (kind == 2) return ld_after_vec32<V8>(static_cast<const float*>(g) + i);
  const uint4 a = ld_after_v4(static_cast<const uint16_t*>(g) + i);
  U8x32 r;
  r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
  return r;
}
__device__ __forceinline__ void grad_f32(const U8x32& w, int kind, float f[kVec]) {
  if (kind == 2) {
#pragma unroll
    for (int k = 0; k < kVec; ++k) f[k] = __uint_as_float(w.w[k]);
  } else {
#pragma unroll
    for (int k = 0; k < kVec / 2; ++k) {
      const float2 p = kind == 0 ? unpack2(w.w[k], F16()) : unpack2(w.w[k], BF16());
      f[2 * k] = p.x;
      f[2 * k + 1] = p.y;
    }
  }
}
// Two e4m3 codes -> floats (exact).
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t w) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3);
  return __half22float2(__half2(h));
}
// Two floats that are e4m3 values (or NaN) -> codes.
__device__ __forceinline__ uint32_t f32_to_e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// 32 bits for element number i: low 16 round m, high 16 round sqrt(v). Two multiply-xorshift
// rounds over a Weyl sequence; the odd constants are fractional bits of the golden ratio and of
// the square roots of 3, 7 and 13. A block's numbers start at a multiple of 256, so they share
// their high word: hash_start gives the sequence at the block's first number, hash_at the bits
// of the o-th after it, the last xorshift left to the two users (it changes the low half only).
__device__ __forceinline__ uint32_t hash_start(uint64_t i, uint32_t key) {
  return static_cast<uint32_t>(i) * 0x9E3779B9u + static_cast<uint32_t>(i >> 32) * 0xA54FF53Bu + key;
}
__device__ __forceinline__ uint32_t hash_at(uint32_t start, uint32_t o, uint32_t key) {
  uint32_t x = start + o * 0x9E3779B9u;
  x = (x ^ (x >> 16)) * 0xBB67AE85u + key;
  return (x ^ (x >> 15)) * 0x9B05688Du;
}
// k + 1/2 in units of 2^-20 of a step, k the 16 bits for m or for sqrt(v).
__device__ __forceinline__ uint32_t bits_m(uint32_t x) { return ((x ^ (x >> 16)) << 4 & 0xFFFF0u) | 8u; }
__device__ __forceinline__ uint32_t bits_r(uint32_t x) { return (x >> 12 & 0xFFFF0u) | 8u; }

// The e4m3 value that x * inv rounds to, floor(|x inv| / h + (k + 1/2) / 65536) h: the random
// bits are added below the third mantissa bit and the sum is cut there. Below 2^-6 the grid
// is uniform (2^-9), which is the spacing of [2^-6, 2^-5): the value is shifted there and
// back. KEEP (x >= 0): x > 0 gives at least the smallest code. GUARD: a non-finite x becomes
// NaN (without it x has to be finite).
template <bool KEEP, bool GUARD>
__device__ __forceinline__ float e4m3_round(float x, float inv, uint32_t k) {
  const float s = __fmul_rn(fabsf(x), inv);
  const float shift = s < 0.015625f ? 0.015625f : 0.0f;
  const uint32_t b = (__float_as_uint(__fadd_rn(s, shift)) + k) & 0xFFF00000u;
  float r = __fadd_rn(__uint_as_float(b), -shift);
  if (KEEP && s > 0.0f) r = fmaxf(r, 0.001953125f);
  if (GUARD && !(fabsf(x) <= kFltMax)) r = __int_as_float(0x7fc00000);
  return KEEP ? r : copysignf(r, x);
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
  return a <= kFltMax ? a : 0.0f;
}
// max(a, |x|), NaN if either is.
__device__ __forceinline__ float max_abs_nan(float a, float x) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(x)));
  return r;
}
// Magnitudes order as their bit patterns, NaN above infinity.
__device__ __forceinline__ float warp_max_bits(float a) {
  return __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(a) & 0x7FFFFFFFu));
}
// 1 / x to one ulp; 0 for x above 2^126 and infinity for x below 2^-126.
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// sqrt(v) for v = 0 and for normal v by one Newton step with a fused residual (P. Markstein,
// Computation of elementary functions on the IBM RISC System/6000 processor, IBM J. Res. Dev. 34,
// 1990) from the approximate reciprocal root y: s = v y, then s + (v - s^2) y / 2. From v = 2^-102 on
// the residual is exact and the error before the last rounding below 2^-44, so the result is the
// correctly rounded root but for 2^-19 of the values at most; down to 2^-126 it is within one ulp. 268,435,456
// elements with 8-bit states: 680 us, 747 with __fsqrt_rn. v below 2^-126 gives a root below 2^-63,
// too small by up to a factor of 2000; an infinite v gives NaN.
__device__ __forceinline__ float sqrt_newton(float v) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fmaxf(v, 1.17549435e-38f)));
  const float s = __fmul_rn(v, y);
  return __fmaf_rn(__fmaf_rn(-s, s, v), __fmul_rn(0.5f, y), s);
}

// The factors that depend on the step's number and on its gradients. COUNTED: from its record, in
// registers; else they are kernel arguments but for the gradients' scale.
template <bool COUNTED>
struct Factors {
  float c;
  float step_size, inv_root_bc2;
  uint32_t key;
};

// One element: p, m, v updated in place, root = sqrt(v). For the states every operation is
// rounded by itself (no fused multiply-add), so that m and v, and the codes and scales of m, can be
// reproduced bit for bit by elementary fp32 arithmetic; those of the root but where it is not the
// rounded one. The quotient needs no such care: a reciprocal within one ulp.
template <bool FP8, bool COUNTED>
__device__ __forceinline__ void update(const AdamwArgs& a, const Factors<COUNTED>& f, float g, float& p,
                                       float& m, float& v, float& root) {
  m = __fadd_rn(__fmul_rn(a.beta1, m), __fmul_rn(a.one_minus_beta1, g));
  v = __fadd_rn(__fmul_rn(a.beta2, v), __fmul_rn(a.one_minus_beta2, __fmul_rn(g, g)));
  root = FP8 ? sqrt_newton(v) : __fsqrt_rn(v);
  const float q = __fmul_rn(m, rcp_approx(__fmaf_rn(root, COUNTED ? f.inv_root_bc2 : a.inv_root_bc2, a.eps)));
  p = __fadd_rn(p, -__fmaf_rn(a.decay, p, __fmul_rn(COUNTED ? f.step_size : a.step_size, q)));
}

// The codes of a lane's 8 consecutive elements. start: hash_start of the block; o: the first
// element's place in it.
template <bool GUARD>
__device__ __forceinline__ void encode8(const float m[kVec], const float root[kVec], float inv_m,
                                        float inv_r, uint32_t start, uint32_t o, uint32_t key,
                                        uint2& cm, uint2& cr) {
  uint32_t wm[kVec / 2], wr[kVec / 2];
#pragma unroll
  for (int k = 0; k < kVec / 2; ++k) {
    float x[2], y[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t h = hash_at(start, o + 2 * k + j, key);
      x[j] = e4m3_round<false, GUARD>(m[2 * k + j], inv_m, bits_m(h));
      y[j] = e4m3_round<true, GUARD>(root[2 * k + j], inv_r, bits_r(h));
    }
    wm[k] = f32_to_e4m3x2(x[0], x[1]);
    wr[k] = f32_to_e4m3x2(y[0], y[1]);
  }
  cm = make_uint2(wm[0] | wm[1] << 16, wm[2] | wm[3] << 16);
  cr = make_uint2(wr[0] | wr[1] << 16, wr[2] | wr[3] << 16);
}

// What a lane reads of a state block: 8 consecutive elements, the first `cnt` of them in the
// tensor. Every load is issued before the first use, also in a tensor's last, shorter block
// (PART): its warp would otherwise finish some 10 us after all others.
template <bool FP8>
struct Loaded {
  U8x32 g;
  float p[kVec], m[FP8 ? 1 : kVec], v[FP8 ? 1 : kVec];
  uint2 mq, vq;
  float ms, vs;
};
template <bool FP8, bool V8, bool PART>
__device__ __forceinline__ void load_block(const AdamwTensor& t, const AdamwArgs& a, int64_t block,
                                           int lane, int cnt, Loaded<FP8>& l) {
  const int64_t i = block * kStateBlock + lane * kVec;
  if constexpr (FP8) {
    l.ms = t.m_scale[block];
    l.vs = t.v_scale[block];
  }
  if (!PART || cnt == kVec) {
    l.g = ld_grad<V8>(t.grad, i, a.g_kind);
    ld_f32x8<V8>(t.param + i, l.p);
    if constexpr (FP8) {
      l.mq = ld_b32x2(static_cast<uint8_t*>(t.m) + i);
      l.vq = ld_b32x2(static_cast<uint8_t*>(t.v) + i);
    } else {
      ld_f32x8<V8>(static_cast<float*>(t.m) + i, l.m);
      ld_f32x8<V8>(static_cast<float*>(t.v) + i, l.v);
    }
    return;
  }
  uint32_t mq[2] = {0u, 0u}, vq[2] = {0u, 0u};
#pragma unroll
  for (int k = 0; k < kVec; ++k) {
    l.p[k] = 0.0f;
    l.g.w[k] = 0u;
    if constexpr (!FP8) l.m[k] = l.v[k] = 0.0f;
  }
#pragma unroll
  for (int k = 0; k < kVec; ++k) {
    if (k >= cnt) continue;
    l.p[k] = t.param[i + k];
    if (a.g_kind == 2) l.g.w[k] = __float_as_uint(static_cast<const float*>(t.grad)[i + k]);
    else
      l.g.w[k / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(t.grad)[i + k]) << (16 * (k & 1));
    if constexpr (FP8) {
      mq[k / 4] |= static_cast<uint32_t>(static_cast<uint8_t*>(t.m)[i + k]) << (8 * (k & 3));
      vq[k / 4] |= static_cast<uint32_t>(static_cast<uint8_t*>(t.v)[i + k]) << (8 * (k & 3));
    } else {
      l.m[k] = static_cast<float*>(t.m)[i + k];
      l.v[k] = static_cast<float*>(t.v)[i + k];
    }
  }
  l.mq = make_uint2(mq[0], mq[1]);
  l.vq = make_uint2(vq[0], vq[1]);
}

// One state block by a warp. number: the block's first element number in the list.
template <bool FP8, bool V8, bool PART, bool COUNTED>
__device__ __forceinline__ void step_block(const AdamwTensor& t, const AdamwArgs& a,
                                           const Factors<COUNTED>& f, int64_t block, int64_t number,
                                           int lane, int cnt, const Loaded<FP8>& l) {
  const int64_t i = block * kStateBlock + lane * kVec;
  float p[kVec], m[kVec], v[kVec], root[kVec], g[kVec];
  float ms = l.ms, vs = l.vs;
#pragma unroll
  for (int k = 0; k < kVec; ++k) {
    p[k] = l.p[k];
    if constexpr (!FP8) {
      m[k] = l.m[k];
      v[k] = l.v[k];
    }
  }
  grad_f32(l.g, a.g_kind, g);
  if constexpr (FP8) {
#pragma unroll
    for (int k = 0; k < kVec / 2; ++k) {
      const float2 x = e4m3x2_to_f32((k < 2 ? l.mq.x : l.mq.y) >> (16 * (k & 1)) & 0xffffu);
      const float2 y = e4m3x2_to_f32((k < 2 ? l.vq.x : l.vq.y) >> (16 * (k & 1)) & 0xffffu);
      m[2 * k] = __fmul_rn(x.x, ms);
      m[2 * k + 1] = __fmul_rn(x.y, ms);
      const float r0 = __fmul_rn(y.x, vs), r1 = __fmul_rn(y.y, vs);
      v[2 * k] = __fmul_rn(r0, r0);
      v[2 * k + 1] = __fmul_rn(r1, r1);
    }
  }
  float amax_m = 0.0f, amax_r = 0.0f;
#pragma unroll
  for (int k = 0; k < kVec; ++k) {
    update<FP8, COUNTED>(a, f, __fmul_rn(g[k], f.c), p[k], m[k], v[k], root[k]);
    if constexpr (FP8) {
      if (PART && k >= cnt) m[k] = root[k] = 0.0f;
      amax_m = max_abs_nan(amax_m, m[k]);
      amax_r = max_abs_nan(amax_r, root[k]);
    }
  }
  const bool whole = !PART || cnt == kVec;
  if (whole) {
    st_f32x8<V8>(t.param + i, p);
  } else {
#pragma unroll
    for (int k = 0; k < kVec; ++k)
      if (k < cnt) t.param[i + k] = p[k];
  }
  if (t.weight) {
    uint32_t w[kVec / 2];
#pragma unroll
    for (int k = 0; k < kVec / 2; ++k)
      w[k] = a.w_kind == 0 ? pack2(p[2 * k], p[2 * k + 1], F16())
                           : pack2(p[2 * k], p[2 * k + 1], BF16());
    uint16_t* to = static_cast<uint16_t*>(t.weight) + i;
    if (whole) {
      st_v4(to, make_uint4(w[0], w[1], w[2], w[3]));
    } else {
#pragma unroll
      for (int k = 0; k < kVec; ++k)
        if (k < cnt) to[k] = static_cast<uint16_t>(w[k / 2] >> (16 * (k & 1)));
    }
  }
  if constexpr (FP8) {
    amax_m = warp_max_bits(amax_m);
    amax_r = warp_max_bits(amax_r);
    const bool finite = amax_m <= kFltMax && amax_r <= kFltMax;  // the same in all lanes
    if (!finite) {  // scales over the finite values
      amax_m = amax_r = 0.0f;
#pragma unroll
      for (int k = 0; k < kVec; ++k) {
        amax_m = fmaxf(amax_m, finite_abs(m[k]));
        amax_r = fmaxf(amax_r, finite_abs(root[k]));
      }
      amax_m = warp_max_bits(amax_m);
      amax_r = warp_max_bits(amax_r);
    }
    float inv_m, inv_r;
    state_scale(amax_m, ms, inv_m);
    state_scale(amax_r, vs, inv_r);
    const uint32_t key = COUNTED ? f.key : a.key, start = hash_start(number, key);
    uint2 cm, cr;
    if (finite) encode8<false>(m, root, inv_m, inv_r, start, lane * kVec, key, cm, cr);
    else encode8<true>(m, root, inv_m, inv_r, start, lane * kVec, key, cm, cr);
    uint8_t *tm = static_cast<uint8_t*>(t.m) + i, *tv = static_cast<uint8_t*>(t.v) + i;
    if (whole) {
      st_v2(tm, cm);
      st_v2(tv, cr);
    } else {
#pragma unroll
      for (int k = 0; k < kVec; ++k)
        if (k < cnt) {
          tm[k] = static_cast<uint8_t>((k < 4 ? cm.x : cm.y) >> (8 * (k & 3)));
          tv[k] = static_cast<uint8_t>((k < 4 ? cr.x : cr.y) >> (8 * (k & 3)));
        }
    }
    if (lane == 0) {
      t.m_scale[block] = ms;
      t.v_scale[block] = vs;
    }
  } else {
    float *tm = static_cast<float*>(t.m) + i, *tv = static_cast<float*>(t.v) + i;
    if (whole) {
      st_f32x8<V8>(tm, m);
      st_f32x8<V8>(tv, v);
    } else {
#pragma unroll
      for (int k = 0; k < kVec; ++k)
        if (k < cnt) {
          tm[k] = m[k];
          tv[k] = v[k];
        }
    }
  }
}

// V8: p, fp32 states and fp32 gradients of every tensor start 32-byte aligned. COUNTED: the factors
// are those of the record, which an earlier launch wrote.
template <bool FP8, bool V8, bool COUNTED, int CAP>
__global__ void __launch_bounds__(kThreads) k_adamw(const __grid_constant__ AdamwTableOf<CAP> tab) {
  const AdamwArgs& a = tab.a;
  grid_wait();  // everything before this launch is done and visible
  Factors<COUNTED> f;
  if constexpr (COUNTED) {
    const uint4 r = ld_after_shared_v4(&a.record->factor);
    f = {__uint_as_float(r.x), __uint_as_float(r.y), __uint_as_float(r.z), r.w};
  } else {
    f.c = a.grad_scale ? *static_cast<const volatile float*>(a.grad_scale) : 1.0f;
  }
  if (!isfinite(f.c)) return;  // overflowed gradients: the step is skipped
  const int lo = tensor_of(tab.hints, tab.first, static_cast<int>(blockIdx.x));
  const AdamwTensor& t = tab.t[lo];
  const int lane = threadIdx.x & 31;
  constexpr int NB = adamw_warp_blocks(FP8 ? 8 : 32);
  const int64_t block =
      static_cast<int64_t>(blockIdx.x - tab.first[lo]) * (kWarps * NB) + (threadIdx.x >> 5) * NB;
  const int64_t left = t.n - block * kStateBlock;
  if (left <= 0) return;
  const int64_t number = (tab.first_block + tab.block0[lo] + block) * kStateBlock;
  if (left >= NB * kStateBlock) {
    Loaded<FP8> l[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) load_block<FP8, V8, false>(t, a, block + b, lane, kVec, l[b]);
#pragma unroll
    for (int b = 0; b < NB; ++b)
      step_block<FP8, V8, false, COUNTED>(t, a, f, block + b, number + b * kStateBlock, lane, kVec, l[b]);
  } else {
    for (int b = 0; b < NB && left > b * kStateBlock; ++b) {
      const int cnt =
          static_cast<int>(min(left - b * kStateBlock - lane * kVec, static_cast<int64_t>(kVec)));
      Loaded<FP8> l;
      load_block<FP8, V8, true>(t, a, block + b, lane, max(cnt, 0), l);
      step_block<FP8, V8, true, COUNTED>(t, a, f, block + b, number + b * kStateBlock, lane, max(cnt, 0), l);
    }
  }
  // A step whose number the host knows leaves it in the record. (Before the step's own work this
  // branch costs 17 us of 680 on 268,435,456 elements with 8-bit states.)
  if constexpr (!COUNTED)
    if (a.record && blockIdx.x == 0 && threadIdx.x < 2) {  // (a beta of 0: no power is kept)
      a.record->beta[threadIdx.x] = a.record->power[threadIdx.x] = 0.0;
      if (threadIdx.x == 0) a.record->step = a.step;
    }
}

template <bool COUNTED, int CAP>
static cudaError_t run_counted(AdamwTableOf<CAP>& tab, int state_bits, bool v8, cudaStream_t s) {
  const int grid = tab.first[tab.count];
  tab.hints.fill(tab.first, tab.count);
  auto kern = state_bits == 8
                  ? (v8 ? k_adamw<true, true, COUNTED, CAP> : k_adamw<true, false, COUNTED, CAP>)
                  : (v8 ? k_adamw<false, true, COUNTED, CAP> : k_adamw<false, false, COUNTED, CAP>);
  return launch_overlapped(kern, grid, kThreads, s, tab);
}
template <int CAP>
static cudaError_t run_adamw(AdamwTableOf<CAP>& tab, int state_bits, bool v8, cudaStream_t s) {
  return tab.a.record && tab.a.step == 0 ? run_counted<true>(tab, state_bits, v8, s)
                                         : run_counted<false>(tab, state_bits, v8, s);
}

__global__ void __launch_bounds__(32) k_step_count(const StepCount c, const float* grad_scale) {
  grid_wait();
  grid_release();
  const int lane = threadIdx.x;
  const float factor = grad_scale ? *static_cast<const volatile float*>(grad_scale) : 1.0f;
  StepFactor f{};
  if (lane < 2) f = step_factor(c, lane);
  const float inv_root_bc2 = __shfl_sync(~0u, f.made, 1);
  if (lane < 2) write_record(c, f, lane, factor, inv_root_bc2);
}

cudaError_t launch_step_count(const StepCount& count, const float* grad_scale, cudaStream_t s) {
  return launch_overlapped(k_step_count, 1, 32, s, count, grad_scale);
}

cudaError_t launch_adamw(AdamwTable& tab, int state_bits, cudaStream_t s) {
  uintptr_t bits = 0;
  for (int i = 0; i < tab.count; ++i) {
    const AdamwTensor& t = tab.t[i];
    bits |= reinterpret_cast<uintptr_t>(t.param);
    if (tab.a.g_kind == 2) bits |= reinterpret_cast<uintptr_t>(t.grad);
    if (state_bits == 32) bits |= reinterpret_cast<uintptr_t>(t.m) | reinterpret_cast<uintptr_t>(t.v);
  }
  const bool v8 = (bits & 31) == 0;
  if (tab.count > kFewTensors) return run_adamw(tab, state_bits, v8, s);
  AdamwTableOf<kFewTensors> few;
  for (int i = 0; i < tab.count; ++i) {
    few.t[i] = tab.t[i];
    few.first[i] = tab.first[i];
    few.block0[i] = tab.block0[i];
  }
  few.first[tab.count] = tab.first[tab.count];
  few.count = tab.count;
  few.first_block = tab.first_block;
  few.a = tab.a;
  return run_adamw(few, state_bits, v8, s);
}

}  // namespace zpp
