// matvec.cu -- K9: y = x W^T (+ bias) straight from block-quantised codes.
//
//   y[j][r] = sum_c q[r][c] scale[(r cols + c) / block] x[j][c] + bias[r]
//
// Memory-bound: the codes are read once for up to 32 vectors. What would bound it first is the
// work per code, so the fast kernel gives the products to the matrix unit: codes become
// exact fp16 / bf16 integers with one logic and one half-precision operation per two, a
// fragment of 16 rows meets 8 vectors, and products (exact) and sums are fp32.
#include <cooperative_groups.h>

#include "zpp_device.cuh"
#include "zpp_launch.h"

namespace zpp {
namespace cg = cooperative_groups;

__device__ __forceinline__ void store_y(void* y, int64_t i, float v, int kind) {
  if (kind == 2) static_cast<float*>(y)[i] = v;
  else if (kind == 0) static_cast<__half*>(y)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(y)[i] = __float2bfloat16_rn(v);
}

// ---------------------------------------------------------------------------------
// A word of codes -> pairs of exact 16-bit floats. Pair p of an INT4 word holds codes (p, p + 4),
// of an INT8 word (p, p + 2): the two halves of a 32-bit word, so a mask serves both at once.
// One logic operation, (w & mask) ^ flip, puts a code with its sign bit flipped (q + 8 or
// q + 128) into mantissa bits of a power of two; a half-precision operation, exact too, leaves q.
// (Leaving the offset in and starting the fp32 sums at -offset sum(x) saves that operation,
// but not time: these run on another pipe than the logic.)
// ---------------------------------------------------------------------------------
struct Masks {
  uint32_t k[4];
};
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b, F16) {
  const __half2 r = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b, BF16) {
  const __nv_bfloat162 r =
      __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// The constants come as kernel arguments: as immediates the compiler rebuilds one of them in a
// register before every use.
__device__ __forceinline__ uint32_t and_xor(uint32_t w, uint32_t mask, uint32_t flip) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(r) : "r"(w), "r"(mask), "r"(flip));
  return r;
}

template <typename TT, int BITS>
struct Codes;
template <>
struct Codes<F16, 4> {
  static constexpr Masks kMasks{{0x000F000Fu, 0x64086408u, 0x00F000F0u, 0x64806480u}};
  static __device__ __forceinline__ void pairs(uint32_t w, const Masks& m, uint32_t p[4]) {
    const __half2 sixteenth = __half2half2(__ushort_as_half(0x2C00));  // 2^-4
    const __half2 m72 = __half2half2(__ushort_as_half(0xD480));        // -(64 + 8)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t v = w >> (8 * h);
      p[2 * h] = sub2(and_xor(v, m.k[0], m.k[1]), m.k[1], F16());  // 1024 + (q + 8) - 1032
      const uint32_t b = and_xor(v, m.k[2], m.k[3]);               // 1024 + 16 (q + 8)
      const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&b), sixteenth, m72);
      p[2 * h + 1] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
};
template <>
struct Codes<BF16, 4> {
  static constexpr Masks kMasks{{0x000F000Fu, 0x43084308u, 0u, 0u}};
  static __device__ __forceinline__ void pairs(uint32_t w, const Masks& m, uint32_t p[4]) {
#pragma unroll
    for (int h = 0; h < 4; ++h)  // 128 + (q + 8) - 136
      p[h] = sub2(and_xor(w >> (4 * h), m.k[0], m.k[1]), m.k[1], BF16());
  }
};
template <>
struct Codes<F16, 8> {
  static constexpr Masks kMasks{{0x00FF00FFu, 0x64806480u, 0u, 0u}};
  static __device__ __forceinline__ void pairs(uint32_t w, const Masks& m, uint32_t p[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)  // 1024 + (q + 128) - 1152
      p[h] = sub2(and_xor(w >> (8 * h), m.k[0], m.k[1]), m.k[1], F16());
  }
};
template <>
struct Codes<BF16, 8> {  // bf16 holds 7 bits after the leading one: the sign bit goes apart
  static constexpr Masks kMasks{{0x007F007Fu, 0x43004300u, 0x00800080u, 0u}};
  static __device__ __forceinline__ void pairs(uint32_t w, const Masks& m, uint32_t p[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t v = w >> (8 * h);
      // (128 + low seven bits) - (128, or 256 for a negative code)
      p[h] = sub2(and_xor(v, m.k[0], m.k[1]), and_xor(v, m.k[2], m.k[1]), BF16());
    }
  }
};

// c = A B + d, 16 x 8 x 16, fp32 sums.
#define ZPP_MMA(TYPE)                                                                          \
  asm("mma.sync.aligned.m16n8k16.row.col.f32." TYPE "." TYPE ".f32 {%0,%1,%2,%3}, "            \
      "{%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"                                             \
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])                                         \
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(d[0]), "f"(d[1]),    \
        "f"(d[2]), "f"(d[3]))
__device__ __forceinline__ void mma16816(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1,
                                         const float d[4], F16) {
  ZPP_MMA("f16");
}
__device__ __forceinline__ void mma16816(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1,
                                         const float d[4], BF16) {
  ZPP_MMA("bf16");
}
#undef ZPP_MMA

// ---------------------------------------------------------------------------------
// The kernel for cols a multiple of block. A segment is the columns that 16 code bytes per
// lane cover: 128 of INT4, 64 of INT8. In a segment lane (g, t) (g = lane / 4, t = lane % 4)
// holds a quarter, the columns from t SEG / 4 on, of the rows g and g + 8 of each 16-row
// fragment, and the same columns of the vector in column g of the other operand: the order of
// the columns inside a matrix product is free as long as both operands agree.
//
// The other operand has 8 columns. With fewer vectors (NV = 1, 2, 4) its columns hold them for
// 8 / NV segments at once, so that x costs no more registers, loads and permutations per
// segment than there are vectors; each segment's product is wanted in its own columns only
// (the rest is dropped by a select). A block of 64 is half a segment: then a segment takes
// two columns per vector, each zero in the half that is not its own (SP = 2). A column's
// result is a sum over one block, so it is multiplied by the row's scale and added up in fp32.
//
// A warp loads U segments of its rows before it works on the first. A row's batches of U segments
// are dealt round robin to the warps that share its tile (wk of a CTA's, times `split` CTAs of a
// cluster); their sums are joined in a fixed order through shared memory.
// ---------------------------------------------------------------------------------
template <int BITS, int MT, int NV, int SP, int NT>
struct MvShape {
  static constexpr int SEG = BITS == 4 ? 128 : 64;
  static constexpr int ROWS = 16 * MT, VECS = NV == 8 ? 8 * NT : NV;
  static constexpr int COLS = SEG / 4;                         // columns per lane
  static constexpr int TJ = COLS / 8;                          // 16-byte chunks of x per lane
  static constexpr int PW = 16 / BITS;                         // pairs per word
  static constexpr int SG = NV * SP >= 8 ? 1 : 8 / (NV * SP);  // segments per set of columns
  static constexpr int TILES = NV * SP > 8 ? NT * SP : NT;     // sets of 8 columns
  static_assert(NT == 1 || NV == 8, "more than one set of vectors only when they fill it");
};

template <typename TT, int BITS, int MT, int NV, int SP, int NT, int U>
__global__ void __launch_bounds__(kThreads, 2) k_matvec_mma(const MatvecArgs a, int log2b, int wk,
                                                            int split, const Masks masks) {
  using S = MvShape<BITS, MT, NV, SP, NT>;
  constexpr int SEG = S::SEG, T = S::TILES, NS = NV * SP;
  static_assert(U % S::SG == 0, "whole sets of columns per batch");
  extern __shared__ float part[];  // [kWarps][VECS * ROWS]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int rank = static_cast<int>(blockIdx.x) % split;  // = the CTA's rank in its cluster
  const int wr = kWarps / wk;                             // row tiles of a CTA
  const int64_t row0 = (static_cast<int64_t>(blockIdx.x / split) * wr + warp / wk) * S::ROWS;
  const int64_t vec0 = static_cast<int64_t>(blockIdx.y) * S::VECS;
  const int vecs = static_cast<int>(min(a.vecs - vec0, static_cast<int64_t>(S::VECS)));
  const int segs = static_cast<int>(a.cols / SEG), batches = (segs + U - 1) / U;
  const int step = wk * split;

  // Rows past the end read the last one, vectors past the end the last one: not stored.
  const uint8_t* codes[MT][2];
  const float* scale[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t r = min(row0 + 16 * m + 8 * h + g, a.rows - 1);
      codes[m][h] = a.codes + r * (a.cols * BITS / 8) + t * 16;
      scale[m][h] = a.scales + r * (a.cols >> log2b);
    }
  // Column g of set i: vector, and which segment of its group and half of it.
  const uint16_t* x[T];
  int col_seg = 0;
  bool col_on[T];
#pragma unroll
  for (int i = 0; i < T; ++i) {
    const int slot = NS > 8 ? i % SP : g / NV;  // (segment, half)
    const int v = NS > 8 ? i / SP * 8 + g : NV == 8 ? i * 8 + g : g % NV;
    col_seg = NS > 8 ? 0 : slot / SP;
    col_on[i] = SP == 1 || (t >> 1) == slot % SP;
    x[i] = a.x + (vec0 + min(v, vecs - 1)) * a.x_stride + col_seg * SEG + t * S::COLS;
  }
  const int my_seg = NS >= 8 ? 0 : 2 * t / NS;  // segment of this lane's result columns 2t ..

  float y[MT][T][4] = {};
  for (int b = rank * wk + warp % wk; b < batches; b += step) {
    const int seg0 = b * U, left = segs - seg0;
    uint32_t w[U][MT][2][4];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u < left)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 v = ld_stream_v4(codes[m][h] + static_cast<int64_t>(seg0) * 64 + u * 64);
            w[u][m][h][0] = v.x, w[u][m][h][1] = v.y, w[u][m][h][2] = v.z, w[u][m][h][3] = v.w;
          }
#pragma unroll
    for (int u0 = 0; u0 < U; u0 += S::SG) {  // one set of columns at a time
      if (u0 >= left) break;
      uint32_t f[T][S::TJ][4];  // fragments of x: the pairs that go with the code pairs
#pragma unroll
      for (int i = 0; i < T; ++i)
#pragma unroll
        for (int j = 0; j < S::TJ; ++j) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (col_on[i] && u0 + col_seg < left)
            v = __ldg(reinterpret_cast<const uint4*>(x[i] + static_cast<int64_t>(seg0 + u0) * SEG) + j);
          if constexpr (BITS == 4) {  // pairs (p, p + 4)
            f[i][j][0] = __byte_perm(v.x, v.z, 0x5410u), f[i][j][1] = __byte_perm(v.x, v.z, 0x7632u);
            f[i][j][2] = __byte_perm(v.y, v.w, 0x5410u), f[i][j][3] = __byte_perm(v.y, v.w, 0x7632u);
          } else {  // pairs (p, p + 2) of each four
            f[i][j][0] = __byte_perm(v.x, v.y, 0x5410u), f[i][j][1] = __byte_perm(v.x, v.y, 0x7632u);
            f[i][j][2] = __byte_perm(v.z, v.w, 0x5410u), f[i][j][3] = __byte_perm(v.z, v.w, 0x7632u);
          }
        }
      // scales of this lane's result columns 2t and 2t + 1 (with two vectors or more they lie
      // in one block)
      float sc[MT][2][T][2];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < T; ++i)
#pragma unroll
            for (int e = 0; e < (NV == 1 ? 2 : 1); ++e) {
              const int slot = NS > 8 ? i % SP : (2 * t + e) / NV;
              const int at = seg0 + u0 + (NS > 8 ? 0 : slot / SP);
              const int64_t col = static_cast<int64_t>(min(at, segs - 1)) * SEG + slot % SP * 64;
              sc[m][h][i][e] = __ldg(scale[m][h] + (col >> log2b));
              if (NV > 1) sc[m][h][i][1] = sc[m][h][i][0];
            }
      float r[MT][T][4] = {};
#pragma unroll
      for (int s = 0; s < S::SG; ++s) {
        if (s > 0 && u0 + s >= left) break;
        float c[MT][T][4] = {};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            uint32_t q[2][S::PW];
            Codes<TT, BITS>::pairs(w[u0 + s][m][0][j], masks, q[0]);
            Codes<TT, BITS>::pairs(w[u0 + s][m][1][j], masks, q[1]);
#pragma unroll
            for (int p = 0; p < S::PW; p += 2) {
              const uint32_t fa[4] = {q[0][p], q[1][p], q[0][p + 1], q[1][p + 1]};
              const int fj = j * S::PW / 4, fp = j * S::PW % 4 + p;
#pragma unroll
              for (int i = 0; i < T; ++i)
                mma16816(c[m][i], fa, f[i][fj][fp], f[i][fj][fp + 1], c[m][i], TT());
            }
          }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < T; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (S::SG == 1) r[m][i][k] = c[m][i][k];
              else if (NS == 1) { if ((k & 1) == (s & 1) && t == s >> 1) r[m][i][k] = c[m][i][k]; }
              else if (my_seg == s) r[m][i][k] = c[m][i][k];
            }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < T; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            y[m][i][k] = __fmaf_rn(r[m][i][k], sc[m][k >> 1][i][k & 1], y[m][i][k]);
    }
  }

  // Join: the columns of a vector, the warps of a tile, the CTAs of a cluster.
  constexpr int OUTS = S::VECS * S::ROWS;
  float* mine = part + warp * OUTS;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float* at = mine + 16 * m + 8 * h + g;
      if constexpr (NS > 8) {  // both halves of the segments
#pragma unroll
        for (int i = 0; i < T; i += 2)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            at[(i / 2 * 8 + 2 * t + e) * S::ROWS] = y[m][i][2 * h + e] + y[m][i + 1][2 * h + e];
      } else if constexpr (NV == 8) {
#pragma unroll
        for (int i = 0; i < T; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) at[(i * 8 + 2 * t + e) * S::ROWS] = y[m][i][2 * h + e];
      } else {
        float v[2] = {y[m][0][2 * h], y[m][0][2 * h + 1]};
        if (NV == 1) v[0] += v[1];
#pragma unroll
        for (int e = 0; e < (NV == 1 ? 1 : 2); ++e) {
          if (NV < 4) v[e] += __shfl_xor_sync(~0u, v[e], 1);
          v[e] += __shfl_xor_sync(~0u, v[e], 2);
          if (t < (NV + 1) / 2) at[(2 * t + e) * S::ROWS] = v[e];
        }
      }
    }
  __syncthreads();
  const int outs = wr * OUTS;
  for (int o = threadIdx.x; o < outs; o += kThreads) {
    float* p = part + o / OUTS * wk * OUTS + o % OUTS;
    float sum = *p;
    for (int k = 1; k < wk; ++k) sum += p[k * OUTS];
    *p = sum;  // read and written by this thread only
  }
  if (split > 1) cg::this_cluster().sync();
  if (rank == 0) {
    const int64_t first = static_cast<int64_t>(blockIdx.x / split) * wr * S::ROWS;
    for (int o = threadIdx.x; o < outs; o += kThreads) {
      const int at = o / OUTS * wk * OUTS + o % OUTS, v = o % OUTS / S::ROWS;
      const int64_t r = first + o / OUTS * S::ROWS + o % S::ROWS;
      float sum = part[at];
      for (int k = 1; k < split; ++k) sum += cg::this_cluster().map_shared_rank(part, k)[at];
      if (r < a.rows && v < vecs) {
        if (a.bias) sum += bits16_to_float(__ldg(a.bias + r), TT());
        store_y(a.y, (vec0 + v) * a.y_stride + r, sum, a.y_kind);
      }
    }
  }
  if (split > 1) cg::this_cluster().sync();  // a CTA's sums outlive their readers
}

// Any width: a warp per row and vector, lanes striding over the row's codes.
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

// How a launch splits a product: row fragments and segments in flight per warp, warps of a CTA and
// CTAs that share a row tile.
struct MvPlan {
  int mt, wk, split;
};

template <typename TT, int BITS, int MT, int NV, int SP, int NT, int U>
static cudaError_t run_mma(const MatvecArgs& a, int log2b, const MvPlan& p, cudaStream_t s) {
  using S = MvShape<BITS, MT, NV, SP, NT>;
  const int64_t rows = static_cast<int64_t>(S::ROWS) * (kWarps / p.wk);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.rows + rows - 1) / rows * p.split),
                     static_cast<unsigned>((a.vecs + S::VECS - 1) / S::VECS));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kWarps * S::VECS * S::ROWS * sizeof(float);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = p.split;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = p.split > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k_matvec_mma<TT, BITS, MT, NV, SP, NT, U>, a, log2b, p.wk, p.split,
                            Codes<TT, BITS>::kMasks);
}

template <typename TT, int BITS, int SP>
static cudaError_t by_vecs(const MatvecArgs& a, int log2b, const MvPlan& p, cudaStream_t s) {
  if (a.vecs == 1) return run_mma<TT, BITS, 1, 1, SP, 1, 8>(a, log2b, p, s);
  if (a.vecs == 2) return p.mt == 2 ? run_mma<TT, BITS, 2, 2, SP, 1, 4>(a, log2b, p, s) : run_mma<TT, BITS, 1, 2, SP, 1, 8>(a, log2b, p, s);
  if (a.vecs <= 4) return p.mt == 2 ? run_mma<TT, BITS, 2, 4, SP, 1, 4>(a, log2b, p, s) : run_mma<TT, BITS, 1, 4, SP, 1, 8>(a, log2b, p, s);
  if (a.vecs <= 8) return p.mt == 2 ? run_mma<TT, BITS, 2, 8, SP, 1, 4>(a, log2b, p, s) : run_mma<TT, BITS, 1, 8, SP, 1, 4>(a, log2b, p, s);
  return p.mt == 2 ? run_mma<TT, BITS, 2, 8, SP, 2, 2>(a, log2b, p, s) : run_mma<TT, BITS, 1, 8, SP, 2, 4>(a, log2b, p, s);
}

template <typename TT>
static cudaError_t by_codes(const MatvecArgs& a, int log2b, const MvPlan& p, cudaStream_t s) {
  if (a.bits == 8) return by_vecs<TT, 8, 1>(a, log2b, p, s);
  return a.block == 64 ? by_vecs<TT, 4, 2>(a, log2b, p, s) : by_vecs<TT, 4, 1>(a, log2b, p, s);
}

static cudaError_t launch_mma(const MatvecArgs& a, int log2b, const MvPlan& p, cudaStream_t s) {
  return a.x_bf16 ? by_codes<BF16>(a, log2b, p, s) : by_codes<F16>(a, log2b, p, s);
}

cudaError_t launch_matvec(const MatvecArgs& a, cudaStream_t s) {
  const int log2b = __builtin_ctz(static_cast<unsigned>(a.block));
  if (a.cols % a.block == 0 && a.x_stride % 8 == 0 && (a.bits == 8 || a.cols % 128 == 0)) {
    return launch_mma(a, log2b, MvPlan{a.vecs == 1 ? 1 : 2, 8, 1}, s);
  }
  const dim3 grid(tile_grid(a.rows, kWarps), static_cast<unsigned>(a.vecs));
  if (a.x_bf16) k_matvec<BF16><<<grid, kThreads, 0, s>>>(a, log2b);
  else k_matvec<F16><<<grid, kThreads, 0, s>>>(a, log2b);
  return cudaGetLastError();
}

}  // namespace zpp
