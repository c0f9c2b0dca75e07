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
// of an INT8 word (p, p + 2): the two halves of a 32-bit word, so masks serve both at once.
// The logic operation puts the code, its sign bit flipped (q + 8 or q + 128), into the low
// mantissa bits of a power of two whose spacing is 1, and the subtraction is exact.
// ---------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t and_xor(uint32_t w, uint32_t mask, uint32_t flip) {
  return (w & mask) ^ flip;
}
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b, F16) {
  const __half2 r = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b, BF16) {
  const __nv_bfloat162 r =
      __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <typename TT, int BITS>
struct Codes;

template <>
struct Codes<F16, 4> {
  static __device__ __forceinline__ void pairs(uint32_t w, uint32_t p[4]) {
    const uint32_t one = 0x64086408u;                          // 1024 ^ 8
    const uint32_t off = 0x64086408u;                          // 1032
    const __half2 sixteenth = __half2half2(__ushort_as_half(0x2C00));  // 2^-4
    const __half2 m72 = __half2half2(__ushort_as_half(0xD480));        // -(64 + 8)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t v = w >> (8 * h);
      p[2 * h] = sub2(and_xor(v, 0x000F000Fu, one), off, F16());
      // 1024 + 16 (q + 8), so / 16 - 72
      const uint32_t b = and_xor(v, 0x00F000F0u, 0x64806480u);
      const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&b), sixteenth, m72);
      p[2 * h + 1] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
};
template <>
struct Codes<BF16, 4> {
  static __device__ __forceinline__ void pairs(uint32_t w, uint32_t p[4]) {
#pragma unroll
    for (int h = 0; h < 4; ++h)  // 128 + (q + 8) - 136
      p[h] = sub2(and_xor(w >> (4 * h), 0x000F000Fu, 0x43084308u), 0x43084308u, BF16());
  }
};
template <>
struct Codes<F16, 8> {
  static __device__ __forceinline__ void pairs(uint32_t w, uint32_t p[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)  // 1024 + (q + 128) - 1152
      p[h] = sub2(and_xor(w >> (8 * h), 0x00FF00FFu, 0x64806480u), 0x64806480u, F16());
  }
};
template <>
struct Codes<BF16, 8> {  // bf16 holds 7 bits after the leading one: the sign bit goes apart
  static __device__ __forceinline__ void pairs(uint32_t w, uint32_t p[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t v = w >> (8 * h);
      // (128 + low seven bits) - (128, or 256 for a negative code)
      p[h] = sub2(and_xor(v, 0x007F007Fu, 0x43004300u), and_xor(v, 0x00800080u, 0x43004300u), BF16());
    }
  }
};

__device__ __forceinline__ void mma16816(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1,
                                         F16) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1,
                                         BF16) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// WORDS consecutive 32-bit code words of a lane.
template <int WORDS>
__device__ __forceinline__ void ld_words(const uint8_t* p, uint32_t w[WORDS]) {
  if constexpr (WORDS == 4) {
    const uint4 v = ld_stream_v4(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else {
    const uint2 v = ld_stream_v2(p);
    w[0] = v.x, w[1] = v.y;
  }
}

// ---------------------------------------------------------------------------------
// The kernel for cols a multiple of block. A warp takes segments of SEG columns of 16 MT
// rows. In a segment lane (g, t) (g = lane / 4, t = lane % 4) holds SEG / 4 consecutive columns,
// starting at t SEG / 4, of the rows g and g + 8 of each fragment, and the same columns of
// vector g: the order of the columns inside a matrix product is free as long as both
// operands agree. A segment lies in one block, so its fp32 sum is multiplied by the row's scale
// and added to the running one. Segments are dealt round robin to the warps of a CTA and to
// the CTAs of a cluster; their sums are joined in a fixed order through shared memory.
// ---------------------------------------------------------------------------------
template <typename TT, int BITS, int SEG, int MT, int NT>
struct Seg {
  static constexpr int COLS = SEG / 4;          // columns per lane
  static constexpr int WORDS = COLS * BITS / 32;
  static constexpr int PAIRS = COLS / 2;
  uint32_t w[MT][2][WORDS];
  float s[MT][2];
  __device__ __forceinline__ void load(const uint8_t* const (&row)[MT][2],
                                       const int64_t (&first)[MT][2],
                                       const float* __restrict__ scales, int log2b, int64_t seg) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        ld_words<WORDS>(row[m][h] + seg * (SEG * BITS / 8), w[m][h]);
        s[m][h] = __ldg(scales + ((first[m][h] + seg * SEG) >> log2b));
      }
  }
  // x: this lane's columns of the segment in vector g of the first tile (tiles are 8 vectors
  // apart); use[n]: whether that vector exists.
  __device__ __forceinline__ void add(const uint16_t* x, int64_t tile_stride, const bool (&use)[NT],
                                      float (&y)[MT][NT][4]) const {
    uint32_t xw[NT][PAIRS];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < PAIRS / 4; ++k) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (use[n]) v = __ldg(reinterpret_cast<const uint4*>(x + n * tile_stride) + k);
        xw[n][4 * k] = v.x, xw[n][4 * k + 1] = v.y, xw[n][4 * k + 2] = v.z, xw[n][4 * k + 3] = v.w;
      }
    float c[MT][NT][4] = {};
    constexpr int PW = 16 / BITS;  // pairs per word: 4 (INT4), 2 (INT8)
#pragma unroll
    for (int j = 0; j < WORDS; ++j) {
      uint32_t b[NT][PW];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int p = 0; p < PW; p += 2) {  // pairs (p, p + PW) and (p + 1, p + 1 + PW)
          const uint32_t lo = xw[n][j * PW + p / 2], hi = xw[n][j * PW + (p + PW) / 2];
          b[n][p] = __byte_perm(lo, hi, 0x5410u);
          b[n][p + 1] = __byte_perm(lo, hi, 0x7632u);
        }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        uint32_t q[2][PW];
        Codes<TT, BITS>::pairs(w[m][0][j], q[0]);
        Codes<TT, BITS>::pairs(w[m][1][j], q[1]);
#pragma unroll
        for (int p = 0; p < PW; p += 2) {
          const uint32_t f[4] = {q[0][p], q[1][p], q[0][p + 1], q[1][p + 1]};
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816(c[m][n], f, b[n][p], b[n][p + 1], TT());
        }
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        y[m][n][0] = __fmaf_rn(c[m][n][0], s[m][0], y[m][n][0]);
        y[m][n][1] = __fmaf_rn(c[m][n][1], s[m][0], y[m][n][1]);
        y[m][n][2] = __fmaf_rn(c[m][n][2], s[m][1], y[m][n][2]);
        y[m][n][3] = __fmaf_rn(c[m][n][3], s[m][1], y[m][n][3]);
      }
  }
};

template <typename TT, int BITS, int SEG, int MT, int NT>
__global__ void __launch_bounds__(kThreads) k_matvec_mma(const MatvecArgs a, int log2b, int split) {
  constexpr int ROWS = 16 * MT, VECS = 8 * NT;
  extern __shared__ float part[];  // [warps][VECS][ROWS]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int rank = static_cast<int>(blockIdx.x) % split;  // = the CTA's rank in its cluster
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / split) * ROWS;
  const int64_t vec0 = static_cast<int64_t>(blockIdx.y) * VECS;
  const int vecs = static_cast<int>(min(a.vecs - vec0, static_cast<int64_t>(VECS)));

  const uint8_t* row[MT][2];
  int64_t first[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // rows past the end read the last one; not stored
      const int64_t r = min(row0 + 16 * m + 8 * h + g, a.rows - 1);
      first[m][h] = r * a.cols;
      row[m][h] = a.codes + r * a.cols * BITS / 8 + t * (SEG / 4) * BITS / 8;
    }
  bool use[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) use[n] = 8 * n + g < vecs;
  const uint16_t* x = a.x + (vec0 + g) * a.x_stride + t * (SEG / 4);

  float y[MT][NT][4] = {};
  const int64_t segs = a.cols / SEG, step = static_cast<int64_t>(warps) * split;
  int64_t i = static_cast<int64_t>(rank) * warps + warp;
  if (i < segs) {
    Seg<TT, BITS, SEG, MT, NT> now, next;
    now.load(row, first, a.scales, log2b, i);
    for (; i + step < segs; i += step) {
      next.load(row, first, a.scales, log2b, i + step);
      now.add(x + i * SEG, 8 * a.x_stride, use, y);
      now = next;
    }
    now.add(x + i * SEG, 8 * a.x_stride, use, y);
  }

#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int v = 8 * n + 2 * t + (k & 1);
        if (v < vecs) part[(warp * VECS + v) * ROWS + 16 * m + 8 * (k >> 1) + g] = y[m][n][k];
      }
  __syncthreads();
  for (int o = threadIdx.x; o < vecs * ROWS; o += blockDim.x) {
    float sum = part[o];
    for (int w = 1; w < warps; ++w) sum += part[w * VECS * ROWS + o];
    part[o] = sum;  // read and written by this thread only
  }
  if (split > 1) cg::this_cluster().sync();
  if (rank == 0) {
    for (int o = threadIdx.x; o < vecs * ROWS; o += blockDim.x) {
      float sum = part[o];
      for (int r = 1; r < split; ++r) sum += cg::this_cluster().map_shared_rank(part, r)[o];
      const int64_t r = row0 + o % ROWS;
      if (r < a.rows) {
        if (a.bias) sum += bits16_to_float(__ldg(a.bias + r), TT());
        store_y(a.y, (vec0 + o / ROWS) * a.y_stride + r, sum, a.y_kind);
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

template <typename TT, int BITS, int SEG, int MT, int NT>
static cudaError_t run_mma(const MatvecArgs& a, int log2b, int warps, int split, cudaStream_t s) {
  constexpr int ROWS = 16 * MT, VECS = 8 * NT;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.rows + ROWS - 1) / ROWS * split),
                     static_cast<unsigned>((a.vecs + VECS - 1) / VECS));
  cfg.blockDim = dim3(32 * warps);
  cfg.dynamicSmemBytes = static_cast<size_t>(warps) * ROWS * VECS * sizeof(float);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = split;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_matvec_mma<TT, BITS, SEG, MT, NT>, a, log2b, split);
}

template <typename TT, int BITS, int SEG, int MT>
static cudaError_t by_vecs(const MatvecArgs& a, int log2b, int warps, int split, cudaStream_t s) {
  if (a.vecs <= 8) return run_mma<TT, BITS, SEG, MT, 1>(a, log2b, warps, split, s);
  if (a.vecs <= 16) return run_mma<TT, BITS, SEG, MT, 2>(a, log2b, warps, split, s);
  return run_mma<TT, BITS, SEG, MT, 4>(a, log2b, warps, split, s);
}

template <typename TT, int MT>
static cudaError_t by_codes(const MatvecArgs& a, int log2b, int warps, int split, cudaStream_t s) {
  if (a.bits == 8) return by_vecs<TT, 8, 64, MT>(a, log2b, warps, split, s);
  if (a.block == 64) return by_vecs<TT, 4, 64, MT>(a, log2b, warps, split, s);
  return by_vecs<TT, 4, 128, MT>(a, log2b, warps, split, s);
}

static cudaError_t launch_mma(const MatvecArgs& a, int log2b, int mt, int warps, int split,
                              cudaStream_t s) {
  if (a.x_bf16)
    return mt == 2 ? by_codes<BF16, 2>(a, log2b, warps, split, s)
                   : by_codes<BF16, 1>(a, log2b, warps, split, s);
  return mt == 2 ? by_codes<F16, 2>(a, log2b, warps, split, s)
                 : by_codes<F16, 1>(a, log2b, warps, split, s);
}

cudaError_t launch_matvec(const MatvecArgs& a, cudaStream_t s) {
  const int log2b = __builtin_ctz(static_cast<unsigned>(a.block));
  if (a.cols % a.block == 0 && a.x_stride % 8 == 0) {
    const int64_t tiles = (a.rows + 15) / 16;
    int split = 1;
    while (split < 8 && tiles * split < 2 * 152) split *= 2;
    return launch_mma(a, log2b, 1, 8, split, s);
  }
  const dim3 grid(tile_grid(a.rows, kWarps), static_cast<unsigned>(a.vecs));
  if (a.x_bf16) k_matvec<BF16><<<grid, kThreads, 0, s>>>(a, log2b);
  else k_matvec<F16><<<grid, kThreads, 0, s>>>(a, log2b);
  return cudaGetLastError();
}

}  // namespace zpp
