// matvec.cu -- K9: y = x W^T (+ bias) straight from block-quantised codes.
//
//   y[j][r] = sum_c q[r][c] scale[(r cols + c) / block] x[j][c] + bias[r]
//
// Memory-bound in principle: the codes are read once for up to 16 vectors. What bounds it first is
// the work per code, so the products go to the matrix unit: codes become exact fp16 / bf16
// integers with one logic and one half-precision operation per two, a fragment of 16 rows meets
// 8 vectors, and products (exact) and sums are fp32. (The warp-level matrix instruction, since one
// vector fills an eighth of even its tile: what counts is that codes go from registers to the unit.)
//
// Measured (us; bytes at 6.78 TB/s in brackets): 24576 x 8192 INT4, one vector 24.9 (15.8); 8192 x
// 32768 INT4, 8 vectors 38.2 (20.4); 8192 x 8192 INT8 13.1 (9.9); 50001 x 1003 INT4, 3 vectors, rows
// that start inside words 15.7 (4.3); 1024 x 1024 3.9, which is the launch. Loads alone, in this
// pattern, take 17 us for the first. In the rest no unit is saturated (issue slots 52 % busy, the
// matrix unit 26 %): a warp waits for its own chain from shared memory through the conversion to
// the matrix unit, and two CTAs of 124 registers fit an SM, four warps per scheduler. (Whether more
// warps of fewer registers would be faster has not been measured.) The times beside the rules
// below are of captured graphs, weights beyond L2.
#include <cooperative_groups.h>

#include <algorithm>

#include "zpp_device.cuh"
#include "zpp_launch.h"
#include "zpp_overlap.cuh"

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
// The constants come as kernel arguments. (As immediates 24576 x 8192 INT4 takes 24.2 us with one
// vector, 38.5 with eight, so 24.6 and 37.8; 8192 x 32768, 8 vectors 36.7, so 37.8.)
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
// The kernel for cols a multiple of a segment, the columns that 16 code bytes per lane cover: 128
// of INT4, 64 of INT8 (so that a segment lies in one block, or is two of 64). In a segment lane (g,
// t) (g = lane / 4, t = lane % 4) holds a quarter, the columns from t SEG / 4 on, of the rows g and
// g + 8 of each 16-row fragment, and the same columns of the vector in column g of the other
// operand: the order of the columns inside a matrix product is free as long as both operands agree.
//
// The other operand has 8 columns. With fewer vectors (NV = 1, 2, 4) its columns hold them for
// 8 / NV segments at once, so that x costs no more registers, loads and permutations per
// segment than there are vectors; each segment's product is wanted in its own columns only
// (the rest is dropped by a select). A block of 64 is half a segment: then a segment takes
// two columns per vector, each zero in the half that is not its own (SP = 2). A column's
// result is a sum over one block, so it is multiplied by the row's scale and added up in fp32.
//
// A row's units of kUnit segments are dealt round robin to the warps that share its tile (wk of a
// CTA's, times `split` CTAs of a cluster); their sums are joined in a fixed order through shared
// memory. The code bytes of the next U segments are always on their way into shared memory
// (cp.async, so they hold no registers); a lane reads back only what it copied itself, so the
// loop has no barrier.
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
  static constexpr int UNIT = SG > 8 / MT ? SG : 8 / MT;       // segments dealt at a time
  static constexpr int SEG_BYTES = 2 * MT * 32 * 16;           // code bytes of a warp's segment
  static_assert(NT == 1 || NV == 8, "more than one set of vectors only when they fill it");
  static_assert(UNIT % SG == 0, "whole sets of columns per unit");
};

__device__ __forceinline__ uint4 ld_shared_v4(unsigned p) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(p));
  return r;
}

template <typename TT, int BITS, int MT, int NV, int SP, int NT, int U>
__global__ void __launch_bounds__(kThreads, MT == 1 && NT == 1 ? 3 : 2)
    k_matvec_mma(const MatvecArgs a, int log2b, int wk, int split, const Masks masks) {
  using S = MvShape<BITS, MT, NV, SP, NT>;
  constexpr int SEG = S::SEG, T = S::TILES, NS = NV * SP, UNIT = S::UNIT;
  static_assert(UNIT % U == 0, "a segment's place in the ring is known at compile time");
  extern __shared__ __align__(16) uint8_t smem[];  // [kWarps][U segments]; later the sums
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int rank = static_cast<int>(blockIdx.x) % split;  // = the CTA's rank in its cluster
  const int wr = kWarps / wk;                             // row tiles of a CTA
  const int64_t row0 = (static_cast<int64_t>(blockIdx.x / split) * wr + warp / wk) * S::ROWS;
  const int64_t vec0 = static_cast<int64_t>(blockIdx.y) * S::VECS;
  const int vecs = static_cast<int>(min(a.vecs - vec0, static_cast<int64_t>(S::VECS)));
  const int segs = static_cast<int>(a.cols / SEG), units = (segs + UNIT - 1) / UNIT;
  const int step = wk * split, unit0 = rank * wk + warp % wk;

  // Rows past the end read the last one, vectors past the end the last one: not stored.
  const uint8_t* codes[MT][2];
  const float* scale[MT][2];
  unsigned in_block[MT][2];  // where in its block a row begins (blocks of 64, SP = 2: at 0)
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t r = min(row0 + 16 * m + 8 * h + g, a.rows - 1);
      codes[m][h] = a.codes + r * (a.cols * BITS / 8) + static_cast<int64_t>(unit0) * (UNIT * 64) + t * 16;
      scale[m][h] = a.scales + (r * a.cols >> log2b);
      in_block[m][h] = static_cast<unsigned>(r * a.cols) & ((1u << log2b) - 1);
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

  const unsigned ring = smem_addr(smem) + warp * (U * S::SEG_BYTES) + lane * 16;
  // Segment `at` of this warp's unit number n, into its place.
  auto fill = [&](int n, int at) {
    const int seg = (unit0 + n * step) * UNIT + at;
    if (seg < segs)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                           ring + at % U * S::SEG_BYTES + (2 * m + h) * 512),
                       "l"(codes[m][h] + static_cast<int64_t>(n) * step * (UNIT * 64) + at * 64)
                       : "memory");
    cp_async_commit();
  };
  grid_wait();
  grid_release();
#pragma unroll
  for (int u = 0; u < U; ++u) fill(0, u);

  float y[MT][T][4] = {};
  for (int n = 0; unit0 + n * step < units; ++n) {
    const int seg0 = (unit0 + n * step) * UNIT, left = segs - seg0;
#pragma unroll
    for (int u0 = 0; u0 < UNIT; u0 += S::SG) {  // one set of columns at a time
      if (u0 >= left) break;
      uint32_t f[T][S::TJ][4];  // fragments of x: the pairs that go with the code pairs
#pragma unroll
      for (int i = 0; i < T; ++i)
#pragma unroll
        for (int j = 0; j < S::TJ; ++j) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (col_on[i] && u0 + col_seg < left)
            v = ld_after_shared_v4(x[i] + static_cast<int64_t>(seg0 + u0) * SEG + 8 * j);
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
              const unsigned col =
                  static_cast<unsigned>(at) * SEG + slot % SP * 64 + (SP == 1 ? in_block[m][h] : 0u);
              // beyond the row 0, not another block's scale: that may be infinite
              sc[m][h][i][e] = at < segs ? ld_after_f32(scale[m][h] + (col >> log2b)) : 0.0f;
              if (NV > 1) sc[m][h][i][1] = sc[m][h][i][0];
            }
      float r[MT][T][4] = {};
#pragma unroll
      for (int s = 0; s < S::SG; ++s) {
        if (s > 0 && u0 + s >= left) break;
        cp_async_wait<U - 1>();
        uint32_t w[MT][2][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 v = ld_shared_v4(ring + (u0 + s) % U * S::SEG_BYTES + (2 * m + h) * 512);
            w[m][h][0] = v.x, w[m][h][1] = v.y, w[m][h][2] = v.z, w[m][h][3] = v.w;
          }
        float c[MT][T][4] = {};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            uint32_t q[2][S::PW];
            Codes<TT, BITS>::pairs(w[m][0][j], masks, q[0]);
            Codes<TT, BITS>::pairs(w[m][1][j], masks, q[1]);
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
        // the segment's place is free (its codes have been used)
        if (u0 + s + U < UNIT) fill(n, u0 + s + U);
        else fill(n + 1, u0 + s + U - UNIT);
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

  // Join: the columns of a vector, the warps of a tile, the CTAs of a cluster. The warp's sums
  // replace its codes, all of which have landed and been used.
  cp_async_wait<0>();
  __syncwarp();
  constexpr int OUTS = S::VECS * S::ROWS, STRIDE = U * S::SEG_BYTES / 4;
  static_assert(OUTS <= STRIDE, "the sums fit into the ring");
  float* part = reinterpret_cast<float*>(smem);
  float* mine = part + warp * STRIDE;
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
    float* p = part + o / OUTS * wk * STRIDE + o % OUTS;
    float sum = *p;
    for (int k = 1; k < wk; ++k) sum += p[k * STRIDE];
    *p = sum;  // read and written by this thread only
  }
  if (split > 1) cg::this_cluster().sync();
  if (rank == 0) {
    const int64_t first = static_cast<int64_t>(blockIdx.x / split) * wr * S::ROWS;
    for (int o = threadIdx.x; o < outs; o += kThreads) {
      const int at = o / OUTS * wk * STRIDE + o % OUTS, v = o % OUTS / S::ROWS;
      const int64_t r = first + o / OUTS * S::ROWS + o % S::ROWS;
      float sum = part[at];
      for (int k = 1; k < split; ++k) sum += cg::this_cluster().map_shared_rank(part, k)[at];
      if (r < a.rows && v < vecs) {
        if (a.bias) sum += bits16_to_float(ld_after_u16(a.bias + r), TT());
        store_y(a.y, (vec0 + v) * a.y_stride + r, sum, a.y_kind);
      }
    }
  }
  if (split > 1) cg::this_cluster().sync();  // a CTA's sums outlive their readers
}

// ---------------------------------------------------------------------------------
// Any width, any stride of x: rows start inside a block, a word, a byte. The codes are read by
// aligned chunks of 16 bytes (32 or 16 codes, one block each). A row whose first code is number s
// of its chunk meets x shifted by s columns, with zeros beyond both ends for its neighbours'
// codes; rows CH apart (CH codes a chunk) have the same s. So a CTA takes rows of one s only and a
// fragment is 16 of them CH apart. Where rows start at words (WORDS: the width and x's stride are
// multiples of 8 INT4, 4 INT8 columns) a lane reads its words of x where they are; else x is laid
// out in shared memory, shifted, as fragments, by each CTA, which costs more than the products from
// four vectors on. (24576 x 8224 INT4, 1 / 8 vectors: in place 43 / 46 us, laid out 39 / 55; 2861 x
// 20896: 22 / 23 and 22 / 39; 5120 x 1288 INT8: 6.5 / 6.7 and 6.7 / 12.) Blocks begin at other
// columns in every row, so a product covers one chunk and is scaled per row and chunk; lane (g, t)
// takes word t of the chunks of rows g and g + 8. Two sets of 8 vectors share the codes where there
// are more than 8 (NT = 2: 24576 x 8224, 16 vectors 61 us from 80; its INT4 form with x in place
// spills 16 to 20 bytes per lane, the BF16 INT4 form of NT = 1 with x laid out 8).
//
// A stage is four chunks of a warp's 16 rows; a lane copies chunk t of its two rows, and its
// scales, but reads word t of all four (the copies are swapped so that this is free of bank
// conflicts). Stages are dealt round robin as in k_matvec_mma.
// ---------------------------------------------------------------------------------
template <int BITS>
struct AnyShape {
  static constexpr int CH = 128 / BITS;      // codes per chunk, rows apart with one shift
  static constexpr int WC = 32 / BITS;       // codes (columns) per word
  static constexpr int PW = 16 / BITS;       // pairs per word
  static constexpr int XB = WC * 2;          // bytes of a word's columns of x
  static constexpr int STAGE = 2 * 512 + 2 * 128;  // codes, scales
  static constexpr int DEPTH = 3;            // stages on their way (with 4: 50001 x 1003 16.7 us, not 15.9)
  static constexpr int RING = DEPTH * STAGE;
};
// Stages of a row and a CTA's share of them (at most, over its warps and ranks).
__host__ __device__ inline int any_stages(int64_t cols, int ch) {
  return static_cast<int>(((cols + 2 * ch - 2) / ch + 3) / 4);
}
__host__ __device__ inline int any_share(int64_t cols, int ch, int wk, int split) {
  const int step = wk * split;
  return (any_stages(cols, ch) + step - 1) / step * wk;
}

template <typename TT, int BITS, bool WORDS, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 4 : 3)
    k_matvec_any(const MatvecArgs a, int log2b, int wk, int split, const Masks masks) {
  using S = AnyShape<BITS>;
  constexpr int CH = S::CH;
  extern __shared__ __align__(16) uint8_t smem[];  // [kWarps] rings (later sums), then x
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int log2wk = __popc(wk - 1), log2split = __popc(split - 1);  // both powers of two
  const int rank = static_cast<int>(blockIdx.x) & (split - 1);
  const int cta = static_cast<int>(blockIdx.x) >> log2split;
  const int wr = kWarps >> log2wk;  // row tiles of a CTA
  // Rows rho + CH i of this CTA, 16 i per tile.
  const int rho = cta % CH;
  const int64_t tile = static_cast<int64_t>(cta / CH) * wr + (warp >> log2wk);
  const int64_t row0 = rho + tile * (16 * CH);
  const int64_t vec0 = static_cast<int64_t>(blockIdx.y) * (8 * NT);
  const int vecs = static_cast<int>(min(a.vecs - vec0, static_cast<int64_t>(8 * NT)));
  const unsigned cols = static_cast<unsigned>(a.cols);  // less than 2^31
  const int shift = static_cast<int>(rho * a.cols % CH);
  const int chunks = static_cast<int>((a.cols + shift + CH - 1) / CH), stages = (chunks + 3) / 4;
  const int step = wk * split, first = rank * wk + (warp & (wk - 1));
  const int64_t bytes = (a.rows * a.cols * BITS + 7) / 8;  // of all codes
  const int sh = log2b - (BITS == 4 ? 5 : 4);               // log2 of chunks per block
  const bool live = rho < a.rows;                           // (a CTA without rows writes nothing)

  // The next stage to copy: chunk number `to` (in its rows) of this lane's two rows.
  const unsigned ring = smem_addr(smem) + warp * S::RING;
  const unsigned put = ring + g * 64 + ((t ^ ((g >> 1) & 3)) * 16);
  const uint8_t* codes[2];
  const float* scales[2];
  int in_block[2], short_at[2];  // the last chunk of all may end early
#pragma unroll
  for (int h = 0; h < 2; ++h) {  // rows past the end read the first one of this shift; not stored
    int64_t r = row0 + (8 * h + g) * CH;
    if (r >= a.rows) r = min(static_cast<int64_t>(rho), a.rows - 1);
    const int64_t at = r * a.cols / CH;  // chunk of all codes that holds the row's first code
    codes[h] = a.codes + (at + first * 4 + t) * 16;
    scales[h] = a.scales + (at >> sh);
    in_block[h] = static_cast<int>(at & ((1 << sh) - 1));
    short_at[h] = static_cast<int>(min(bytes / 16 - at, static_cast<int64_t>(chunks)));
  }
  const int short_bytes = static_cast<int>(bytes % 16);
  int to = first * 4 + t;
  unsigned to_slot = 0;
  auto fill = [&] {
    const bool on = live && to < chunks;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // (zeros for what is not there; of those nothing is read)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(put + to_slot + h * 512),
                   "l"(codes[h]), "r"(on ? (to == short_at[h] ? short_bytes : 16) : 0)
                   : "memory");
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                       ring + to_slot + 1024 + h * 128 + lane * 4),
                   "l"(scales[h] + (on ? (in_block[h] + to) >> sh : 0)), "r"(on ? 4 : 0)
                   : "memory");
      codes[h] += step * 64;
    }
    to += step * 4;
    to_slot = to_slot == (S::DEPTH - 1) * S::STAGE ? 0 : to_slot + S::STAGE;
    cp_async_commit();
  };
  grid_wait();
  grid_release();
#pragma unroll
  for (int n = 0; n < S::DEPTH - 1; ++n) fill();

  // x as fragments: unit (stage l of the CTA's share, chunk c of it, vector v, t) holds the pairs of
  // columns that go with the code pairs of word t.
  uint8_t* const frag = smem + kWarps * S::RING;
  if constexpr (!WORDS) {
    const int units = ((stages + step - 1) >> (log2wk + log2split) << log2wk) * 16;
    int i = threadIdx.x, v = 0;
    auto settle = [&] {
      while (i >= units) i -= units, ++v;
    };
    settle();
    while (v < vecs) {
      const unsigned l = i >> 4, c = i >> 2 & 3;
      const unsigned stage = rank * wk + (l >> log2wk) * step + (l & (wk - 1));
      const unsigned col = (stage * 4 + c) * CH + (i & 3) * S::WC - shift;  // below 0: above cols
      const uint16_t* x = a.x + (vec0 + v) * a.x_stride;
      uint32_t e[S::WC];
#pragma unroll
      for (int j = 0; j < S::WC; ++j) e[j] = col + j < cols ? ld_after_u16(x + (col + j)) : 0u;
      uint32_t* to_x = reinterpret_cast<uint32_t*>(frag + ((i >> 2) * vecs + v) * (4 * S::XB)) +
                       (i & 3) * (S::XB / 4);
#pragma unroll
      for (int p = 0; p < S::PW; ++p) to_x[p] = e[p] | e[p + S::PW] << 16;
      i += kThreads;
      settle();
    }
    __syncthreads();
  }

  // Where this lane reads: word t of the chunks of rows g and g + 8, the scales of row g, x.
  const uint8_t* const mine = smem + warp * S::RING + g * 64 + t * 4;
  int word[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) word[c] = (c ^ ((g >> 1) & 3)) * 16;
  const uint8_t* xs[NT];
  const uint16_t* xg[NT];
  unsigned col = first * 4 * CH + t * S::WC - shift;
#pragma unroll
  for (int k = 0; k < NT; ++k) {
    const int v = min(8 * k + g, vecs - 1);
    xs[k] = frag + (warp & (wk - 1)) * (16 * vecs * S::XB) + (v * 4 + t) * S::XB;
    xg[k] = a.x + (vec0 + v) * a.x_stride + static_cast<int>(col);
  }

  float y[NT][4] = {};
  int slot = 0;
  for (int stage = first; stage < stages; stage += step) {
    uint4 xw[NT][4];
    if constexpr (WORDS) {
#pragma unroll
      for (int k = 0; k < NT; ++k) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const bool on = 8 * k + g < vecs && col + c * CH < cols;
          xw[k][c] = make_uint4(0u, 0u, 0u, 0u);
          if constexpr (BITS == 4) ld_after_shared_v4_if(on, xg[k] + c * CH, xw[k][c]);
          else ld_after_shared_v2_if(on, xg[k] + c * CH, xw[k][c]);
        }
        xg[k] += step * 4 * CH;
      }
      col += step * 4 * CH;
    }
    cp_async_wait<S::DEPTH - 2>();
    __syncwarp();  // all lanes' copies of this stage have landed, the one before is free
    fill();
    float sc[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 v = *reinterpret_cast<const float4*>(smem + warp * S::RING + slot + 1024 + h * 128 +
                                                        g * 16);
      sc[h][0] = v.x, sc[h][1] = v.y, sc[h][2] = v.z, sc[h][3] = v.w;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t q[2][S::PW];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        Codes<TT, BITS>::pairs(*reinterpret_cast<const uint32_t*>(mine + slot + word[c] + h * 512), masks,
                               q[h]);
#pragma unroll
      for (int k = 0; k < NT; ++k) {
        uint32_t b[S::PW];
        const uint4& w = xw[k][c];
        if constexpr (!WORDS) {
          if constexpr (BITS == 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(xs[k] + c * (vecs * 4 * S::XB));
            b[0] = v.x, b[1] = v.y, b[2] = v.z, b[3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(xs[k] + c * (vecs * 4 * S::XB));
            b[0] = v.x, b[1] = v.y;
          }
        } else if constexpr (BITS == 4) {
          b[0] = __byte_perm(w.x, w.z, 0x5410u), b[1] = __byte_perm(w.x, w.z, 0x7632u);
          b[2] = __byte_perm(w.y, w.w, 0x5410u), b[3] = __byte_perm(w.y, w.w, 0x7632u);
        } else {
          b[0] = __byte_perm(w.x, w.y, 0x5410u), b[1] = __byte_perm(w.x, w.y, 0x7632u);
        }
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int p = 0; p < S::PW; p += 2) {
          const uint32_t f[4] = {q[0][p], q[1][p], q[0][p + 1], q[1][p + 1]};
          mma16816(d, f, b[p], b[p + 1], d, TT());
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) y[k][e] = __fmaf_rn(d[e], sc[e >> 1][c], y[k][e]);
      }
    }
#pragma unroll
    for (int k = 0; k < NT; ++k) xs[k] += wk * (16 * vecs * S::XB);
    slot = slot == (S::DEPTH - 1) * S::STAGE ? 0 : slot + S::STAGE;
  }

  cp_async_wait<0>();
  __syncwarp();
  constexpr int STRIDE = S::RING / 4, OUTS = 128 * NT;
  static_assert(OUTS <= STRIDE, "the sums fit into the ring");
  float* part = reinterpret_cast<float*>(smem);  // a warp's [8 NT][16] sums over its ring
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      part[warp * STRIDE + (8 * n + 2 * t + (k & 1)) * 16 + 8 * (k >> 1) + g] = y[n][k];
  __syncthreads();
  const int outs = wr * OUTS;
  for (int o = threadIdx.x; o < outs; o += kThreads) {
    float* p = part + o / OUTS * wk * STRIDE + o % OUTS;
    float sum = *p;
    for (int k = 1; k < wk; ++k) sum += p[k * STRIDE];
    *p = sum;  // read and written by this thread only
  }
  if (split > 1) cg::this_cluster().sync();
  if (rank == 0) {
    for (int o = threadIdx.x; o < outs; o += kThreads) {
      const int from = o / OUTS * wk * STRIDE + o % OUTS, v = o % OUTS / 16;
      const int64_t r =
          rho + ((static_cast<int64_t>(cta / CH) * wr + o / OUTS) * 16 + o % 16) * CH;
      float sum = part[from];
      for (int k = 1; k < split; ++k) sum += cg::this_cluster().map_shared_rank(part, k)[from];
      if (r < a.rows && v < vecs) {
        if (a.bias) sum += bits16_to_float(ld_after_u16(a.bias + r), TT());
        store_y(a.y, (vec0 + v) * a.y_stride + r, sum, a.y_kind);
      }
    }
  }
  if (split > 1) cg::this_cluster().sync();  // a CTA's sums outlive their readers
}

// Rows so long that a cluster's shared memory cannot hold x (beyond some 700,000 columns): one warp
// per row and vector, x from global memory.
template <typename TT>
__global__ void __launch_bounds__(kThreads) k_matvec_long(const MatvecArgs a, int log2b) {
  const int lane = threadIdx.x & 31;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5), j = blockIdx.y;
  if (r >= a.rows) return;  // (an ordinary launch: no overlap)
  const uint16_t* x = a.x + j * a.x_stride;
  float sum = 0.0f;
#pragma unroll 8
  for (int64_t c = lane; c < a.cols; c += 32) {
    const int64_t e = r * a.cols + c;
    const int q = a.bits == 8 ? static_cast<int>(static_cast<int8_t>(__ldg(a.codes + e)))
                              : code_int4(__ldg(a.codes + (e >> 1)), static_cast<int>(e & 1));
    const float qx = __fmul_rn(static_cast<float>(q), bits16_to_float(__ldg(x + c), TT()));  // exact
    sum = __fmaf_rn(qx, __ldg(a.scales + (e >> log2b)), sum);
  }
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (lane == 0) {
    if (a.bias) sum += bits16_to_float(ld_after_u16(a.bias + r), TT());
    store_y(a.y, j * a.y_stride + r, sum, a.y_kind);
  }
}

// Bytes of x per CTA of k_matvec_any: two CTAs per SM; what one can hold.
constexpr int64_t kAnyX = 64 * 1024, kAnyMaxX = 180 * 1024;
constexpr int kAnyMaxBytes = static_cast<int>(kAnyMaxX) + kWarps * std::max(AnyShape<4>::RING, AnyShape<8>::RING);

// One overlapped launch (zpp_overlap.cuh) with `split` CTAs of a cluster along each row. The opt-in
// limit belongs to the kernel, which other threads launch too with layouts of other sizes, so it
// is always set to the largest.
template <typename... Params, typename... Args>
static cudaError_t launch_split(void (*kern)(Params...), int64_t tiles, int64_t vec_groups, int split,
                                size_t bytes, cudaStream_t s, Args... args) {
  if (bytes > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kAnyMaxBytes);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * split), static_cast<unsigned>(vec_groups));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(split);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<Params>(args)...);
}

// How a launch splits a row: over wk warps of a CTA and `split` CTAs.
struct MvPlan {
  int wk, split;
};

template <typename TT, int BITS, int MT, int NV, int SP, int NT, int U>
static cudaError_t run_mma(const MatvecArgs& a, int log2b, const MvPlan& p, cudaStream_t s) {
  using S = MvShape<BITS, MT, NV, SP, NT>;
  constexpr size_t kBytes = kWarps * U * S::SEG_BYTES;
  static_assert(kBytes <= 48 * 1024, "no opt-in shared memory");
  const int64_t rows = static_cast<int64_t>(S::ROWS) * (kWarps / p.wk);
  return launch_split(k_matvec_mma<TT, BITS, MT, NV, SP, NT, U>, (a.rows + rows - 1) / rows,
                      (a.vecs + S::VECS - 1) / S::VECS, p.split, kBytes, s, a, log2b, p.wk, p.split,
                      Codes<TT, BITS>::kMasks);
}

// `base` warps a row where it has as many units, then more warps and CTAs until some 13 warps per
// SM have work, never more than units. (INT4, 1 / 2 / 4 / 8 warps a row, us. One vector: 24576 x 8192
// 34.3 / 29.3 / 24.6 / 25.2, rule 4; 8192 x 8192 31.0 / 17.9 / 11.2 / 10.1, rule 8; 1024 x 16384, 8
// warps in 1 / 2 / 4 CTAs 6.8 / 5.5 / 8.7, rule 2; 32768 x 1024, 1 / 2 / 4 warps 6.8 / 6.7 / 11.6, rule
// 1. Four vectors, 8192 x 32768: 167 / 89 / 48 / 34, eight 214 / 120 / 64 / 38, sixteen 278 / 142 / 76 / 55,
// rule 8; one warp in each of 4 CTAs 48, 63 and 82. The rule is not the best of 24576 x 8192 with eight
// vectors: 57 / 38 / 38 / 34, rule 4.)
static MvPlan mv_plan(int64_t tiles, int64_t units, int base, bool ctas_first = false) {
  MvPlan p{1, 1};
  constexpr int64_t kBusy = 2000;
  const auto idle = [&] { return 2 * p.split * p.wk <= units && tiles * p.wk * p.split < kBusy; };
  while (p.wk < base && 2 * p.wk <= units) p.wk *= 2;
  if (ctas_first)
    while (p.split < 8 && idle()) p.split *= 2;
  while (p.wk < kWarps && idle()) p.wk *= 2;
  while (p.split < 8 && idle()) p.split *= 2;
  return p;
}

template <typename TT, int BITS, int NT>
static cudaError_t run_any(const MatvecArgs& a, int log2b, cudaStream_t s) {
  using S = AnyShape<BITS>;
  const int64_t groups = ((a.rows + S::CH - 1) / S::CH + 15) / 16;  // tiles of one shift
  const bool words = a.cols % S::WC == 0 && a.x_stride % S::WC == 0;
  // A CTA that lays x out does so for all its tiles: with four vectors or more fewer warps share a
  // row, so that a CTA has more tiles, and CTAs come before warps. (30000 x 6001, 1 / 2 / 4 warps:
  // 8 vectors 54 / 64 / 90 us, rule 1; 4 vectors 43 / 47 / 56, rule 2; one vector 2 / 4 / 8 warps 36.8 / 35.7
  // / 38.7, rule 4. 2861 x 20897, 8 vectors: 8 warps of one CTA 66, one of 8 CTAs 37, two of 4, the
  // rule, 39; 13 vectors 83 / 34 / 45. 5121 x 1283 INT8, 13 vectors: one warp of 8 CTAs, the rule, 13.8,
  // 8 warps of one CTA 13.0, two of 2 12.1.) Short rows: 50001 x 1003, 9 stages a row, 1 / 2 warps: 4
  // vectors 17.7 / 16.8 us, rule 2; 13 vectors 21.2 / 27.0, rule 1.
  const int stages = any_stages(a.cols, S::CH);
  const bool lay_out = !words && a.vecs > 3;
  const int base = stages < 16 ? (!words && a.vecs > 8 ? 1 : 2) : !lay_out ? 4 : a.vecs > 4 ? 1 : 2;
  MvPlan p = mv_plan(groups * S::CH, stages, base, lay_out && stages >= 16);
  const int wr = kWarps / p.wk;
  const int64_t ctas = (groups + wr - 1) / wr * S::CH;
  if (words)
    return launch_split(k_matvec_any<TT, BITS, true, NT>, ctas, (a.vecs + 8 * NT - 1) / (8 * NT), p.split,
                        kWarps * S::RING, s, a, log2b, p.wk, p.split, Codes<TT, BITS>::kMasks);
  // x of a CTA's share lies in shared memory: more CTAs along a row, then fewer vectors at a time
  const auto x_bytes = [&](int64_t vecs) {
    return static_cast<int64_t>(any_share(a.cols, S::CH, p.wk, p.split)) * 16 * vecs * S::XB;
  };
  int64_t vecs = a.vecs < 8 * NT ? a.vecs : 8 * NT;
  while (p.split < 8 && x_bytes(vecs) > kAnyX) p.split *= 2;
  while (vecs > 1 && x_bytes(vecs) > kAnyMaxX) vecs /= 2;
  if (x_bytes(vecs) > kAnyMaxX) {
    const dim3 grid(tile_grid(a.rows, kWarps), static_cast<unsigned>(a.vecs));
    k_matvec_long<TT><<<grid, kThreads, 0, s>>>(a, log2b);
    return cudaGetLastError();
  }
  const int64_t at_once = vecs < 8 * NT ? vecs : a.vecs;  // of one launch
  for (int64_t v = 0; v < a.vecs; v += at_once) {
    MatvecArgs part = a;
    part.x = a.x + v * a.x_stride;
    part.y = static_cast<uint8_t*>(a.y) + v * a.y_stride * (a.y_kind == 2 ? 4 : 2);
    part.vecs = std::min(at_once, a.vecs - v);
    const cudaError_t e = launch_split(
        k_matvec_any<TT, BITS, false, NT>, ctas, (part.vecs + 8 * NT - 1) / (8 * NT), p.split,
        kWarps * S::RING + static_cast<size_t>(x_bytes(std::min<int64_t>(part.vecs, 8 * NT))), s, part, log2b,
        p.wk, p.split, Codes<TT, BITS>::kMasks);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename TT>
static cudaError_t launch_any(const MatvecArgs& a, int log2b, cudaStream_t s) {
  if (a.vecs > 8) return a.bits == 8 ? run_any<TT, 8, 2>(a, log2b, s) : run_any<TT, 4, 2>(a, log2b, s);
  return a.bits == 8 ? run_any<TT, 8, 1>(a, log2b, s) : run_any<TT, 4, 1>(a, log2b, s);
}

template <typename TT, int BITS, int SP, int MT, int NV, int NT>
static cudaError_t run_planned(const MatvecArgs& a, int log2b, cudaStream_t s) {
  using S = MvShape<BITS, MT, NV, SP, NT>;
  const int64_t segs = a.cols / S::SEG;
  const MvPlan p = mv_plan((a.rows + S::ROWS - 1) / S::ROWS, (segs + S::UNIT - 1) / S::UNIT, 4);
  return run_mma<TT, BITS, MT, NV, SP, NT, 4 / MT>(a, log2b, p, s);  // 4 KB on their way per warp
}

// Two fragments of rows per warp share every load and permutation of x. One vector has little of
// those, so there the second fragment pays only once some seven warps per SM have a unit to do.
// (One vector, one / two fragments: 24576 x 8192 24.7 / 24.6 us, 8192 x 8192 13.4 / 10.1; but 4096
// x 4096 4.8 / 6.6, 2048 x 2048 INT8 3.8 / 5.4 us. Four vectors: 2048 x 2048 INT8 4.7 / 3.9, 4096 x
// 4096 6.1 / 5.3, 8192 x 8192 15.8 / 11.1.) More than eight vectors of blocks of 64 take one: four
// sets of results of 32 rows do not fit the registers. Some INT4 forms in use spill all the same:
// with 9 to 16 vectors 20 to 56 bytes per lane, fp16 with 5 to 8 vectors of blocks of 64 16, fp16 with
// one vector and one fragment 8; INT8 forms none.
template <typename TT, int BITS, int SP>
static cudaError_t by_vecs(const MatvecArgs& a, int log2b, cudaStream_t s) {
  if (a.vecs == 1) {
    using S = MvShape<BITS, 2, 1, SP, 1>;
    const int64_t units = (a.rows + S::ROWS - 1) / S::ROWS * ((a.cols / S::SEG + S::UNIT - 1) / S::UNIT);
    return units >= 1000 ? run_planned<TT, BITS, SP, 2, 1, 1>(a, log2b, s)
                         : run_planned<TT, BITS, SP, 1, 1, 1>(a, log2b, s);
  }
  if (a.vecs == 2) return run_planned<TT, BITS, SP, 2, 2, 1>(a, log2b, s);
  if (a.vecs <= 4) return run_planned<TT, BITS, SP, 2, 4, 1>(a, log2b, s);
  if (a.vecs <= 8) return run_planned<TT, BITS, SP, 2, 8, 1>(a, log2b, s);
  return run_planned<TT, BITS, SP, SP == 1 ? 2 : 1, 8, 2>(a, log2b, s);
}

template <typename TT>
static cudaError_t launch_type(const MatvecArgs& a, int log2b, cudaStream_t s) {
  if (a.cols % (a.bits == 8 ? 64 : 128) != 0 || a.x_stride % 8 != 0)
    return launch_any<TT>(a, log2b, s);
  if (a.bits == 8) return by_vecs<TT, 8, 1>(a, log2b, s);
  return a.block == 64 ? by_vecs<TT, 4, 2>(a, log2b, s) : by_vecs<TT, 4, 1>(a, log2b, s);
}

cudaError_t launch_matvec(const MatvecArgs& a, cudaStream_t s) {
  const int log2b = __builtin_ctz(static_cast<unsigned>(a.block));
  return a.x_bf16 ? launch_type<BF16>(a, log2b, s) : launch_type<F16>(a, log2b, s);
}

}  // namespace zpp
