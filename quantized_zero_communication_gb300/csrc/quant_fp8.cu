// quant_fp8.cu -- K11: a matrix to e4m3 codes with a power-of-two scale per block, as it lies and
// transposed.
//
//   scale = the smallest 2^e, e >= -126, with amax <= 448 * 2^e (0 where amax is 0),  code = x / scale
//
// rounded to nearest even: a product with a power of two is exact, so the code is that of the exact
// quotient. A block is 128 columns of one row, or a tile of 128 x 128. amax is over finite values; an
// infinite or NaN value has the code NaN.
//
// One CTA per tile of 128 x 128; a thread holds 4 consecutive rows of 16 columns, which it reads
// once. The transposed codes go through shared memory in words of 4 rows, their places permuted so
// that neither side meets a bank twice.
#include "zpp_launch.h"
#include "zpp_overlap.cuh"

namespace zpp {

constexpr int kQuantTile = 128;

struct QuantFp8Run {
  const void* x;
  int64_t rows, cols, x_stride;
  uint8_t* codes;
  int64_t codes_stride;
  float* scales;
  int64_t scale_row, scale_block;  // strides of the scales along rows and blocks
  uint8_t* codes_t;
  int64_t codes_t_stride;
  float* scales_t;
  int64_t scale_t_row, scale_t_block;
  bool whole;  // x, its rows and the codes' rows allow vector accesses
};

// 2^e and 2^-e for a block's largest magnitude (finite, >= 0).
__device__ __forceinline__ void power_scale(float amax, float& scale, float& inv) {
  // 448 is 1.75 * 2^8: the exponent is amax's less 8, one more above a mantissa of 1.75.
  int e = static_cast<int>((__float_as_uint(amax) + 0x1FFFFFu) >> 23) - 127 - 8;
  e = max(e, -126);
  scale = amax > 0.0f ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23) : 0.0f;
  inv = amax > 0.0f ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : 0.0f;
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// x times the inverse scale; an infinite value (`odd`: the block may hold one) becomes NaN.
__device__ __forceinline__ float scaled(float x, float inv, bool odd) {
  float v = __fmul_rn(x, inv);
  if (odd && !(fabsf(x) <= 3.402823466e38f)) v = __int_as_float(0x7fc00000);
  return v;
}
__device__ __forceinline__ uint32_t codes4(const float* x, const float* inv, int inv_step, bool odd) {
  const uint32_t a = e4m3x2(scaled(x[0], inv[0], odd), scaled(x[1], inv[inv_step], odd));
  const uint32_t b = e4m3x2(scaled(x[2], inv[2 * inv_step], odd), scaled(x[3], inv[3 * inv_step], odd));
  return a | (b << 16);
}

template <int KIND>
__device__ __forceinline__ float element(const void* p, int64_t i) {
  if constexpr (KIND == 2) return static_cast<const float*>(p)[i];
  const uint16_t b = static_cast<const uint16_t*>(p)[i];
  return KIND == 0 ? bits16_to_float(b, F16()) : bits16_to_float(b, BF16());
}

// 16 values of a row, zeros outside the matrix.
template <int KIND>
__device__ __forceinline__ void load_row(const QuantFp8Run& a, int64_t row, int64_t col, float (&v)[16]) {
  if (row < a.rows && a.whole && col + 16 <= a.cols) {
    const char* p = static_cast<const char*>(a.x) + (row * a.x_stride + col) * (KIND == 2 ? 4 : 2);
#pragma unroll
    for (int h = 0; h < (KIND == 2 ? 4 : 2); ++h) {
      const uint4 w = ld_after_v4(p + 16 * h);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (KIND == 2) {
          v[4 * h + k] = __uint_as_float(u[k]);
        } else {
          const float2 f = KIND == 0 ? unpack2(u[k], F16()) : unpack2(u[k], BF16());
          v[8 * h + 2 * k] = f.x, v[8 * h + 2 * k + 1] = f.y;
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      v[j] = row < a.rows && col + j < a.cols ? element<KIND>(a.x, row * a.x_stride + col + j) : 0.0f;
  }
}

// 16 codes to a row of `n` bytes, from byte `at` on; the row's tail byte by byte.
__device__ __forceinline__ void store_codes(uint8_t* row, int64_t at, int64_t n, const uint32_t (&w)[4]) {
  if (at + 16 <= n) {
    st_v4(row + at, make_uint4(w[0], w[1], w[2], w[3]));
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (at + j < n) row[at + j] = static_cast<uint8_t>(w[j >> 2] >> (8 * (j & 3)));
  }
}

// The largest finite magnitude, and whether there is an infinite one (a NaN is passed over).
__device__ __forceinline__ float finite_max(float m, float v) {
  const float a = fabsf(v);
  return a <= 3.402823466e38f ? fmaxf(m, a) : m;
}

template <int KIND, bool TILE, bool TRANS>
__global__ void __launch_bounds__(256) k_quant_fp8(const QuantFp8Run a) {
  __shared__ float red[8][kQuantTile];
  __shared__ float col_inv[kQuantTile];
  __shared__ __align__(16) uint32_t turned[TRANS ? kQuantTile * 32 : 1];
  grid_wait();
  grid_release();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * kQuantTile, c0 = static_cast<int64_t>(blockIdx.x) * kQuantTile;
  const int rq = warp * 4 + (lane >> 3);  // which 4 rows of the tile
  const int cg = lane & 7;                // which 16 columns
  const int64_t row = r0 + rq * 4, col = c0 + cg * 16;
  float v[4][16];
#pragma unroll
  for (int i = 0; i < 4; ++i) load_row<KIND>(a, row + i, col, v[i]);

  float row_inv[4], tile_inv = 0.0f;
  if constexpr (TILE) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) m = finite_max(m, v[i][j]);
    m = warp_max(m, 32);
    if (lane == 0) red[0][warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = fmaxf(m, red[0][w]);
    float scale;
    power_scale(m, scale, tile_inv);
    if (threadIdx.x == 0)
      a.scales[static_cast<int64_t>(blockIdx.y) * a.scale_row + static_cast<int64_t>(blockIdx.x) * a.scale_block] = scale;
#pragma unroll
    for (int i = 0; i < 4; ++i) row_inv[i] = tile_inv;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float m = 0.0f, scale;
#pragma unroll
      for (int j = 0; j < 16; ++j) m = finite_max(m, v[i][j]);
      m = warp_max(m, 8);
      power_scale(m, scale, row_inv[i]);
      if (cg == 0 && row + i < a.rows)
        a.scales[(row + i) * a.scale_row + static_cast<int64_t>(blockIdx.x) * a.scale_block] = scale;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (row + i >= a.rows) break;
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = codes4(&v[i][4 * k], &row_inv[i], 0, true);
    store_codes(a.codes + (row + i) * a.codes_stride, col, a.cols, w);
  }
  if constexpr (TRANS) {
    if constexpr (!TILE) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = finite_max(m, v[i][j]);
        m = fmaxf(m, __shfl_xor_sync(~0u, m, 8));
        m = fmaxf(m, __shfl_xor_sync(~0u, m, 16));
        if (lane < 8) red[warp][cg * 16 + j] = m;
      }
      __syncthreads();
      if (threadIdx.x < kQuantTile) {
        float m = 0.0f, scale, inv;
#pragma unroll
        for (int w = 0; w < 8; ++w) m = fmaxf(m, red[w][threadIdx.x]);
        power_scale(m, scale, inv);
        col_inv[threadIdx.x] = inv;
        if (c0 + threadIdx.x < a.cols)
          a.scales_t[(c0 + threadIdx.x) * a.scale_t_row + static_cast<int64_t>(blockIdx.y) * a.scale_t_block] = scale;
      }
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int c = cg * 16 + j;
      const float inv = TILE ? tile_inv : col_inv[c];
      const float x[4] = {v[0][j], v[1][j], v[2][j], v[3][j]};
      turned[c * 32 + (rq ^ (cg << 2))] = codes4(x, &inv, 0, true);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // 16 rows of codes at a time: 8 threads a column of the tile
      const int c = k * 32 + (threadIdx.x >> 3), g = threadIdx.x & 7;
      const uint4 t = *reinterpret_cast<const uint4*>(&turned[c * 32 + ((g ^ ((c >> 4) & 7)) << 2)]);
      const uint32_t w[4] = {t.x, t.y, t.z, t.w};
      if (c0 + c < a.cols) store_codes(a.codes_t + (c0 + c) * a.codes_t_stride, r0 + g * 16, a.rows, w);
    }
  }
}

template <int KIND>
static cudaError_t run_quant_fp8(const QuantFp8Run& a, bool tile, cudaStream_t s) {
  auto kern = a.codes_t ? (tile ? k_quant_fp8<KIND, true, true> : k_quant_fp8<KIND, false, true>)
                        : (tile ? k_quant_fp8<KIND, true, false> : k_quant_fp8<KIND, false, false>);
  const int64_t per = 65535 * static_cast<int64_t>(kQuantTile);
  for (int64_t r = 0; r < a.rows; r += per) {  // the grid's second dimension ends at 65535
    QuantFp8Run b = a;
    const int64_t size = KIND == 2 ? 4 : 2, down = r / kQuantTile;
    b.rows = a.rows - r < per ? a.rows - r : per;
    b.x = static_cast<const char*>(a.x) + r * a.x_stride * size;
    b.codes = a.codes + r * a.codes_stride;
    b.scales = a.scales + (tile ? down : r) * a.scale_row;
    if (a.codes_t) {
      b.codes_t = a.codes_t + r;
      b.scales_t = a.scales_t ? a.scales_t + down * a.scale_t_block : nullptr;
    }
    const dim3 grid(static_cast<unsigned>((a.cols + kQuantTile - 1) / kQuantTile),
                    static_cast<unsigned>((b.rows + kQuantTile - 1) / kQuantTile));
    const cudaError_t e = launch_overlapped_smem(kern, grid, 256, 0, s, b);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_quant_fp8(const QuantFp8Args& q, cudaStream_t s) {
  QuantFp8Run a{};
  a.x = q.x, a.rows = q.rows, a.cols = q.cols, a.x_stride = q.x_stride;
  a.codes = q.codes, a.codes_stride = q.codes_stride;
  a.scales = q.scales, a.scale_row = q.scale_row, a.scale_block = q.scale_block;
  a.codes_t = q.codes_t, a.codes_t_stride = q.codes_t_stride;
  a.scales_t = q.scales_t, a.scale_t_row = q.scale_t_row, a.scale_t_block = q.scale_t_block;
  const int64_t size = q.x_kind == 2 ? 4 : 2;
  a.whole = ((reinterpret_cast<uintptr_t>(q.x) | static_cast<uintptr_t>(q.x_stride * size)) & 15) == 0;
  return q.x_kind == 2   ? run_quant_fp8<2>(a, q.tile == 128, s)
         : q.x_kind == 1 ? run_quant_fp8<1>(a, q.tile == 128, s)
                         : run_quant_fp8<0>(a, q.tile == 128, s);
}

}  // namespace zpp
