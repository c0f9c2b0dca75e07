// quant_fp8.cu -- K11: a matrix to e4m3 codes with a power-of-two scale per block, as it lies and
// transposed.
//
//   scale = the smallest 2^e, e >= -126, with amax <= 448 * 2^e (0 where amax is 0),  code = x / scale
//
// rounded to nearest even: a product with a power of two is exact, so the code is that of the exact
// quotient. A block is 128 columns of one row, or a tile of 128 x 128. amax is over finite values; an
// infinite or NaN value has the code NaN.
//
// Bound by DRAM for tiles (24576 x 8192 fp32, both ways: 184 us, 6.55 TB/s), by issue where rows and columns
// have scales of their own (16384 x 8192 bf16, both ways: 97 us, 5.6 TB/s; rows alone 61 us, 6.6 TB/s).
//
// One CTA per tile of 128 x 128; a thread holds 4 consecutive rows of 16 columns, which it reads
// once. The transposed codes go through shared memory in words of 4 rows, their places permuted so
// that neither side meets a bank twice.
#include "zpp_launch.h"
#include "zpp_overlap.cuh"

namespace zpp {

constexpr int kQuantTile = 128;
// Tiles that are brought into L2 ahead: 2 for each SM (24576 x 8192 fp32: 184 us; 4 for each 189, 6 223, none 245).
constexpr int kAheadTiles = 304;

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
__device__ __forceinline__ uint32_t codes4(f32x2 a, f32x2 b) {
  float x, y, z, w;
  f2_split(a, x, y);
  f2_split(b, z, w);
  return __byte_perm(e4m3x2(x, y), e4m3x2(z, w), 0x5410u);
}

// 16 values of a row as they lie in memory: 8 words of two 16-bit values, or 16 words.
template <int KIND>
struct Row {
  static constexpr int WORDS = KIND == 2 ? 16 : 8;
  uint32_t w[WORDS];
  // values 2k and 2k + 1
  __device__ __forceinline__ f32x2 pair(int k) const {
    if constexpr (KIND == 2) return f2(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
    const float2 f = KIND == 0 ? unpack2(w[k], F16()) : unpack2(w[k], BF16());
    return f2(f.x, f.y);
  }
};

template <int KIND>
__device__ __forceinline__ uint32_t element_bits(const void* p, int64_t i) {
  return KIND == 2 ? static_cast<const uint32_t*>(p)[i] : static_cast<const uint16_t*>(p)[i];
}

// 16 values of a row, zeros outside the matrix.
template <int KIND>
__device__ __forceinline__ void load_row(const QuantFp8Run& a, int64_t row, int64_t col, Row<KIND>& v) {
  if (row < a.rows && a.whole && col + 16 <= a.cols) {
    const char* p = static_cast<const char*>(a.x) + (row * a.x_stride + col) * (KIND == 2 ? 4 : 2);
#pragma unroll
    for (int h = 0; h < Row<KIND>::WORDS / 4; ++h) {
      const uint4 w = ld_after_v4(p + 16 * h);
      v.w[4 * h] = w.x, v.w[4 * h + 1] = w.y, v.w[4 * h + 2] = w.z, v.w[4 * h + 3] = w.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < Row<KIND>::WORDS; ++j) {
      v.w[j] = 0u;
#pragma unroll
      for (int h = 0; h < 16 / Row<KIND>::WORDS; ++h) {
        const int64_t c = col + j * (16 / Row<KIND>::WORDS) + h;
        if (row < a.rows && c < a.cols) v.w[j] |= element_bits<KIND>(a.x, row * a.x_stride + c) << (16 * h);
      }
    }
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

// Magnitudes are compared as bits, which order as the values do: 32-bit ones, or 16-bit ones two to a
// word. finite_only: an infinite or NaN one counts as 0.
template <int KIND>
struct Top {
  static constexpr uint32_t SIGN = KIND == 2 ? 0x7fffffffu : 0x7fff7fffu;
  static constexpr uint32_t INF = KIND == 2 ? 0x7f800000u : KIND == 1 ? 0x7f80u : 0x7c00u;
  __device__ __forceinline__ static uint32_t more(uint32_t a, uint32_t b) {
    return KIND == 2 ? max(a, b) : __vmaxu2(a, b);
  }
  __device__ __forceinline__ static uint32_t size(uint32_t w, bool finite_only) {
    w &= SIGN;
    if (finite_only) {
      if constexpr (KIND == 2) {
        if (w >= INF) w = 0u;
      } else {
        if ((w & 0xffffu) >= INF) w &= 0xffff0000u;
        if ((w >> 16) >= INF) w &= 0xffffu;
      }
    }
    return w;
  }
  __device__ __forceinline__ static float value(uint32_t bits) {  // of one magnitude
    return KIND == 2 ? __uint_as_float(bits) : KIND == 1 ? bits16_to_float(bits, BF16()) : bits16_to_float(bits, F16());
  }
};
// x times the inverse scale. odd: an infinite value becomes NaN.
__device__ __forceinline__ f32x2 scaled(f32x2 x, f32x2 inv, bool odd) {
  f32x2 r = f2_mul(x, inv);
  if (odd) {
    float a, b, u, v;
    f2_split(x, a, b);
    f2_split(r, u, v);
    if (!(fabsf(a) <= 3.402823466e38f)) u = __int_as_float(0x7fc00000);
    if (!(fabsf(b) <= 3.402823466e38f)) v = __int_as_float(0x7fc00000);
    r = f2(u, v);
  }
  return r;
}

template <int KIND, bool TILE, bool TRANS>
struct QuantShared {
  uint32_t red[8][KIND == 2 ? kQuantTile : kQuantTile / 2];
  float col_inv[kQuantTile];
  alignas(16) uint32_t turned[TRANS ? kQuantTile * 32 : 1];
};

// The largest magnitude of each of a thread's rows.
template <int KIND, bool FINITE_ONLY>
__device__ __forceinline__ void row_tops(const Row<KIND> (&v)[4], uint32_t (&top)[4]) {
  using T = Top<KIND>;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    top[i] = T::size(v[i].w[0], FINITE_ONLY);
#pragma unroll
    for (int k = 1; k < Row<KIND>::WORDS; ++k) top[i] = T::more(top[i], T::size(v[i].w[k], FINITE_ONLY));
    if constexpr (KIND != 2) top[i] = max(top[i] & 0xffffu, top[i] >> 16);
  }
}

// A tile whose values have been loaded; top: of each row (ODD: made again). ODD: some of them may be infinite or NaN.
template <int KIND, bool TILE, bool TRANS, bool ODD>
__device__ __forceinline__ void quant_tile_fp8(const QuantFp8Run& a, QuantShared<KIND, TILE, TRANS>& sh,
                                               const Row<KIND> (&v)[4], uint32_t (&top)[4], int64_t r0,
                                               int64_t c0) {
  using T = Top<KIND>;
  constexpr int WORDS = Row<KIND>::WORDS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rq = warp * 4 + (lane >> 3), cg = lane & 7;
  const int64_t row = r0 + rq * 4, col = c0 + cg * 16;
  if constexpr (ODD) row_tops<KIND, true>(v, top);
  float row_inv[4];
  if constexpr (TILE) {
    uint32_t m = max(max(top[0], top[1]), max(top[2], top[3]));
    m = __reduce_max_sync(~0u, m);
    if (lane == 0) sh.red[0][warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = max(m, sh.red[0][w]);
    float scale;
    power_scale(T::value(m), scale, row_inv[0]);
    if (threadIdx.x == 0)
      a.scales[static_cast<int64_t>(blockIdx.y) * a.scale_row + static_cast<int64_t>(blockIdx.x) * a.scale_block] = scale;
#pragma unroll
    for (int i = 1; i < 4; ++i) row_inv[i] = row_inv[0];
  } else {
#pragma unroll
    for (int off = 4; off > 0; off >>= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) top[i] = max(top[i], __shfl_xor_sync(~0u, top[i], off));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float scale;
      power_scale(T::value(top[i]), scale, row_inv[i]);
      if (cg == 0 && row + i < a.rows)
        a.scales[(row + i) * a.scale_row + static_cast<int64_t>(blockIdx.x) * a.scale_block] = scale;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (row + i >= a.rows) break;
    uint32_t w[4];
    const f32x2 inv = f2(row_inv[i], row_inv[i]);
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = codes4(scaled(v[i].pair(2 * k), inv, ODD), scaled(v[i].pair(2 * k + 1), inv, ODD));
    store_codes(a.codes + (row + i) * a.codes_stride, col, a.cols, w);
  }
  if constexpr (TRANS) {
    if constexpr (!TILE) {
#pragma unroll
      for (int k = 0; k < WORDS; ++k) {
        uint32_t m = T::more(T::more(T::size(v[0].w[k], ODD), T::size(v[1].w[k], ODD)),
                             T::more(T::size(v[2].w[k], ODD), T::size(v[3].w[k], ODD)));
        m = T::more(m, __shfl_xor_sync(~0u, m, 8));
        m = T::more(m, __shfl_xor_sync(~0u, m, 16));
        if (lane < 8) sh.red[warp][cg * WORDS + k] = m;
      }
      __syncthreads();
      if (threadIdx.x < kQuantTile) {
        const int word = KIND == 2 ? threadIdx.x : threadIdx.x >> 1;
        uint32_t m = 0u;
        float scale, inv;
#pragma unroll
        for (int w = 0; w < 8; ++w) m = T::more(m, sh.red[w][word]);
        if constexpr (KIND != 2) m = (threadIdx.x & 1) ? m >> 16 : m & 0xffffu;
        power_scale(T::value(m), scale, inv);
        sh.col_inv[threadIdx.x] = inv;
        if (c0 + threadIdx.x < a.cols)
          a.scales_t[(c0 + threadIdx.x) * a.scale_t_row + static_cast<int64_t>(blockIdx.y) * a.scale_t_block] = scale;
      }
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {  // columns 2k and 2k + 1: words of 4 rows
      const int c = cg * 16 + 2 * k;
      const f32x2 inv = TILE ? f2(row_inv[0], row_inv[0]) : *reinterpret_cast<const f32x2*>(&sh.col_inv[c]);
      float x[4], y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) f2_split(scaled(v[i].pair(k), inv, ODD), x[i], y[i]);
      sh.turned[c * 32 + (rq ^ (cg << 2))] = codes4(f2(x[0], x[1]), f2(x[2], x[3]));
      sh.turned[(c + 1) * 32 + (rq ^ (cg << 2))] = codes4(f2(y[0], y[1]), f2(y[2], y[3]));
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // 16 rows of codes at a time: 8 threads a column of the tile
      const int c = k * 32 + (threadIdx.x >> 3), g = threadIdx.x & 7;
      const uint4 t = *reinterpret_cast<const uint4*>(&sh.turned[c * 32 + ((g ^ ((c >> 4) & 7)) << 2)]);
      const uint32_t w[4] = {t.x, t.y, t.z, t.w};
      if (c0 + c < a.cols) store_codes(a.codes_t + (c0 + c) * a.codes_t_stride, r0 + g * 16, a.rows, w);
    }
  }
}

// Brings a tile that some CTA will take a little later into L2: a thread a row.
template <int KIND>
__device__ __forceinline__ void prefetch_tile(const QuantFp8Run& a) {
  constexpr int64_t SIZE = KIND == 2 ? 4 : 2;
  const int64_t t = static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x + kAheadTiles;
  const int64_t row = t / gridDim.x * kQuantTile + threadIdx.x, col = t % gridDim.x * kQuantTile;
  if (!a.whole || threadIdx.x >= kQuantTile || row >= a.rows) return;
  const int64_t left = a.cols - col;
  const uint32_t bytes = static_cast<uint32_t>((left < kQuantTile ? left : kQuantTile) * SIZE) & ~15u;
  if (bytes)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const char*>(a.x) +
                                                                     (row * a.x_stride + col) * SIZE),
                 "r"(bytes)
                 : "memory");
}

template <int KIND, bool TILE, bool TRANS>
__global__ void __launch_bounds__(256, KIND == 2 ? 2 : 3) k_quant_fp8(const QuantFp8Run a) {
  __shared__ QuantShared<KIND, TILE, TRANS> sh;
  grid_wait();
  grid_release();
  const int rq = (threadIdx.x >> 5) * 4 + ((threadIdx.x & 31) >> 3), cg = threadIdx.x & 7;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * kQuantTile, c0 = static_cast<int64_t>(blockIdx.x) * kQuantTile;
  Row<KIND> v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) load_row<KIND>(a, r0 + rq * 4 + i, c0 + cg * 16, v[i]);
  prefetch_tile<KIND>(a);
  uint32_t top[4];
  row_tops<KIND, false>(v, top);
  const bool odd = max(max(top[0], top[1]), max(top[2], top[3])) >= Top<KIND>::INF;
  // (values that are not finite take code of their own: the common one has no selections)
  if (__syncthreads_or(odd)) quant_tile_fp8<KIND, TILE, TRANS, true>(a, sh, v, top, r0, c0);
  else quant_tile_fp8<KIND, TILE, TRANS, false>(a, sh, v, top, r0, c0);
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
