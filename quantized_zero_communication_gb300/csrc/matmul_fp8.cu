// matmul_fp8.cu -- K10: products of e4m3 matrices with a scale per block of 128 along the sum.
//
//   y[m][n] = sum over blocks kb of  sa[m][kb] sb[n][kb] (sum over k in kb of a[m][k] b[n][k])  (+ bias[n])
//
// The inner sums are tcgen05 products (fp32 in tensor memory), one block of 128 a slot of a ring there;
// eight warps read each slot, multiply it by its scales and add it to the tile's sums, which stay in
// registers, while the matrix unit fills the next slot. So a sum never mixes scales, and its length
// in the matrix unit is 128.
//
// P is the operand whose rows are the 128 lanes of tensor memory, Q the one whose rows are a tile's
// columns: a and b, or b and a where there are few rows of a.
#include "zpp_launch.h"
#include "zpp_overlap.cuh"
#include "zpp_tcgen05.cuh"
#include "zpp_tensor_map.h"

namespace zpp {

static __device__ unsigned g_matmul_fault;
constexpr unsigned kMatmulFault = 8;  // its bit of the fault word

constexpr int kLanes = 128;        // rows of P in a tile
constexpr int kStep = 128;         // codes of the sum in a block, and bytes of a row of a stage
constexpr int kSumWarps = 8;       // warps that scale and add
constexpr int kMatmulThreads = (kSumWarps + 2) * 32;

template <int BN>
struct MatmulGeo {
  static constexpr int STAGE = (kLanes + BN) * kStep;
  static constexpr int STAGES = BN == 256 ? 4 : (BN == 128 ? 6 : 8);
  static constexpr int SLOT = BN < 32 ? 32 : BN;  // tensor-memory columns of a slot
  static constexpr int SLOTS = 512 / SLOT < 4 ? 512 / SLOT : 4;
  static constexpr int HALF = BN / 2;  // columns of a warp
  static constexpr int BARS = STAGES * STAGE;
  static constexpr int SCALES = BARS + (2 * STAGES + 2 * SLOTS + 1) * 8 + 16;
  static constexpr int SMEM = 1024 + SCALES + 2 * BN * 4;
};

struct MatmulSide {
  const float* scales;
  int64_t row, block;  // strides of the scales
  int64_t rows;
  int32_t shift;       // rows that share a scale: 1 << shift
};
struct MatmulRun {
  MatmulSide p, q;
  int32_t blocks;       // of the sum
  int32_t p_tiles, q_tiles;
  void* y;
  int64_t y_p, y_q;     // strides of y along P's and Q's rows; one of them is 1
  int32_t y_kind;
  const void* bias;     // of y's type, along Q's rows (or P's: bias_p)
  int32_t bias_p;
};

__device__ __forceinline__ float load_kind(const void* p, int64_t i, int kind) {
  if (kind == 2) return static_cast<const float*>(p)[i];
  const uint16_t b = static_cast<const uint16_t*>(p)[i];
  return kind == 0 ? bits16_to_float(b, F16()) : bits16_to_float(b, BF16());
}
__device__ __forceinline__ void store_kind(void* p, int64_t i, float v, int kind) {
  if (kind == 2) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(kind == 0 ? pack2(v, v, F16()) : pack2(v, v, BF16()));
}

// QROWS: Q has a scale for each row (else per tile of 128 rows, in which a warp's columns lie).
template <int BN, bool QROWS>
__global__ void __launch_bounds__(kMatmulThreads, 1)
    k_matmul_fp8(const __grid_constant__ CUtensorMap p_map, const __grid_constant__ CUtensorMap q_map,
                 const MatmulRun run) {
  using G = MatmulGeo<BN>;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + G::BARS);
  uint64_t* empty = full + G::STAGES;
  uint64_t* summed = empty + G::STAGES;  // a slot holds a block's sums
  uint64_t* taken = summed + G::SLOTS;   // and has been read
  uint64_t* drained = taken + G::SLOTS;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(drained + 1);
  float* q_scales = reinterpret_cast<float*>(smem + G::SCALES);  // [2][BN]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < G::STAGES; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
    for (int i = 0; i < G::SLOTS; ++i) mbar_init(&summed[i], 1), mbar_init(&taken[i], kSumWarps);
    mbar_init(drained, 1);
    mbar_init_fence();
    tma_prefetch(&p_map);
    tma_prefetch(&q_map);
  }
  if (warp == kSumWarps) {
    tmem_alloc<1>(tmem_at, G::SLOT * G::SLOTS);
    tmem_alloc_done<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  grid_wait();
  grid_release();

  const int tiles = run.p_tiles * run.q_tiles, blocks = run.blocks;
  bool alive = true;

  if (warp == kSumWarps) {  // ---------------------------------------------- copies into the stages
    if (lane == 0) {
      Ring<G::STAGES> r;
      int64_t issued = 0;
      for (int t = blockIdx.x; t < tiles && alive; t += gridDim.x) {
        const int p0 = t % run.p_tiles * kLanes, q0 = t / run.p_tiles * BN;
        for (int kb = 0; kb < blocks; ++kb) {
          tc_wait(&empty[r.at], r.phase ^ 1u, alive, &g_matmul_fault, kMatmulFault);
          if (!alive) break;
          uint8_t* stage = smem + r.at * G::STAGE;
          mbar_arrive_expect_tx(&full[r.at], G::STAGE);
          tma_load(stage, &p_map, kb * kStep, p0, &full[r.at]);
          tma_load(stage + kLanes * kStep, &q_map, kb * kStep, q0, &full[r.at]);
          ++issued;
          r.next();
        }
      }
      if (!alive) {  // copies that nobody may have waited for
        bool wait = true;
        for (int64_t d = 0; d < G::STAGES && d < issued; ++d) {
          if (--r.at < 0) r.at = G::STAGES - 1, r.phase ^= 1u;
          tc_wait(&full[r.at], r.phase, wait, &g_matmul_fault, kMatmulFault);
        }
      }
    }
  } else if (warp == kSumWarps + 1) {  // ---------------------------------------------- the products
    if (lane == 0) {
      constexpr uint32_t instr = tc_instruction(kLanes, BN, 0, 0, false, false);
      Ring<G::STAGES> r;
      Ring<G::SLOTS> s;
      for (int t = blockIdx.x; t < tiles && alive; t += gridDim.x)
        for (int kb = 0; kb < blocks; ++kb) {
          tc_wait(&taken[s.at], s.phase ^ 1u, alive, &g_matmul_fault, kMatmulFault);
          tc_wait(&full[r.at], r.phase, alive, &g_matmul_fault, kMatmulFault);
          if (!alive) break;
          tc_fence_after();
          const uint32_t p = smem_addr(smem + r.at * G::STAGE), q = p + kLanes * kStep;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_f8<1>(tmem + s.at * G::SLOT, tc_operand(p + 32 * k, 16, 1024),
                         tc_operand(q + 32 * k, 16, 1024), instr, k > 0);
          tc_commit(&empty[r.at]);
          tc_commit(&summed[s.at]);
          r.next();
          s.next();
        }
      if (!alive) {
        bool wait = true;
        tc_commit(drained);
        tc_wait(drained, 0, wait, &g_matmul_fault, kMatmulFault);
      }
    }
  } else {  // -------------------------------------------------------------- scales, sums, results
    constexpr int HALF = G::HALF, CHUNK = HALF < 32 ? HALF : 32;
    const int half = warp >> 2, in_half = threadIdx.x & 127;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21) + half * HALF;
    Ring<G::SLOTS> s;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
      const int64_t p0 = static_cast<int64_t>(t % run.p_tiles) * kLanes + (warp & 3) * 32 + lane;
      const int64_t q0 = static_cast<int64_t>(t / run.p_tiles) * BN + half * HALF;
      const bool p_in = p0 < run.p.rows;
      const float* sp = run.p.scales + (p_in ? p0 >> run.p.shift : 0) * run.p.row;
      const int64_t q_row = QROWS ? q0 + in_half : q0;
      const bool q_in = (!QROWS || in_half < HALF) && q_row < run.q.rows;
      const float* sq = run.q.scales + (q_in ? q_row >> run.q.shift : 0) * run.q.row;
      float sums[HALF];
#pragma unroll
      for (int i = 0; i < HALF; ++i) sums[i] = 0.0f;
      float sp_next = blocks ? *sp : 0.0f, sq_next = blocks ? *sq : 0.0f;
      for (int kb = 0; kb < blocks; ++kb) {
        float scale = sp_next;
        const float sq_now = sq_next;
        if (kb + 1 < blocks) {
          sp_next = sp[(kb + 1) * run.p.block];
          sq_next = sq[(kb + 1) * run.q.block];
        }
        float* qs = q_scales + (kb & 1) * BN + half * HALF;
        if constexpr (QROWS) {
          if (in_half < HALF) qs[in_half] = sq_now;
          named_barrier(1 + half, 128);
        } else {
          scale = __fmul_rn(scale, sq_now);
        }
        tc_wait(&summed[s.at], s.phase, alive, &g_matmul_fault, kMatmulFault);
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < HALF; c += CHUNK) {
          uint32_t v[CHUNK];
          tmem_ld(lanes + s.at * G::SLOT + c, v);
          tmem_ld_wait(v);
#pragma unroll
          for (int i = 0; i < CHUNK; ++i) {
            float x = __uint_as_float(v[i]);
            if constexpr (QROWS) x = __fmul_rn(x, qs[c + i]);
            sums[c + i] = __fmaf_rn(x, scale, sums[c + i]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&taken[s.at]);
        s.next();
      }
      if (p_in) {
#pragma unroll
        for (int i = 0; i < HALF; ++i) {
          const int64_t q = q0 + i;
          if (q < run.q.rows) {
            float v = sums[i];
            if (run.bias) v = __fadd_rn(v, load_kind(run.bias, run.bias_p ? p0 : q, run.y_kind));
            store_kind(run.y, p0 * run.y_p + q * run.y_q, v, run.y_kind);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kSumWarps) {
    tc_fence_after();
    tmem_free<1>(tmem, G::SLOT * G::SLOTS);
  }
}

template <int BN, bool QROWS>
static cudaError_t run_matmul(const CUtensorMap& p, const CUtensorMap& q, const MatmulRun& run,
                              cudaStream_t s) {
  auto kern = k_matmul_fp8<BN, QROWS>;
  constexpr int smem = MatmulGeo<BN>::SMEM;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  int64_t tiles = static_cast<int64_t>(run.p_tiles) * run.q_tiles;
  const int grid = static_cast<int>(tiles < 152 ? tiles : 152);
  return launch_overlapped_smem(kern, dim3(grid), kMatmulThreads, smem, s, p, q, run);
}

cudaError_t launch_matmul_fp8(const MatmulArgs& a, cudaStream_t s) {
  // Few rows of a: they are the columns of the tiles, which are narrow then.
  const bool swap = a.a.rows <= 64;
  const MatmulOperand &p = swap ? a.b : a.a, &q = swap ? a.a : a.b;
  const int bn = !swap ? 128 : q.rows <= 16 ? 16 : q.rows <= 32 ? 32 : 64;
  MatmulRun run{};
  const auto side = [](const MatmulOperand& o) {
    return MatmulSide{o.scales, o.scale_row, o.scale_block, o.rows, o.tile == 128 ? 7 : 0};
  };
  run.p = side(p);
  run.q = side(q);
  run.blocks = static_cast<int32_t>((a.depth + kStep - 1) / kStep);
  run.p_tiles = static_cast<int32_t>((p.rows + kLanes - 1) / kLanes);
  run.q_tiles = static_cast<int32_t>((q.rows + bn - 1) / bn);
  run.y = a.y;
  run.y_p = swap ? 1 : a.y_stride;
  run.y_q = swap ? a.y_stride : 1;
  run.y_kind = a.y_kind;
  run.bias = a.bias;
  run.bias_p = swap;
  CUtensorMap p_map{}, q_map{};
  if (run.blocks > 0) {
    cudaError_t e = make_tensor_map(&p_map, p.codes, 1, a.depth, p.rows, p.stride, 0, 0, kLanes);
    if (e == cudaSuccess) e = make_tensor_map(&q_map, q.codes, 1, a.depth, q.rows, q.stride, 0, 0, bn);
    if (e != cudaSuccess) return e;
  }
  const bool rows = run.q.shift == 0;
  switch (bn) {
    case 16: return rows ? run_matmul<16, true>(p_map, q_map, run, s) : run_matmul<16, false>(p_map, q_map, run, s);
    case 32: return rows ? run_matmul<32, true>(p_map, q_map, run, s) : run_matmul<32, false>(p_map, q_map, run, s);
    case 64: return rows ? run_matmul<64, true>(p_map, q_map, run, s) : run_matmul<64, false>(p_map, q_map, run, s);
    default: return rows ? run_matmul<128, true>(p_map, q_map, run, s) : run_matmul<128, false>(p_map, q_map, run, s);
  }
}

cudaError_t read_matmul_fault(unsigned* flags, bool clear) {
  const cudaError_t err = cudaMemcpyFromSymbol(flags, g_matmul_fault, sizeof(unsigned));
  if (err != cudaSuccess || !clear) return err;
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_matmul_fault, &zero, sizeof(unsigned));
}

}  // namespace zpp
