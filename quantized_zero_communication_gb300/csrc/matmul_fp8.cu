// matmul_fp8.cu -- K10: products of e4m3 matrices with a scale per block of 128 along the sum.
//
//   y[m][n] = sum over blocks kb of  sa[m][kb] sb[n][kb] (sum over k in kb of a[m][k] b[n][k])  (+ bias[n])
//
// The inner sums are tcgen05 products (fp32 in tensor memory), one block of 128 a slot of a ring there;
// eight warps read each slot, multiply it by its scales and add it to the tile's sums, which stay in
// registers, while the matrix unit fills the next slot. So a sum never mixes scales, and its length
// in the matrix unit is 128. A warp each fetches the scales of P and Q, up to 16 blocks ahead: fetched one
// block ahead by the warps that use them, their latency (about 1 us beside the operands' traffic) was
// the time of a block (8192 x 8192 x 8192: 1280 us).
//
// P is the operand whose rows are the 128 lanes of tensor memory, Q the one whose rows are a tile's
// columns: a and b, or b and a where there are few rows of a (a kernel of its own, below).
#include "zpp_launch.h"
#include "zpp_overlap.cuh"
#include "zpp_tcgen05.cuh"
#include "zpp_tensor_map.h"

namespace zpp {

static __device__ unsigned g_matmul_fault;
constexpr unsigned kMatmulFault = 8;  // its bit of the fault word

constexpr int kLanes = 128;        // rows of P in a tile
constexpr int kStep = 128;         // codes of the sum in a block, and bytes of a row of a stage

// CTAS 2: a pair of CTAs on a tile of 256 x BN; each holds its half of both operands.
template <int CTAS, int BN, bool QROWS>
struct MatmulGeo {
  static constexpr int Q_ROWS = BN / CTAS;  // of a CTA's stage
  static constexpr int STAGE = (kLanes + Q_ROWS) * kStep;
  static constexpr int STAGES = 6;
  static constexpr int SLOT = BN == 96 ? 128 : BN;  // tensor-memory columns of a slot
  static constexpr int SLOTS = 512 / SLOT;
  static constexpr int HALF = BN / 2;  // columns of a warp
  // Blocks whose scales are waited for together. (A wait costs some 100 clocks; where Q has a scale a
  // column, one for every block measured better: 8192^3 613 us against 664.)
  static constexpr int GROUP = QROWS ? 1 : 4, GROUPS = QROWS ? 8 : 4;
  static constexpr int SCALES = STAGES * STAGE;
  static constexpr int BARS = SCALES + GROUPS * GROUP * (kLanes + BN) * 4;
  static constexpr int SMEM = 1024 + BARS + (2 * STAGES + 2 * SLOTS + 2 * GROUPS + 1) * 8 + 16;
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
  int32_t band;         // P tiles that are walked through together, column by column
  void* y;
  int64_t y_p, y_q;     // strides of y along P's and Q's rows; one of them is 1
  int32_t y_kind;
  const void* bias;     // of y's type, along Q's rows (or P's: bias_p)
  int32_t bias_p;
  bool vec;             // y's rows lie along Q's, and 8 results start at multiples of 16 bytes
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

// 8 columns of row p of P, from column q on (a bias by P's rows is in v already).
__device__ __forceinline__ void store_sums(const MatmulRun& run, int64_t p, int64_t q, float (&v)[8]) {
  if (run.bias && !run.bias_p) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (q + i < run.q.rows) v[i] = __fadd_rn(v[i], load_kind(run.bias, q + i, run.y_kind));
  }
  const int64_t at = p * run.y_p + q * run.y_q;
  if (run.vec && q + 8 <= run.q.rows) {  // consecutive and whole
    if (run.y_kind == 2) {
      float* y = static_cast<float*>(run.y) + at;
      st_v4(y, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
      st_v4(y + 4, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                              __float_as_uint(v[7])));
    } else {
      uint16_t* y = static_cast<uint16_t*>(run.y) + at;
      st_v4(y, run.y_kind == 0 ? make_uint4(pack2(v[0], v[1], F16()), pack2(v[2], v[3], F16()),
                                            pack2(v[4], v[5], F16()), pack2(v[6], v[7], F16()))
                               : make_uint4(pack2(v[0], v[1], BF16()), pack2(v[2], v[3], BF16()),
                                            pack2(v[4], v[5], BF16()), pack2(v[6], v[7], BF16())));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (q + i < run.q.rows) store_kind(run.y, at + i * run.y_q, v[i], run.y_kind);
}

// One result (neighbouring lanes have neighbouring rows of P: of y's columns where P is b).
// bias: that of row p of P.
__device__ __forceinline__ void store_one(const MatmulRun& run, int64_t p, int64_t q, float v, float bias) {
  if (q >= run.q.rows) return;
  if (run.bias) v = __fadd_rn(v, bias);
  store_kind(run.y, p * run.y_p + q * run.y_q, v, run.y_kind);
}

// The tiles in the order they are taken: bands of P tiles, column by column, so that the CTAs at work at
// one time share rows of both operands in L2.
__device__ __forceinline__ void matmul_tile(const MatmulRun& run, int t, int& p, int& q) {
  const int per = run.band * run.q_tiles, b = t / per;
  const int height = min(run.band, run.p_tiles - b * run.band);
  t -= b * per;
  p = b * run.band + t % height;
  q = t / height;
}

// QROWS: Q has a scale for each row (else per tile of 128 rows, in which a warp's columns lie).
template <int CTAS, int BN, bool QROWS>
__global__ void __launch_bounds__(kTensorThreads, 1)
    k_matmul_fp8(const __grid_constant__ CUtensorMap p_map, const __grid_constant__ CUtensorMap q_map,
                 const MatmulRun run) {
  using G = MatmulGeo<CTAS, BN, QROWS>;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + G::BARS);
  uint64_t* empty = full + G::STAGES;
  uint64_t* summed = empty + G::STAGES;  // a slot holds a block's sums
  uint64_t* taken = summed + G::SLOTS;   // and has been read
  uint64_t* scaled = taken + G::SLOTS;   // a group of blocks' scales are there
  uint64_t* used = scaled + G::GROUPS;   // and have been used
  uint64_t* drained = used + G::GROUPS;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(drained + 1);
  float* p_scales = reinterpret_cast<float*>(smem + G::SCALES);  // [GROUPS * GROUP][kLanes]
  float* q_scales = p_scales + G::GROUPS * G::GROUP * kLanes;    // [GROUPS * GROUP][BN]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CTAS == 2 ? cluster_rank() : 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < G::STAGES; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
    for (int i = 0; i < G::SLOTS; ++i) mbar_init(&summed[i], 1), mbar_init(&taken[i], CTAS * kResultWarps);
    for (int i = 0; i < G::GROUPS; ++i) mbar_init(&scaled[i], 64), mbar_init(&used[i], kResultWarps);
    mbar_init(drained, 1);
    mbar_init_fence();
    tma_prefetch(&p_map);
    tma_prefetch(&q_map);
  }
  __syncwarp();  // (what follows takes whole warps together)
  if (warp == kCopyWarp) {
    tmem_alloc<CTAS>(tmem_at, G::SLOT * G::SLOTS);
    tmem_alloc_done<CTAS>();
  }
  tc_fence_before();
  if constexpr (CTAS == 2) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  grid_wait();
  grid_release();

  const int tiles = run.p_tiles * run.q_tiles, blocks = run.blocks;
  const int first = blockIdx.x / CTAS, apart = gridDim.x / CTAS;
  bool alive = true;

  if (warp < kFirstResultWarp) {
    fewer_registers();
    if (warp == kCopyWarp && lane == 0) {  // -------------------------------- copies into the stages
      Ring<G::STAGES> r;
      int64_t issued = 0;
      for (int t = first; t < tiles && alive; t += apart) {
        int p, q;
        matmul_tile(run, t, p, q);
        const int p0 = (p * CTAS + rank) * kLanes, q0 = q * BN + rank * G::Q_ROWS;
        for (int kb = 0; kb < blocks; ++kb) {
          tc_wait(&empty[r.at], r.phase ^ 1u, alive, &g_matmul_fault, kMatmulFault);
          if (!alive) break;
          uint8_t* stage = smem + r.at * G::STAGE;
          // (a pair's copies are counted by the first CTA, which uses them)
          if (rank == 0) mbar_arrive_expect_tx(&full[r.at], CTAS * G::STAGE);
          if constexpr (CTAS == 2) {
            const uint32_t bar = cluster_addr(&full[r.at], 0);
            tma_load_pair(stage, &p_map, kb * kStep, p0, bar);
            tma_load_pair(stage + kLanes * kStep, &q_map, kb * kStep, q0, bar);
          } else {
            tma_load(stage, &p_map, kb * kStep, p0, &full[r.at]);
            tma_load(stage + kLanes * kStep, &q_map, kb * kStep, q0, &full[r.at]);
          }
          ++issued;
          r.next();
        }
      }
      if (!alive && rank == 0) {  // copies that nobody may have waited for
        bool wait = true;
        for (int64_t d = 0; d < G::STAGES && d < issued; ++d) {
          if (--r.at < 0) r.at = G::STAGES - 1, r.phase ^= 1u;
          tc_wait(&full[r.at], r.phase, wait, &g_matmul_fault, kMatmulFault);
        }
      }
    } else if (warp == kProductWarp && rank == 0) {  // ------------------------------- the products
      constexpr uint32_t instr = tc_instruction(CTAS * kLanes, BN, 0, 0, false, false);
      const uint64_t p_desc = tc_operand(smem_addr(smem), 16, 1024),
                     q_desc = tc_operand(smem_addr(smem) + kLanes * kStep, 16, 1024);
      Ring<G::STAGES> r;
      Ring<G::SLOTS> s;
      bool free = false, there = false;  // what the block's waits are for has been seen already
      for (int t = first; t < tiles && alive; t += apart)
        for (int kb = 0; kb < blocks; ++kb) {
          if (!free) tc_wait(&taken[s.at], s.phase ^ 1u, alive, &g_matmul_fault, kMatmulFault);
          if (!there) tc_wait(&full[r.at], r.phase, alive, &g_matmul_fault, kMatmulFault);
          if (!__all_sync(~0u, alive)) {
            alive = false;
            break;
          }
          tc_fence_after();
          const uint64_t at = static_cast<uint64_t>(r.at * (G::STAGE >> 4));
          const uint32_t to = tmem + s.at * G::SLOT;
          uint64_t *use = &empty[r.at], *done = &summed[s.at];
          r.next();
          s.next();
          there = mbar_test(&full[r.at], r.phase);
          free = mbar_test(&taken[s.at], s.phase ^ 1u);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc_mma_f8<CTAS>(to, p_desc + at + 2 * k, q_desc + at + 2 * k, instr, k > 0);
            tc_commit_to<CTAS>(done);
            tc_commit_to<CTAS>(use);
          }
          __syncwarp();
        }
      if (!alive) {
        bool wait = true;
        if (elect_one()) tc_commit_to<CTAS>(drained);
        __syncwarp();
        tc_wait(drained, 0, wait, &g_matmul_fault, kMatmulFault);
      }
    }
    if (warp >= kFirstScaleWarp) {  // ------------------------------------------------- the scales
      const bool of_p = warp == kFirstScaleWarp;
      const MatmulSide& side = of_p ? run.p : run.q;
      // rows of scales: all lanes of P; Q's columns, or the tiles of 128 that they are in
      constexpr int Q_SCALES = QROWS ? BN : (BN + 127) / 128;
      const int count = of_p ? kLanes : Q_SCALES, step = of_p || QROWS ? 1 : 128;
      float* to = of_p ? p_scales : q_scales;
      const int to_step = of_p ? kLanes : BN;
      Ring<G::GROUPS> x;
      for (int t = first; t < tiles; t += apart) {
        int p, q;
        matmul_tile(run, t, p, q);
        const int64_t row0 = of_p ? (static_cast<int64_t>(p) * CTAS + rank) * kLanes : static_cast<int64_t>(q) * BN;
        const float* from[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // (rows beyond the last take the first row's; nothing uses them)
          const int64_t row = row0 + static_cast<int64_t>(lane + 32 * i) * step;
          from[i] = side.scales + (row < side.rows ? row >> side.shift : 0) * side.row;
        }
        for (int kb = 0; kb < blocks; kb += G::GROUP) {
          tc_wait(&used[x.at], x.phase ^ 1u, alive, &g_matmul_fault, kMatmulFault);
          for (int b = 0; b < G::GROUP && kb + b < blocks; ++b)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (lane + 32 * i < count)
                cp_async4(to + (x.at * G::GROUP + b) * to_step + lane + 32 * i, from[i] + (kb + b) * side.block);
          cp_async_arrive_noinc(&scaled[x.at]);  // counts even with no copies of its own
          x.next();
        }
      }
      cp_async_commit();
      cp_async_wait<0>();
    }
  } else {  // -------------------------------------------------------------- scales, sums, results
    more_registers();
    constexpr int HALF = G::HALF, CHUNK = HALF % 32 ? 16 : 32;
    const int half = (warp - kFirstResultWarp) >> 2, in_cta = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21) + half * HALF;
    const uint32_t taken_at = CTAS == 2 ? cluster_addr(taken, 0) : smem_addr(taken);
    const float* qs0 = q_scales + (QROWS ? half * HALF : half * HALF / 128);
    Ring<G::SLOTS> s;
    Ring<G::GROUPS> x;
    for (int t = first; t < tiles; t += apart) {
      int p, q;
      matmul_tile(run, t, p, q);
      const int64_t p0 = (static_cast<int64_t>(p) * CTAS + rank) * kLanes + in_cta;
      const int64_t q0 = static_cast<int64_t>(q) * BN + half * HALF;
      f32x2 sums[HALF / 2];
#pragma unroll
      for (int i = 0; i < HALF / 2; ++i) sums[i] = f2(0.0f, 0.0f);
      const float bias = run.bias && run.bias_p && p0 < run.p.rows ? load_kind(run.bias, p0, run.y_kind) : 0.0f;
      for (int kb = 0; kb < blocks; ++kb) {
        const int in_group = kb % G::GROUP;
        if (in_group == 0) tc_wait(&scaled[x.at], x.phase, alive, &g_matmul_fault, kMatmulFault);
        const float* qs = qs0 + (x.at * G::GROUP + in_group) * BN;
        float scale = p_scales[(x.at * G::GROUP + in_group) * kLanes + in_cta];
        if constexpr (!QROWS) scale = __fmul_rn(scale, *qs);
        tc_wait(&summed[s.at], s.phase, alive, &g_matmul_fault, kMatmulFault);
        tc_fence_after();
        const uint32_t from = lanes + s.at * G::SLOT;
        uint32_t v[2][CHUNK];
        tmem_ld(from, v[0]);
#pragma unroll
        for (int c = 0; c < HALF; c += CHUNK) {
          uint32_t(&now)[CHUNK] = v[(c / CHUNK) & 1];
          tmem_ld_wait(now);
          if (c + CHUNK < HALF) {
            tmem_ld(from + c + CHUNK, v[(c / CHUNK + 1) & 1]);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if constexpr (CTAS == 2) mbar_arrive_cluster(taken_at + 8 * s.at);
              else mbar_arrive(&taken[s.at]);
            }
            s.next();
          }
#pragma unroll
          for (int i = 0; i < CHUNK; i += 4) {
            f32x2 y0 = f2(__uint_as_float(now[i]), __uint_as_float(now[i + 1])),
                  y1 = f2(__uint_as_float(now[i + 2]), __uint_as_float(now[i + 3]));
            if constexpr (QROWS) {
              const float4 w = *reinterpret_cast<const float4*>(qs + c + i);
              y0 = f2_mul(y0, f2(w.x, w.y));
              y1 = f2_mul(y1, f2(w.z, w.w));
            }
            sums[(c + i) / 2] = f2_fma(y0, f2(scale, scale), sums[(c + i) / 2]);
            sums[(c + i) / 2 + 1] = f2_fma(y1, f2(scale, scale), sums[(c + i) / 2 + 1]);
          }
        }
        if (in_group == G::GROUP - 1 || kb + 1 == blocks) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&used[x.at]);
          x.next();
        }
      }
      if (p0 < run.p.rows) {
        if (run.bias && run.bias_p) {
#pragma unroll
          for (int i = 0; i < HALF / 2; ++i) sums[i] = f2_add(sums[i], f2(bias, bias));
        }
#pragma unroll
        for (int i = 0; i < HALF; i += 8) {
          float v[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) f2_split(sums[i / 2 + k], v[2 * k], v[2 * k + 1]);
          store_sums(run, p0, q0 + i, v);
        }
      }
    }
  }
  __syncwarp();  // (as do the barrier and the release of tensor memory: the copies were one lane's)
  tc_fence_before();
  if constexpr (CTAS == 2) cluster_sync();
  else __syncthreads();
  if (warp == kCopyWarp) {
    tc_fence_after();
    tmem_free<CTAS>(tmem, G::SLOT * G::SLOTS);
  }
}

// swap: P is b. Tiles of p_side x q_side, of whose Q a CTA holds q_rows.
static cudaError_t describe(const MatmulArgs& a, bool swap, int p_side, int q_side, int q_rows, MatmulRun& run,
                            CUtensorMap& p_map, CUtensorMap& q_map) {
  const MatmulOperand &p = swap ? a.b : a.a, &q = swap ? a.a : a.b;
  const auto side = [](const MatmulOperand& o) {
    return MatmulSide{o.scales, o.scale_row, o.scale_block, o.rows, o.tile == 128 ? 7 : 0};
  };
  run.p = side(p);
  run.q = side(q);
  run.blocks = static_cast<int32_t>((a.depth + kStep - 1) / kStep);
  run.p_tiles = static_cast<int32_t>((p.rows + p_side - 1) / p_side);
  run.q_tiles = static_cast<int32_t>((q.rows + q_side - 1) / q_side);
  run.band = 8;
  run.y = a.y;
  run.y_p = swap ? 1 : a.y_stride;
  run.y_q = swap ? a.y_stride : 1;
  run.y_kind = a.y_kind;
  run.bias = a.bias;
  run.bias_p = swap;
  const int64_t size = a.y_kind == 2 ? 4 : 2;
  run.vec = !swap && ((reinterpret_cast<uintptr_t>(a.y) | static_cast<uintptr_t>(a.y_stride * size)) & 15) == 0;
  const cudaError_t e = make_tensor_map(&p_map, p.codes, 1, a.depth, p.rows, p.stride, 0, 0, kLanes);
  return e != cudaSuccess ? e : make_tensor_map(&q_map, q.codes, 1, a.depth, q.rows, q.stride, 0, 0, q_rows);
}

template <int CTAS, int BN, bool QROWS>
static cudaError_t run_tiles(const MatmulArgs& a, bool swap, cudaStream_t s) {
  using G = MatmulGeo<CTAS, BN, QROWS>;
  MatmulRun run{};
  CUtensorMap p_map, q_map;
  cudaError_t e = describe(a, swap, CTAS * kLanes, BN, G::Q_ROWS, run, p_map, q_map);
  auto kern = k_matmul_fp8<CTAS, BN, QROWS>;
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>(run.p_tiles) * run.q_tiles, most = 152 / CTAS;
  const unsigned grid = static_cast<unsigned>((tiles < most ? tiles : most) * CTAS);
  return launch_overlapped_cluster(kern, dim3(grid), CTAS, kTensorThreads, G::SMEM, s, p_map, q_map, run);
}


// ------------------------------------------------------------------------------------------------
// Few rows of a, or few tiles: P is b, 128 of its rows a CTA, and Q is a, up to BN rows. Bound by reading b, so what
// counts is that every SM has copies in flight until the end: CTAs are small enough that two share an
// SM, take one tile each, and the CTAs of a cluster share a tile's sum where there are few tiles
// (each adds up its part of the blocks; the parts are exchanged through shared memory and added in the order
// of the blocks, so the result does not depend on which CTA was first).
template <int BN>
struct FewGeo {
  static constexpr int RESULT_WARPS = BN == 128 ? 8 : 4;
  static constexpr int THREADS = (RESULT_WARPS + 4) * 32;
  static constexpr int PER_SM = BN == 128 ? 1 : 2;
  static constexpr int STAGE = (kLanes + BN) * kStep;
  static constexpr int STAGES = BN == 128 ? 6 : BN == 64 ? 4 : 5;
  static constexpr int SLOT = BN < 32 ? 32 : BN;
  static constexpr int SLOTS = 4;
  static constexpr int COLS = BN / (RESULT_WARPS / 4);  // of a warp
  static constexpr int GROUPS = 8;                      // blocks whose scales are on their way
  static constexpr int SCALES = STAGES * STAGE;
  static constexpr int BARS = SCALES + GROUPS * (kLanes + BN) * 4;
  static constexpr int SMEM = 1024 + BARS + (2 * STAGES + 2 * SLOTS + 2 * GROUPS + 1) * 8 + 16;
  static_assert(kLanes * BN * 4 <= STAGES * STAGE, "the exchanged sums take the stages' place");
};

template <int BN, bool QROWS>
__global__ void __launch_bounds__(FewGeo<BN>::THREADS, FewGeo<BN>::PER_SM)
    k_matmul_fp8_few(const __grid_constant__ CUtensorMap p_map, const __grid_constant__ CUtensorMap q_map,
                     const MatmulRun run, const int split) {
  using G = FewGeo<BN>;
  constexpr int R = G::RESULT_WARPS;  // warps R .. R + 3 copy, multiply, and fetch scales
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + G::BARS);
  uint64_t* empty = full + G::STAGES;
  uint64_t* summed = empty + G::STAGES;
  uint64_t* taken = summed + G::SLOTS;
  uint64_t* scaled = taken + G::SLOTS;
  uint64_t* used = scaled + G::GROUPS;
  uint64_t* drained = used + G::GROUPS;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(drained + 1);
  float* p_scales = reinterpret_cast<float*>(smem + G::SCALES);  // [GROUPS][kLanes]
  float* q_scales = p_scales + G::GROUPS * kLanes;               // [GROUPS][BN]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < G::STAGES; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
    for (int i = 0; i < G::SLOTS; ++i) mbar_init(&summed[i], 1), mbar_init(&taken[i], R);
    for (int i = 0; i < G::GROUPS; ++i) mbar_init(&scaled[i], 64), mbar_init(&used[i], R);
    mbar_init(drained, 1);
    mbar_init_fence();
    tma_prefetch(&p_map);
    tma_prefetch(&q_map);
  }
  if (warp == R) {
    tmem_alloc<1>(tmem_at, G::SLOT * G::SLOTS);
    tmem_alloc_done<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  grid_wait();
  grid_release();

  const int rank = blockIdx.x % split, tile = blockIdx.x / split;  // (a cluster is `split` CTAs in a row)
  const int p_tile = tile % run.p_tiles, q_tile = tile / run.p_tiles;
  const int begin = static_cast<int>(static_cast<int64_t>(run.blocks) * rank / split);
  const int end = static_cast<int>(static_cast<int64_t>(run.blocks) * (rank + 1) / split);
  bool alive = true;
  f32x2 sums[G::COLS / 2];
#pragma unroll
  for (int i = 0; i < G::COLS / 2; ++i) sums[i] = f2(0.0f, 0.0f);

  const int in_cta = (warp & 3) * 32 + lane;
  const int64_t p = static_cast<int64_t>(p_tile) * kLanes + in_cta, q0 = static_cast<int64_t>(q_tile) * BN;
  const float bias = run.bias && warp < R && p < run.p.rows ? load_kind(run.bias, p, run.y_kind) : 0.0f;

  if (warp == R) {
    if (lane == 0) {
      Ring<G::STAGES> r;
      int issued = 0;
      for (int kb = begin; kb < end; ++kb) {
        tc_wait(&empty[r.at], r.phase ^ 1u, alive, &g_matmul_fault, kMatmulFault);
        if (!alive) break;
        uint8_t* stage = smem + r.at * G::STAGE;
        mbar_arrive_expect_tx(&full[r.at], G::STAGE);
        tma_load(stage, &p_map, kb * kStep, p_tile * kLanes, &full[r.at]);
        tma_load(stage + kLanes * kStep, &q_map, kb * kStep, q_tile * BN, &full[r.at]);
        ++issued;
        r.next();
      }
      if (!alive) {  // copies that nobody may have waited for
        bool wait = true;
        for (int d = 0; d < G::STAGES && d < issued; ++d) {
          if (--r.at < 0) r.at = G::STAGES - 1, r.phase ^= 1u;
          tc_wait(&full[r.at], r.phase, wait, &g_matmul_fault, kMatmulFault);
        }
      }
    }
  } else if (warp == R + 1) {
    constexpr uint32_t instr = tc_instruction(kLanes, BN, 0, 0, false, false);
    const uint64_t p_desc = tc_operand(smem_addr(smem), 16, 1024),
                   q_desc = tc_operand(smem_addr(smem) + kLanes * kStep, 16, 1024);
    Ring<G::STAGES> r;
    Ring<G::SLOTS> s;
    for (int kb = begin; kb < end; ++kb) {
      tc_wait(&taken[s.at], s.phase ^ 1u, alive, &g_matmul_fault, kMatmulFault);
      tc_wait(&full[r.at], r.phase, alive, &g_matmul_fault, kMatmulFault);
      if (!__all_sync(~0u, alive)) {
        alive = false;
        break;
      }
      tc_fence_after();
      const uint64_t at = static_cast<uint64_t>(r.at * (G::STAGE >> 4));
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc_mma_f8<1>(tmem + s.at * G::SLOT, p_desc + at + 2 * k, q_desc + at + 2 * k, instr, k > 0);
        tc_commit(&summed[s.at]);
        tc_commit(&empty[r.at]);
      }
      __syncwarp();
      r.next();
      s.next();
    }
    if (!alive) {
      bool wait = true;
      if (elect_one()) tc_commit(drained);
      __syncwarp();
      tc_wait(drained, 0, wait, &g_matmul_fault, kMatmulFault);
    }
  } else if (warp >= R + 2) {
    const bool of_p = warp == R + 2;
    const MatmulSide& side = of_p ? run.p : run.q;
    const int64_t row0 = of_p ? static_cast<int64_t>(p_tile) * kLanes : static_cast<int64_t>(q_tile) * BN;
    const int count = side.shift ? 1 : of_p ? kLanes : BN;  // a tile of 128 rows has one scale
    float* to = of_p ? p_scales : q_scales;
    const int to_step = of_p ? kLanes : BN;
    const float* from[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // (rows beyond the last take the first row's; nothing uses them)
      const int64_t row = row0 + lane + 32 * i;
      from[i] = side.scales + (row < side.rows ? row >> side.shift : 0) * side.row;
    }
    Ring<G::GROUPS> x;
    for (int kb = begin; kb < end; ++kb) {
      tc_wait(&used[x.at], x.phase ^ 1u, alive, &g_matmul_fault, kMatmulFault);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < count) cp_async4(to + x.at * to_step + lane + 32 * i, from[i] + kb * side.block);
      cp_async_arrive_noinc(&scaled[x.at]);  // counts even with no copies of its own
      x.next();
    }
    cp_async_commit();
    cp_async_wait<0>();
  } else {
    constexpr int CHUNK = G::COLS < 32 ? G::COLS : 32;
    const int part = warp >> 2;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21) + part * G::COLS;
    const int p_at = run.p.shift ? 0 : in_cta;
    Ring<G::SLOTS> s;
    Ring<G::GROUPS> x;
    for (int kb = begin; kb < end; ++kb) {
      tc_wait(&scaled[x.at], x.phase, alive, &g_matmul_fault, kMatmulFault);
      const float* qs = q_scales + x.at * BN + (QROWS ? part * G::COLS : 0);
      float scale = p_scales[x.at * kLanes + p_at];
      if constexpr (!QROWS) scale = __fmul_rn(scale, *qs);
      tc_wait(&summed[s.at], s.phase, alive, &g_matmul_fault, kMatmulFault);
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < G::COLS; c += CHUNK) {
        uint32_t v[CHUNK];
        tmem_ld(lanes + s.at * G::SLOT + c, v);
        tmem_ld_wait(v);
        if (c + CHUNK == G::COLS) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&taken[s.at]);
        }
#pragma unroll
        for (int i = 0; i < CHUNK; i += 2) {
          f32x2 y = f2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
          if constexpr (QROWS) y = f2_mul(y, *reinterpret_cast<const f32x2*>(qs + c + i));
          sums[(c + i) / 2] = f2_fma(y, f2(scale, scale), sums[(c + i) / 2]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&used[x.at]);
      s.next();
      x.next();
    }
  }

  // Every product of this CTA has been read, so the stages are free; the other CTAs' are after the barrier.
  __syncwarp();
  const bool results = warp < R;
  const int part = warp >> 2;
  if (split == 1) {
    if (results && p < run.p.rows) {
#pragma unroll
      for (int i = 0; i < G::COLS / 2; ++i) {
        float a, b;
        f2_split(sums[i], a, b);
        store_one(run, p, q0 + part * G::COLS + 2 * i, a, bias);
        store_one(run, p, q0 + part * G::COLS + 2 * i + 1, b, bias);
      }
    }
  } else {
    // columns that a CTA adds up, a power of two: [source][column][lane] in its stages
    const int shift = __ffs(BN / split) - 1, own = 1 << shift;
    cluster_sync();
    if (results) {
      const uint32_t at = smem_addr(smem);
#pragma unroll
      for (int i = 0; i < G::COLS; ++i) {
        float a, b;
        f2_split(sums[i / 2], a, b);
        const int c = part * G::COLS + i, owner = c >> shift;
        st_cluster(map_rank(at + ((rank * own + (c & (own - 1))) * kLanes + in_cta) * 4, owner), (i & 1) ? b : a);
      }
    }
    cluster_sync();
    if (results && p < run.p.rows) {
      const float* parts = reinterpret_cast<const float*>(smem);
      for (int c = part; c < own; c += R / 4) {
        float sum = parts[c * kLanes + in_cta];
        for (int k = 1; k < split; ++k) sum = __fadd_rn(sum, parts[(k * own + c) * kLanes + in_cta]);
        store_one(run, p, q0 + rank * own + c, sum, bias);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == R) {
    tc_fence_after();
    tmem_free<1>(tmem, G::SLOT * G::SLOTS);
  }
}

template <int BN, bool QROWS>
static cudaError_t run_few_as(const MatmulArgs& a, cudaStream_t s) {
  using G = FewGeo<BN>;
  MatmulRun run{};
  CUtensorMap p_map, q_map;
  cudaError_t e = describe(a, true, kLanes, BN, BN, run, p_map, q_map);
  auto kern = k_matmul_fp8_few<BN, QROWS>;
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM);
  if (e != cudaSuccess) return e;
  // As many CTAs as run at one time, if each has two blocks or more.
  const int64_t tiles = static_cast<int64_t>(run.p_tiles) * run.q_tiles;
  int split = 1;
  while (split < 8 && tiles * split * 2 <= 152 * G::PER_SM && run.blocks >= 4 * split) split *= 2;
  return launch_overlapped_cluster(kern, dim3(static_cast<unsigned>(tiles * split)), split, G::THREADS, G::SMEM, s, p_map,
                                   q_map, run, split);
}
template <int BN>
static cudaError_t run_few(const MatmulArgs& a, cudaStream_t s) {
  return a.a.tile == 1 ? run_few_as<BN, true>(a, s) : run_few_as<BN, false>(a, s);
}

template <int CTAS, int BN>
static cudaError_t run_tiles(const MatmulArgs& a, bool swap, cudaStream_t s) {
  return (swap ? a.a : a.b).tile == 1 ? run_tiles<CTAS, BN, true>(a, swap, s) : run_tiles<CTAS, BN, false>(a, swap, s);
}

cudaError_t launch_matmul_fp8(const MatmulArgs& a, cudaStream_t s) {
  if (a.a.rows <= 16) return run_few<16>(a, s);
  if (a.a.rows <= 32) return run_few<32>(a, s);
  if (a.a.rows <= 64) return run_few<64>(a, s);
  // So few tiles and so long a sum that the CTAs of a cluster share each (100 x 1024 x 8192: 11 us from 28;
  // at a depth of 4096 both take 13 us, at 1024 the exchange costs 3 us more than it saves).
  const int64_t squares = ((a.a.rows + 127) / 128) * ((a.b.rows + 127) / 128);
  if (squares <= 38 && a.depth > 32 * kStep) return run_few<128>(a, s);
  // A warp's stores: 32 rows of P, 16 bytes of each, or, with P and Q exchanged, 32 neighbours. So
  // they are exchanged where y's rows do not start at multiples of 16 bytes, and where a fits one tile's
  // columns (77 x 50001 x 1003 in fp32: 20 us against 65).
  const int64_t size = a.y_kind == 2 ? 4 : 2;
  const bool whole = ((reinterpret_cast<uintptr_t>(a.y) | static_cast<uintptr_t>(a.y_stride * size)) & 15) == 0;
  const bool swap = a.a.rows <= 128 || !whole;
  // Squares of 128 while one round takes them (1024 x 2048 x 4096: 128 of them 14.6 us, 32 pairs 19.1), then
  // pairs (1280 x 2304 x 4096: 180 squares 26.4 us, 45 pairs 21.1).
  if (a.a.rows > 128 && squares > 152) return run_tiles<2, 256>(a, swap, s);
  return a.a.rows <= 96 ? run_tiles<1, 96>(a, true, s) : run_tiles<1, 128>(a, swap, s);
}

cudaError_t read_matmul_fault(unsigned* flags, bool clear) {
  const cudaError_t err = cudaMemcpyFromSymbol(flags, g_matmul_fault, sizeof(unsigned));
  if (err != cudaSuccess || !clear) return err;
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_matmul_fault, &zero, sizeof(unsigned));
}

}  // namespace zpp
