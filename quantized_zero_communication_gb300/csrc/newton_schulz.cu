// newton_schulz.cu -- K14: the products of the Newton-Schulz steps on the tensor cores.
//
//   A = X X^T,  B = b A + c A A,  X = a X + B X          (X with fewer rows than columns; else A = X^T X
//                                                          and X = a X + X B)
//
// Operands are fp16, sums fp32 in tensor memory. What the steps lose early they multiply by up to 3.4^5,
// so plain 16-bit operands are poor: bf16 leaves 1.1e-2 of the result's norm in error on normal values
// of 512 x 1024, fp16 1.3e-3, and 4.6e-2 and 6.8e-3 where singular values lie over four decades. Hence:
//
//  - What fp16 loses of X is kept in a second fp16 and enters a X. (B hardly reaches the directions that
//    grow most, so B X does with the first.)
//  - The diagonals of A and B are kept in fp32 and enter elementwise:
//      A = A' + D,  A A = A' A' + D A' + A' D + D D,  B X = B' X + E X
//    A' and B' are small beside them, and so is what their rounding and X's leaves. In E X, X counts
//    with both parts; with the first alone while three steps or more follow, where B X of a direction
//    that is still to grow has to cancel.
//  - Matrices with a side of up to 128 take all products of both parts but the smallest.
//
// That leaves 0.2e-3 .. 1.1e-3, and 1e-6 .. 3e-6 for the small ones (256 x 1024 noise 0.5e-3).
//
// A and B are symmetric: only tiles on and above the diagonal are computed, and stored twice.
#include "newton_schulz.cuh"
#include "zpp_overlap.cuh"
#include "zpp_tcgen05.cuh"

namespace zpp {

static __device__ unsigned g_muon_fault;
constexpr unsigned kMuonFault = 16;  // its bit of the fault word

constexpr int kNsSide = 128, kNsStep = 64;  // rows of an operand in a CTA, steps of the sum in a stage
constexpr int kNsOperand = kNsSide * kNsStep * 2;
constexpr int kNsStage = 2 * kNsOperand;
constexpr int kNsStages = 6;
constexpr int kNsBars = kNsStages * kNsStage;
constexpr int kNsSmem = 1024 + kNsBars + (2 * kNsStages + 2 * 2 + 1) * 8 + 16;
// Tiles are squares of CTAS * 128: of one CTA, or of a pair that holds half of each operand.
constexpr int kNsSlots = 2;

struct NsTile {
  int group, matrix, p, q;
};
__device__ __forceinline__ NsTile ns_tile(const NsLaunch& n, int t) {
  NsTile r;
  r.group = 0;
  while (r.group + 1 < n.groups && n.group[r.group + 1].first_tile <= t) ++r.group;
  const NsGroup& g = n.group[r.group];
  int in = t - g.first_tile;
  r.matrix = in / g.per_matrix;
  in -= r.matrix * g.per_matrix;
  if (n.op <= kNsPoly) {  // row by row of the upper triangle
    r.p = 0;
    int left = g.p_tiles;
    while (in >= left) in -= left, --left, ++r.p;
    r.q = r.p + in;
  } else {
    r.p = in % g.p_tiles;
    r.q = in / g.p_tiles;
  }
  return r;
}

// 128 rows of an operand, from row `at` on, over 64 steps of the sum from k on.
template <int CTAS>
__device__ __forceinline__ void ns_load(uint8_t* dst, const CUtensorMap* map, bool mn, int at, int k, int z,
                                        uint64_t* bar) {
  if constexpr (CTAS == 2) {
    const uint32_t there = cluster_addr(bar, 0);
    tma_load_pair(dst, map, mn ? at : k, mn ? k : at, z, there);
    if (mn) tma_load_pair(dst + kNsOperand / 2, map, at + 64, k, z, there);
  } else {
    tma_load(dst, map, mn ? at : k, mn ? k : at, z, bar);
    if (mn) tma_load(dst + kNsOperand / 2, map, at + 64, k, z, bar);
  }
}
__device__ __forceinline__ uint64_t ns_operand(uint32_t at, bool mn) {
  return mn ? tc_operand(at, kNsOperand / 2, 1024) : tc_operand(at, 16, 1024);
}

// v as two fp16 each: the nearest ones, and those nearest to what they lost.
__device__ __forceinline__ void two_halves(const float (&v)[8], uint4& high, uint4& low) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    h[k] = pack2(v[2 * k], v[2 * k + 1], F16());
    const float2 f = unpack2(h[k], F16());
    l[k] = pack2(__fsub_rn(v[2 * k], f.x), __fsub_rn(v[2 * k + 1], f.y), F16());
  }
  high = make_uint4(h[0], h[1], h[2], h[3]);
  low = make_uint4(l[0], l[1], l[2], l[3]);
}
__device__ __forceinline__ void halves(const uint16_t* at, float (&v)[8]) {
  const uint4 w = ld_after_v4(at);
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = unpack2(u[k], F16());
    v[2 * k] = f.x, v[2 * k + 1] = f.y;
  }
}
__device__ __forceinline__ void mirror8(uint16_t* to, const NsGroup& g, int p, int q, uint4 w) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (q + i < g.cols) to[static_cast<int64_t>(q + i) * g.ld + p] = static_cast<uint16_t>(u[i >> 1] >> (16 * (i & 1)));
}

// 8 consecutive columns of row p, from column q on (a multiple of 8).
__device__ __forceinline__ void ns_store(const NsLaunch& n, const NsGroup& g, int matrix, bool mirror, int p,
                                         int q, float (&d)[8]) {
  const int64_t base = static_cast<int64_t>(matrix) * g.apart;
  const int64_t at = base + static_cast<int64_t>(p) * g.ld + q;
  uint4 high, low;
  if (n.op <= kNsPoly) {
    if (n.op == kNsGram) {
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = __fmul_rn(d[i], 1.0f / (kXScale * kXScale));
    } else {
      const float* diag = g.diag_in + static_cast<int64_t>(matrix) * g.diag_apart;
      const float dp = ld_after_f32(diag + p);
      float x[8], dq[8];
      halves(g.in + at, x);
      if (g.in_low) {
        halves(g.in_low + at, dq);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __fadd_rn(x[i], dq[i]);
      }
      const uint4 w0 = ld_after_shared_v4(diag + q), w1 = ld_after_shared_v4(diag + q + 4);
      const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dq[i] = __uint_as_float(w[i]);
        const float a = p == q + i ? dp : x[i], with = p == q + i ? dp : __fadd_rn(dp, dq[i]);
        d[i] = __fmaf_rn(n.c, __fmaf_rn(with, a, d[i]), __fmul_rn(n.b, a));
      }
    }
    if (p >= q && p < q + 8) {
      float* to = g.diag_out + static_cast<int64_t>(matrix) * g.diag_apart + p;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (p == q + i) *to = d[i], d[i] = 0.0f;
    }
    two_halves(d, high, low);
    st_v4(g.out + at, high);
    if (mirror) mirror8(g.out + base, g, p, q, high);
    if (g.out_low) {
      st_v4(g.out_low + at, low);
      if (mirror) mirror8(g.out_low + base, g, p, q, low);
    }
    return;
  }
  // B is on the left of a matrix with fewer rows than columns, its diagonal goes by rows there.
  const float* diag = g.diag_in + static_cast<int64_t>(matrix) * g.diag_apart;
  float x[8], l[8], e[8];
  halves(g.in + at, x);
  halves(g.in_low + at, l);
  if (g.q_mn) {
    const float v = ld_after_f32(diag + p);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = v;
  } else {
    const uint4 w0 = ld_after_shared_v4(diag + q), w1 = ld_after_shared_v4(diag + q + 4);
    const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = __uint_as_float(w[i]);
  }
  const bool both = !n.early || g.parts == 3;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float w = __fadd_rn(x[i], l[i]);
    d[i] = __fmaf_rn(n.a, w, __fmaf_rn(e[i], both ? w : x[i], d[i]));
  }
  if (n.op == kNsApply) {
    two_halves(d, high, low);
    st_v4(g.out + at, high);
    st_v4(g.out_low + at, low);
    return;
  }
  const NsResult& res = n.result[g.first_matrix + matrix];
  const int64_t flat = static_cast<int64_t>(p) * g.cols + q;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (q + i >= g.cols) break;
    float v = __fmul_rn(d[i], 1.0f / kXScale);
    if (res.param) {
      v = __fmaf_rn(-g.step, v, __fmul_rn(res.param[flat + i], n.decay));
      res.param[flat + i] = v;
    }
    if (res.out) {
      uint16_t* o = static_cast<uint16_t*>(res.out) + flat + i;
      *o = static_cast<uint16_t>(n.out_kind == 0 ? pack2(v, v, F16()) : pack2(v, v, BF16()));
    }
  }
}

template <int CTAS>
__global__ void __launch_bounds__(kTensorThreads, 1) k_newton_schulz(const __grid_constant__ NsLaunch n) {
  constexpr int TILE = CTAS * kNsSide, HALF = TILE / 2;  // columns of a warp
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kNsBars);
  uint64_t* empty = full + kNsStages;
  uint64_t* summed = empty + kNsStages;
  uint64_t* taken = summed + kNsSlots;
  uint64_t* drained = taken + kNsSlots;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(drained + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CTAS == 2 ? cluster_rank() : 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kNsStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
    for (int i = 0; i < kNsSlots; ++i) mbar_init(&summed[i], 1), mbar_init(&taken[i], CTAS * kResultWarps);
    mbar_init(drained, 1);
    mbar_init_fence();
  }
  if (warp == kCopyWarp) {
    tmem_alloc<CTAS>(tmem_at, TILE * kNsSlots);
    tmem_alloc_done<CTAS>();
  }
  tc_fence_before();
  if constexpr (CTAS == 2) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  grid_wait();
  grid_release();
  const int first = blockIdx.x / CTAS, apart = gridDim.x / CTAS;
  bool alive = true;

  if (warp == kCopyWarp && lane == 0) {  // ----------------------------------- copies into the stages
    Ring<kNsStages> r;
    int64_t issued = 0;
    for (int t = first; t < n.tiles && alive; t += apart) {
      const NsTile at = ns_tile(n, t);
      const NsGroup& g = n.group[at.group];
      const int p0 = at.p * TILE + rank * kNsSide, q0 = at.q * TILE + rank * kNsSide;
      for (int part = 0; part < g.parts && alive; ++part) {
        const CUtensorMap *p = part == 2 ? &g.p_low : &g.p, *q = part == 1 ? &g.q_low : &g.q;
        for (int k = 0; k < g.depth; k += kNsStep) {
          tc_wait(&empty[r.at], r.phase ^ 1u, alive, &g_muon_fault, kMuonFault);
          if (!alive) break;
          uint8_t* stage = smem + r.at * kNsStage;
          // (a pair's copies are counted by the first CTA, which uses them)
          if (rank == 0) mbar_arrive_expect_tx(&full[r.at], CTAS * kNsStage);
          ns_load<CTAS>(stage, p, g.p_mn, p0, k, at.matrix, &full[r.at]);
          ns_load<CTAS>(stage + kNsOperand, q, g.q_mn, q0, k, at.matrix, &full[r.at]);
          ++issued;
          r.next();
        }
      }
    }
    if (!alive && rank == 0) {  // copies that nobody may have waited for
      bool wait = true;
      for (int64_t d = 0; d < kNsStages && d < issued; ++d) {
        if (--r.at < 0) r.at = kNsStages - 1, r.phase ^= 1u;
        tc_wait(&full[r.at], r.phase, wait, &g_muon_fault, kMuonFault);
      }
    }
  } else if (warp == kProductWarp && rank == 0) {  // ------------------------------------ the products
    Ring<kNsStages> r;
    Ring<kNsSlots> s;
    for (int t = first; t < n.tiles && alive; t += apart) {
      const NsGroup& g = n.group[ns_tile(n, t).group];
      const uint32_t instr = tc_instruction(TILE, TILE, 0, 0, g.p_mn, g.q_mn);
      const uint32_t base = smem_addr(smem), to = tmem + s.at * TILE;
      const uint64_t p_desc = ns_operand(base, g.p_mn), q_desc = ns_operand(base + kNsOperand, g.q_mn);
      const uint64_t p_step = g.p_mn ? 2048 >> 4 : 32 >> 4, q_step = g.q_mn ? 2048 >> 4 : 32 >> 4;
      const int stages = g.parts * ((g.depth + kNsStep - 1) / kNsStep);
      tc_wait(&taken[s.at], s.phase ^ 1u, alive, &g_muon_fault, kMuonFault);
      bool there = false;  // the stage has been seen already
      for (int k = 0; k < stages; ++k) {
        if (!there) tc_wait(&full[r.at], r.phase, alive, &g_muon_fault, kMuonFault);
        if (!__all_sync(~0u, alive)) {
          alive = false;
          break;
        }
        tc_fence_after();
        const uint64_t at = static_cast<uint64_t>(r.at * (kNsStage >> 4));
        uint64_t* use = &empty[r.at];
        r.next();
        there = mbar_test(&full[r.at], r.phase);
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            tc_mma_f16<CTAS>(to, p_desc + at + j * p_step, q_desc + at + j * q_step, instr, k > 0 || j > 0);
          tc_commit_to<CTAS>(use);
          if (k + 1 == stages) tc_commit_to<CTAS>(&summed[s.at]);
        }
        __syncwarp();
      }
      s.next();
    }
    if (!alive) {
      bool wait = true;
      if (elect_one()) tc_commit_to<CTAS>(drained);
      __syncwarp();
      tc_wait(drained, 0, wait, &g_muon_fault, kMuonFault);
    }
  } else if (warp >= kFirstResultWarp) {  // ---------------------------------------------- the results
    const int half = (warp - kFirstResultWarp) >> 2;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21) + half * HALF;
    const uint32_t taken_at = CTAS == 2 ? cluster_addr(taken, 0) : 0;
    const bool skip = n.op == kNsLast && n.factor && !isfinite(ld_after_f32(n.factor));
    Ring<kNsSlots> s;
    for (int t = first; t < n.tiles; t += apart) {
      const NsTile at = ns_tile(n, t);
      const NsGroup& g = n.group[at.group];
      const int p = at.p * TILE + rank * kNsSide + (warp & 3) * 32 + lane;
      tc_wait(&summed[s.at], s.phase, alive, &g_muon_fault, kMuonFault);
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < HALF; c += 32) {
        uint32_t v[32];
        tmem_ld(lanes + s.at * TILE + c, v);
        tmem_ld_wait(v);
        if (c + 32 == HALF) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if constexpr (CTAS == 2) mbar_arrive_cluster(taken_at + 8 * s.at);
            else mbar_arrive(&taken[s.at]);
          }
        }
        if (p < g.rows && !skip) {
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            const int q = at.q * TILE + half * HALF + c + j;
            float d[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = __uint_as_float(v[j + i]);
            if (q < g.cols) ns_store(n, g, at.matrix, at.p != at.q, p, q, d);
          }
        }
      }
      s.next();
    }
  }
  tc_fence_before();
  if constexpr (CTAS == 2) cluster_sync();
  else __syncthreads();
  if (warp == kCopyWarp) {
    tc_fence_after();
    tmem_free<CTAS>(tmem, TILE * kNsSlots);
  }
}

template <int CTAS>
static cudaError_t run_ns(const NsLaunch& n, cudaStream_t s) {
  const cudaError_t e =
      cudaFuncSetAttribute(k_newton_schulz<CTAS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kNsSmem);
  if (e != cudaSuccess) return e;
  const int most = 152 / CTAS;
  return launch_overlapped_cluster(k_newton_schulz<CTAS>,
                                   dim3(static_cast<unsigned>((n.tiles < most ? n.tiles : most) * CTAS)), CTAS,
                                   kTensorThreads, kNsSmem, s, n);
}
cudaError_t launch_ns(const NsLaunch& n, cudaStream_t s) { return n.side == 256 ? run_ns<2>(n, s) : run_ns<1>(n, s); }

cudaError_t read_muon_fault(unsigned* flags, bool clear) {
  const cudaError_t err = cudaMemcpyFromSymbol(flags, g_muon_fault, sizeof(unsigned));
  if (err != cudaSuccess || !clear) return err;
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_muon_fault, &zero, sizeof(unsigned));
}

}  // namespace zpp
