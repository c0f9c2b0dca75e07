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

constexpr int kNsTile = 128, kNsStep = 64;  // tile side, steps of the sum in a stage
constexpr int kNsOperand = kNsTile * kNsStep * 2;
constexpr int kNsStage = 2 * kNsOperand;
constexpr int kNsStages = 6, kNsSlots = 4;
constexpr int kNsBars = kNsStages * kNsStage;
constexpr int kNsSmem = 1024 + kNsBars + (2 * kNsStages + 2 * kNsSlots + 1) * 8 + 16;
constexpr int kNsWarps = 8;  // of the epilogue
constexpr int kNsThreads = (kNsWarps + 2) * 32;

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

__device__ __forceinline__ void ns_load(uint8_t* dst, const CUtensorMap* map, bool mn, int at, int k, int z,
                                        uint64_t* bar) {
  if (mn) {
    tma_load(dst, map, at, k, z, bar);
    tma_load(dst + kNsOperand / 2, map, at + 64, k, z, bar);
  } else {
    tma_load(dst, map, k, at, z, bar);
  }
}
__device__ __forceinline__ uint64_t ns_operand(uint32_t at, bool mn, int k) {
  return mn ? tc_operand(at + 2048 * k, kNsOperand / 2, 1024) : tc_operand(at + 32 * k, 16, 1024);
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

__global__ void __launch_bounds__(kNsThreads, 1) k_newton_schulz(const __grid_constant__ NsLaunch n) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kNsBars);
  uint64_t* empty = full + kNsStages;
  uint64_t* summed = empty + kNsStages;
  uint64_t* taken = summed + kNsSlots;
  uint64_t* drained = taken + kNsSlots;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(drained + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kNsStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
    for (int i = 0; i < kNsSlots; ++i) mbar_init(&summed[i], 1), mbar_init(&taken[i], kNsWarps);
    mbar_init(drained, 1);
    mbar_init_fence();
  }
  if (warp == kNsWarps) {
    tmem_alloc<1>(tmem_at, kNsTile * kNsSlots);
    tmem_alloc_done<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  grid_wait();
  grid_release();
  bool alive = true;

  if (warp == kNsWarps) {  // ------------------------------------------------- copies into the stages
    if (lane == 0) {
      Ring<kNsStages> r;
      int64_t issued = 0;
      for (int t = blockIdx.x; t < n.tiles && alive; t += gridDim.x) {
        const NsTile at = ns_tile(n, t);
        const NsGroup& g = n.group[at.group];
        for (int part = 0; part < g.parts && alive; ++part) {
          const CUtensorMap *p = part == 2 ? &g.p_low : &g.p, *q = part == 1 ? &g.q_low : &g.q;
          for (int k = 0; k < g.depth; k += kNsStep) {
            tc_wait(&empty[r.at], r.phase ^ 1u, alive, &g_muon_fault, kMuonFault);
            if (!alive) break;
            uint8_t* stage = smem + r.at * kNsStage;
            mbar_arrive_expect_tx(&full[r.at], kNsStage);
            ns_load(stage, p, g.p_mn, at.p * kNsTile, k, at.matrix, &full[r.at]);
            ns_load(stage + kNsOperand, q, g.q_mn, at.q * kNsTile, k, at.matrix, &full[r.at]);
            ++issued;
            r.next();
          }
        }
      }
      if (!alive) {  // copies that nobody may have waited for
        bool wait = true;
        for (int64_t d = 0; d < kNsStages && d < issued; ++d) {
          if (--r.at < 0) r.at = kNsStages - 1, r.phase ^= 1u;
          tc_wait(&full[r.at], r.phase, wait, &g_muon_fault, kMuonFault);
        }
      }
    }
  } else if (warp == kNsWarps + 1) {  // ------------------------------------------------ the products
    if (lane == 0) {
      Ring<kNsStages> r;
      Ring<kNsSlots> s;
      for (int t = blockIdx.x; t < n.tiles && alive; t += gridDim.x) {
        const NsGroup& g = n.group[ns_tile(n, t).group];
        const uint32_t instr = tc_instruction(kNsTile, kNsTile, 0, 0, g.p_mn, g.q_mn);
        tc_wait(&taken[s.at], s.phase ^ 1u, alive, &g_muon_fault, kMuonFault);
        const int stages = g.parts * ((g.depth + kNsStep - 1) / kNsStep);
        for (int k = 0; k < stages; ++k) {
          tc_wait(&full[r.at], r.phase, alive, &g_muon_fault, kMuonFault);
          if (!alive) break;
          tc_fence_after();
          const uint32_t p = smem_addr(smem + r.at * kNsStage), q = p + kNsOperand;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            tc_mma_f16<1>(tmem + s.at * kNsTile, ns_operand(p, g.p_mn, j), ns_operand(q, g.q_mn, j), instr,
                          k > 0 || j > 0);
          tc_commit(&empty[r.at]);
          r.next();
        }
        if (!alive) break;
        tc_commit(&summed[s.at]);
        s.next();
      }
      if (!alive) {
        bool wait = true;
        tc_commit(drained);
        tc_wait(drained, 0, wait, &g_muon_fault, kMuonFault);
      }
    }
  } else {  // -------------------------------------------------------------------------- the results
    const int half = warp >> 2;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21) + half * (kNsTile / 2);
    const bool skip = n.op == kNsLast && n.factor && !isfinite(ld_after_f32(n.factor));
    Ring<kNsSlots> s;
    for (int t = blockIdx.x; t < n.tiles; t += gridDim.x) {
      const NsTile at = ns_tile(n, t);
      const NsGroup& g = n.group[at.group];
      const int p = at.p * kNsTile + (warp & 3) * 32 + lane;
      tc_wait(&summed[s.at], s.phase, alive, &g_muon_fault, kMuonFault);
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < kNsTile / 2; c += 32) {
        uint32_t v[32];
        tmem_ld(lanes + s.at * kNsTile + c, v);
        tmem_ld_wait(v);
        if (c + 32 == kNsTile / 2) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&taken[s.at]);
        }
        if (p < g.rows && !skip) {
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            const int q = at.q * kNsTile + half * (kNsTile / 2) + c + j;
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
  __syncthreads();
  if (warp == kNsWarps) {
    tc_fence_after();
    tmem_free<1>(tmem, kNsTile * kNsSlots);
  }
}

cudaError_t launch_ns(const NsLaunch& n, cudaStream_t s) {
  const cudaError_t e =
      cudaFuncSetAttribute(k_newton_schulz, cudaFuncAttributeMaxDynamicSharedMemorySize, kNsSmem);
  if (e != cudaSuccess) return e;
  return launch_overlapped_smem(k_newton_schulz, dim3(static_cast<unsigned>(n.tiles < 152 ? n.tiles : 152)),
                                kNsThreads, kNsSmem, s, n);
}

cudaError_t read_muon_fault(unsigned* flags, bool clear) {
  const cudaError_t err = cudaMemcpyFromSymbol(flags, g_muon_fault, sizeof(unsigned));
  if (err != cudaSuccess || !clear) return err;
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_muon_fault, &zero, sizeof(unsigned));
}

}  // namespace zpp
