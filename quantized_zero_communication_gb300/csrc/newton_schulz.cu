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
#include <atomic>

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

// ------------------------------------------------------------------------- between two products
// Every CTA of the launch ends a product before any begins the next one. `arrived` counts ends; each role
// of a CTA waits for it by itself. (The launch is cooperative, so all CTAs run at once.)
constexpr long long kGridWaitClocks = 40000000000ll;  // some 20 s: a product may take long
__device__ __forceinline__ void ns_wait_grid(const uint32_t* arrived, uint32_t ends, bool& alive) {
  const long long t0 = clock64();
  while (alive) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(arrived) : "memory");
    if (v >= ends) return;
    if (clock64() - t0 > kGridWaitClocks) {
      alive = false;
      atomicOr(&g_muon_fault, kMuonFault);
    }
  }
}
// By every thread that wrote, before one of them tells: the next product's copies read through another
// path (the asynchronous proxy).
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async;" ::: "memory"); }

struct NsTile {
  int shape, matrix, p, q;
};
template <typename L>
__device__ __forceinline__ NsTile ns_tile(const L& n, int op, int t) {
  const int kind = op == kNsApply;
  NsTile r;
  r.shape = 0;
  while (r.shape + 1 < n.shapes && n.shape[r.shape + 1].first_tile[kind] <= t) ++r.shape;
  const NsShape& g = n.shape[r.shape];
  int in = t - g.first_tile[kind];
  if (kind) {
    const int per = g.row_tiles * g.col_tiles;
    r.matrix = in / per;
    in -= r.matrix * per;
    // bands of 8 tiles down, column by column: the CTAs at work at one time share both operands in L2
    const int band = 8 * g.col_tiles, b = in / band, height = min(8, g.row_tiles - 8 * b);
    in -= b * band;
    r.p = 8 * b + in % height;
    r.q = in / height;
  } else {
    const int per = g.side_tiles * (g.side_tiles + 1) / 2;
    r.matrix = in / per;
    in -= r.matrix * per;
    r.p = 0;  // row by row of the upper triangle
    for (int left = g.side_tiles; in >= left; --left) in -= left, ++r.p;
    r.q = r.p + in;
  }
  return r;
}
__device__ __forceinline__ int ns_depth(const NsShape& g, int op) {
  return (op == kNsGram) == (g.wide != 0) ? g.cols : g.rows;  // gram: the longer side, else the shorter
}
// Whether the operands' rows are steps of the sum.
__device__ __forceinline__ bool ns_p_mn(const NsShape& g, int op) { return op == kNsGram && !g.wide; }
__device__ __forceinline__ bool ns_q_mn(const NsShape& g, int op) {
  return op == kNsGram ? !g.wide : op == kNsApply && g.wide;
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

// ---------------------------------------------------------------------------------------- the results
// A thread has a row p and 16 consecutive columns at a time, from q on (a multiple of 16). Rows of the
// matrices in the workspace start at multiples of 32 bytes, so whole vectors of 16 stay inside them.
struct NsIn {         // what a result needs beside its sum
  U8x32 x, low;       // poly: A; apply: X
  float diag_p;       // of A (poly) or B (apply) at the row
  float diag_q[16];   // at the columns
};
__device__ __forceinline__ void ns_diag_q(const float* diag, float (&d)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 w = ld_after_shared_v4(diag + 4 * i);
    d[4 * i] = __uint_as_float(w.x), d[4 * i + 1] = __uint_as_float(w.y);
    d[4 * i + 2] = __uint_as_float(w.z), d[4 * i + 3] = __uint_as_float(w.w);
  }
}
__device__ __forceinline__ void ns_fetch(const NsShape& g, int op, int from, int matrix, int p, int q, NsIn& in) {
  if (op == kNsGram) return;
  const bool apply = op == kNsApply;
  const int64_t at = matrix * (apply ? g.x_apart : g.a_apart) + static_cast<int64_t>(p) * (apply ? g.x_ld : g.a_ld) + q;
  in.x = ld_after_vec32<true>((apply ? g.x_at[from] : g.a_at) + at);
  if (apply || g.exact) in.low = ld_after_vec32<true>((apply ? g.x_low_at[from] : g.a_low_at) + at);
  const float* diag = (apply ? g.b_diag : g.a_diag) + static_cast<int64_t>(matrix) * g.diag_apart;
  if (!apply || g.wide) in.diag_p = ld_after_f32(diag + p);
  if (!apply || !g.wide) ns_diag_q(diag + q, in.diag_q);
}
__device__ __forceinline__ void halves(const U8x32& w, float (&v)[16]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 f = unpack2(w.w[k], F16());
    v[2 * k] = f.x, v[2 * k + 1] = f.y;
  }
}
// v as two fp16 each: the nearest ones, and those nearest to what they lost.
__device__ __forceinline__ void two_halves(const float (&v)[16], U8x32& high, U8x32& low) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    high.w[k] = pack2(v[2 * k], v[2 * k + 1], F16());
    const float2 f = unpack2(high.w[k], F16());
    low.w[k] = pack2(__fsub_rn(v[2 * k], f.x), __fsub_rn(v[2 * k + 1], f.y), F16());
  }
}
// The transposed place of 16 columns of a row: a warp's 32 rows lie side by side there.
__device__ __forceinline__ void ns_mirror(uint16_t* to, int ld, int side, int p, int q, const U8x32& w) {
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (q + i < side) to[static_cast<int64_t>(q + i) * ld + p] = static_cast<uint16_t>(w.w[i >> 1] >> (16 * (i & 1)));
}

__device__ __forceinline__ void ns_symmetric(const NsShape& g, int op, float b, float c, int matrix, bool mirror,
                                             int p, int q, int side, const NsIn& in, float (&d)[16]) {
  if (op == kNsGram) {
#pragma unroll
    for (int i = 0; i < 16; ++i) d[i] = __fmul_rn(d[i], 1.0f / (kXScale * kXScale));
  } else {
    float x[16];
    halves(in.x, x);
    if (g.exact) {
      float l[16];
      halves(in.low, l);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = __fadd_rn(x[i], l[i]);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const bool on = p == q + i;  // the diagonal: A' is 0 there
      const float a = on ? in.diag_p : x[i], with = on ? in.diag_p : __fadd_rn(in.diag_p, in.diag_q[i]);
      d[i] = __fmaf_rn(c, __fmaf_rn(with, a, d[i]), __fmul_rn(b, a));
    }
  }
  if (p >= q && p < q + 16) {
    float* to = (op == kNsGram ? g.a_diag : g.b_diag) + static_cast<int64_t>(matrix) * g.diag_apart + p;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (p == q + i) *to = d[i], d[i] = 0.0f;
  }
  U8x32 high, low;
  two_halves(d, high, low);
  const int64_t base = matrix * g.a_apart, at = base + static_cast<int64_t>(p) * g.a_ld + q;
  uint16_t* to = op == kNsGram ? g.a_at : g.b_at;
  st_v8(to + at, high);
  if (mirror) ns_mirror(to + base, g.a_ld, side, p, q, high);
  if (g.exact) {
    to = op == kNsGram ? g.a_low_at : g.b_low_at;
    st_v8(to + at, low);
    if (mirror) ns_mirror(to + base, g.a_ld, side, p, q, low);
  }
}
// a X + B X from B' X (d): X counts with its first part alone in E X where `early`.
__device__ __forceinline__ void ns_applied(const NsShape& g, float a, bool early, const NsIn& in, float (&d)[16]) {
  float x[16], l[16];
  halves(in.x, x);
  halves(in.low, l);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float w = __fadd_rn(x[i], l[i]), e = g.wide ? in.diag_p : in.diag_q[i];
    d[i] = __fmaf_rn(a, w, __fmaf_rn(e, early && !g.exact ? x[i] : w, d[i]));
  }
}
template <typename L>
__device__ __forceinline__ void ns_result(const L& n, const NsShape& g, int matrix, int p, int q, float (&d)[16]) {
  const NsResult& r = n.result[g.first_matrix + matrix];
  const int64_t at = static_cast<int64_t>(p) * g.cols + q;
  float* param = r.param + at;
  uint16_t* out = static_cast<uint16_t*>(r.out) + at;
#pragma unroll
  for (int i = 0; i < 16; ++i) d[i] = __fmul_rn(d[i], 1.0f / kXScale);
  if (r.param) {
    const bool vec = q + 16 <= g.cols && (reinterpret_cast<uintptr_t>(param) & 31) == 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (vec) {
        U8x32 w = ld_after_vec32<true>(param + 8 * h);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          d[8 * h + i] = __fmaf_rn(-g.step, d[8 * h + i], __fmul_rn(__uint_as_float(w.w[i]), n.decay));
          w.w[i] = __float_as_uint(d[8 * h + i]);
        }
        st_v8(param + 8 * h, w);
      } else {
#pragma unroll
        for (int i = 8 * h; i < 8 * h + 8; ++i)
          if (q + i < g.cols) param[i] = d[i] = __fmaf_rn(-g.step, d[i], __fmul_rn(param[i], n.decay));
      }
    }
  }
  if (r.out) {
    U8x32 w;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      w.w[k] = n.out_kind == 0 ? pack2(d[2 * k], d[2 * k + 1], F16()) : pack2(d[2 * k], d[2 * k + 1], BF16());
    if (q + 16 <= g.cols && (reinterpret_cast<uintptr_t>(out) & 31) == 0) {
      st_v8(out, w);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (q + i < g.cols) out[i] = static_cast<uint16_t>(w.w[i >> 1] >> (16 * (i & 1)));
    }
  }
}

template <int CTAS, typename L>
__global__ void __launch_bounds__(kTensorThreads, 1) k_newton_schulz(const __grid_constant__ L n) {
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
  const int first = blockIdx.x / CTAS, apart = gridDim.x / CTAS;
  const int ops = 3 * n.steps;
  bool alive = true;

  if (warp == kCopyWarp && lane == 0) {  // ----------------------------------- copies into the stages
    Ring<kNsStages> r;
    int64_t issued = 0;
    for (int at_op = 0; at_op < ops && alive; ++at_op) {
      const int op = at_op % 3, from = (at_op / 3) & 1, tiles = n.tiles[op == kNsApply];
      ns_wait_grid(n.arrived, at_op * gridDim.x, alive);
      proxy_fence();
      for (int t = first; t < tiles && alive; t += apart) {
        const NsTile at = ns_tile(n, op, t);
        const NsShape& g = n.shape[at.shape];
        const int p0 = at.p * TILE + rank * kNsSide, q0 = at.q * TILE + rank * kNsSide;
        const bool p_mn = ns_p_mn(g, op), q_mn = ns_q_mn(g, op);
        const int depth = ns_depth(g, op), parts = g.exact ? 3 : 1;
        for (int part = 0; part < parts && alive; ++part) {
          const bool p_low = part == 2, q_low = part == 1;
          const CUtensorMap *p, *q;
          if (op == kNsGram) {
            p = p_low ? &g.x_low[from] : &g.x[from], q = q_low ? &g.x_low[from] : &g.x[from];
          } else if (op == kNsPoly) {
            p = p_low ? &g.a_low : &g.a, q = q_low ? &g.a_low : &g.a;
          } else {
            p = p_low ? &g.b_low : &g.b, q = q_low ? &g.xt_low[from] : &g.xt[from];
            if (!g.wide) p = p_low ? &g.xt_low[from] : &g.xt[from], q = q_low ? &g.b_low : &g.b;
          }
          for (int k = 0; k < depth; k += kNsStep) {
            tc_wait(&empty[r.at], r.phase ^ 1u, alive, &g_muon_fault, kMuonFault);
            if (!alive) break;
            uint8_t* stage = smem + r.at * kNsStage;
            // (a pair's copies are counted by the first CTA, which uses them)
            if (rank == 0) mbar_arrive_expect_tx(&full[r.at], CTAS * kNsStage);
            ns_load<CTAS>(stage, p, p_mn, p0, k, at.matrix, &full[r.at]);
            ns_load<CTAS>(stage + kNsOperand, q, q_mn, q0, k, at.matrix, &full[r.at]);
            ++issued;
            r.next();
          }
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
    for (int at_op = 0; at_op < ops && alive; ++at_op) {
      const int op = at_op % 3, tiles = n.tiles[op == kNsApply];
      ns_wait_grid(n.arrived, at_op * gridDim.x, alive);
      for (int t = first; t < tiles && alive; t += apart) {
        const NsShape& g = n.shape[ns_tile(n, op, t).shape];
        const bool p_mn = ns_p_mn(g, op), q_mn = ns_q_mn(g, op);
        const uint32_t instr = tc_instruction(TILE, TILE, 0, 0, p_mn, q_mn);
        const uint32_t base = smem_addr(smem), to = tmem + s.at * TILE;
        const uint64_t p_desc = ns_operand(base, p_mn), q_desc = ns_operand(base + kNsOperand, q_mn);
        const uint64_t p_step = p_mn ? 2048 >> 4 : 32 >> 4, q_step = q_mn ? 2048 >> 4 : 32 >> 4;
        const int stages = (g.exact ? 3 : 1) * ((ns_depth(g, op) + kNsStep - 1) / kNsStep);
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
    const bool skip = n.factor && !isfinite(ld_after_f32(n.factor));
    Ring<kNsSlots> s;
    for (int at_op = 0; at_op < ops; ++at_op) {
      const int op = at_op % 3, step = at_op / 3, from = step & 1, tiles = n.tiles[op == kNsApply];
      const float a = n.coefficients[3 * step], b = n.coefficients[3 * step + 1], c = n.coefficients[3 * step + 2];
      const bool early = step < n.steps - 3, last = step == n.steps - 1;
      if (threadIdx.x == kFirstResultWarp * 32) ns_wait_grid(n.arrived, at_op * gridDim.x, alive);
      named_barrier(1, kResultWarps * 32);
      for (int t = first; t < tiles; t += apart) {
        const NsTile at = ns_tile(n, op, t);
        const NsShape& g = n.shape[at.shape];
        const int small = g.wide ? g.rows : g.cols;
        const int rows = op == kNsApply ? g.rows : small, cols = op == kNsApply ? g.cols : small;
        const int p = at.p * TILE + rank * kNsSide + (warp & 3) * 32 + lane, q0 = at.q * TILE + half * HALF;
        const bool on = p < rows && !(skip && op == kNsApply && last);
        NsIn in[2];
        if (on && q0 < cols) ns_fetch(g, op, from, at.matrix, p, q0, in[0]);
        tc_wait_long(&summed[s.at], s.phase, alive, &g_muon_fault, kMuonFault, kGridWaitClocks);
        tc_fence_after();
#pragma unroll 2
        for (int k = 0; k < HALF / 16; ++k) {
          const int q = q0 + 16 * k;
          uint32_t v[16];
          tmem_ld(lanes + s.at * TILE + 16 * k, v);
          if (k + 1 < HALF / 16 && on && q + 16 < cols) ns_fetch(g, op, from, at.matrix, p, q + 16, in[(k + 1) & 1]);
          tmem_ld_wait(v);
          if (k + 1 == HALF / 16) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if constexpr (CTAS == 2) mbar_arrive_cluster(taken_at + 8 * s.at);
              else mbar_arrive(&taken[s.at]);
            }
          }
          if (on && q < cols) {
            float d[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) d[i] = __uint_as_float(v[i]);
            if (op != kNsApply) {
              ns_symmetric(g, op, b, c, at.matrix, at.p != at.q, p, q, small, in[k & 1], d);
            } else {
              ns_applied(g, a, early, in[k & 1], d);
              if (last) {
                ns_result(n, g, at.matrix, p, q, d);
              } else {
                U8x32 high, low;
                two_halves(d, high, low);
                const int64_t to = at.matrix * g.x_apart + static_cast<int64_t>(p) * g.x_ld + q;
                st_v8(g.x_at[from ^ 1] + to, high);
                st_v8(g.x_low_at[from ^ 1] + to, low);
              }
            }
          }
        }
        s.next();
      }
      proxy_fence();
      named_barrier(1, kResultWarps * 32);
      if (threadIdx.x == kFirstResultWarp * 32) {
        __threadfence();
        asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(n.arrived) : "memory");
      }
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

template <int CTAS, typename L>
static cudaError_t run_ns(const L& n, cudaStream_t s) {
  auto kern = k_newton_schulz<CTAS, L>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(152);
  cfg.blockDim = dim3(kTensorThreads);
  cfg.dynamicSmemBytes = kNsSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CTAS;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeCooperative;
  attr[1].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // Clusters that run at one time (no more may wait for each other), asked once for a device.
  static std::atomic<int> known[64];
  int device = 0, fit = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  if (device < 64) fit = known[device].load(std::memory_order_acquire);
  if (fit == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kNsSmem);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&fit, kern, &cfg);
    if (e != cudaSuccess) return e;
    if (fit < 1) return cudaErrorCooperativeLaunchTooLarge;
    if (device < 64) known[device].store(fit, std::memory_order_release);
  }
  const int tiles = n.tiles[0] > n.tiles[1] ? n.tiles[0] : n.tiles[1];
  cfg.gridDim = dim3(static_cast<unsigned>((tiles < fit ? tiles : fit) * CTAS));
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, n);
}
template <typename L>
static cudaError_t run_ns(const L& n, int side, cudaStream_t s) {
  return side == 256 ? run_ns<2>(n, s) : run_ns<1>(n, s);
}
cudaError_t launch_ns(const NsLaunch& n, int side, cudaStream_t s) {
  const NsShape& last = n.shape[n.shapes - 1];
  if (n.shapes > 2 || last.first_matrix + last.count > 32) return run_ns(n, side, s);
  NsLaunchFew few;  // (a launch's parameters are copied by the driver)
  few.steps = n.steps, few.shapes = n.shapes, few.tiles[0] = n.tiles[0], few.tiles[1] = n.tiles[1];
  few.out_kind = n.out_kind, few.decay = n.decay, few.factor = n.factor, few.arrived = n.arrived;
  for (int i = 0; i < 3 * n.steps; ++i) few.coefficients[i] = n.coefficients[i];
  for (int i = 0; i < last.first_matrix + last.count; ++i) few.result[i] = n.result[i];
  for (int i = 0; i < n.shapes; ++i) few.shape[i] = n.shape[i];
  return run_ns(few, side, s);
}

cudaError_t read_muon_fault(unsigned* flags, bool clear) {
  const cudaError_t err = cudaMemcpyFromSymbol(flags, g_muon_fault, sizeof(unsigned));
  if (err != cudaSuccess || !clear) return err;
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_muon_fault, &zero, sizeof(unsigned));
}

}  // namespace zpp
