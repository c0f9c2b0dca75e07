// newton_schulz.cu -- K14: the products of the Newton-Schulz steps on the tensor cores.
//
//   A = X X^T,  B = b A + c A A,  X = a X + B X          (X with fewer rows than columns; else A = X^T X
//                                                          and X = a X + X B)
//
// Sums are fp32 in tensor memory, operands fp16, each value in two of them: the nearest one and the one nearest
// to what that lost. A product takes three of the unit's: first by first part, first by second, second by first.
// What the steps lose early they multiply by up to 3.4^5, so one 16-bit part is poor: bf16 leaves 1.1e-2 of the
// result's norm in error on normal values of 512 x 1024, fp16 1.3e-3, and 4.6e-2 and 6.8e-3 where singular values lie
// over four decades. One part with the diagonals apart, as below, leaves 0.2e-3 .. 1.1e-3 in 1/2.8 of the time,
// several times the rounding of an fp16 result; two leave 2e-6 (256 x 1024) .. 1e-5 (4096 x 16384), as fp32 products do.
//
// The diagonals of A and B are kept in fp32 and enter elementwise:
//   A = A' + D,  A A = A' A' + D A' + A' D + D D,  B X = B' X + E X
// A' and B' are small beside them, and so is what their rounding and X's leaves.
//
// The two products with a second part come first in a sum: the matrix unit cuts the running sum to fp32 in each of
// its steps, and what is cut is in proportion to it. It adds up a limited number of steps in a row (kNsRun).
//
// Tiles of 128 x 128, or of 256 x 256 by a pair of CTAs, a stage 64 steps of a product (5 stages of 32 KB), the sums
// of two tiles in tensor memory, so that one is taken while the next is made. Large matrices are bound
// by the matrix unit at the clock that the power limit leaves (4096 x 16384: 9.1 ms, 1.5 PFLOP/s of the three
// products); sides of 1024 by what a CTA can take in (64 bytes a clock); small ones by the way from one product to
// the next (256 x 1024: 15 of them 195 us).
//
// A and B are symmetric: only tiles on and above the diagonal are computed, and stored twice (the second time
// turned in shared memory, where the tile lies). Where X is long
// and A has few tiles, several CTAs share a tile's sum and another pass adds their parts.
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
constexpr int kNsStages = 5;
// Results go through shared memory: 128 rows of 64 columns at a time, of each half of the tile's columns,
// as 16-bit values and what those lost, laid out as a tensor copy lays them.
constexpr int kNsChunk = 64, kNsHalfChunk = kNsSide * kNsChunk * 2;
constexpr int kNsResults = kNsStages * kNsStage;
constexpr int kNsDiag = kNsResults + 2 * 2 * kNsHalfChunk;  // and the diagonal at a chunk's columns
constexpr int kNsBars = kNsDiag + 2 * kNsChunk * 4;
constexpr int kNsSmem = 1024 + kNsBars + (2 * kNsStages + 2 * 2 + 2 + 2) * 8 + 16;
static_assert(kNsSmem <= 227 * 1024, "shared memory of a CTA");
// Tiles are squares of CTAS * 128: of one CTA, or of a pair that holds half of each operand.
constexpr int kNsSlots = 2;

// ------------------------------------------------------------------------- between two products
// Every CTA of the launch ends a product before any begins the next one. `arrived` counts ends; one thread
// of a CTA reads it (the count's line is one place in L2: asked by every role it answers later), and the
// others wait for that thread. (The launch is cooperative, so all CTAs run at once.)
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
// Between other threads' ordinary writes, which this one knows of, and copies: those go through another path
// (the asynchronous proxy).
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async;" ::: "memory"); }

// The kind of op `at_op` of a launch, the ops of a step being `per`: 3, or 4 with the join.
__device__ __forceinline__ int ns_op(int at_op, int per) {
  const int k = per == 3 ? at_op % 3 : at_op & 3;
  return k == 0 ? kNsGram : k == per - 1 ? kNsApply : k == per - 2 ? kNsPoly : kNsJoin;
}
// Which of NsLaunch::tiles an op walks over.
__device__ __forceinline__ int ns_kind(int op) { return op == kNsApply ? 1 : op == kNsGram ? 2 : 0; }
struct NsTile {
  int shape, matrix, p, q;
  int unit, part;  // (symmetric) the tile's number in its shape; the part of its sum (gram)
};
template <typename L>
__device__ __forceinline__ NsTile ns_tile(const L& n, bool join, int op, int t) {
  const int kind = ns_kind(op);
  NsTile r;
  r.shape = 0;
  while (r.shape + 1 < n.shapes && n.shape[r.shape + 1].first_tile[kind] <= t) ++r.shape;
  const NsShape& g = n.shape[r.shape];
  int in = t - g.first_tile[kind];
  r.unit = r.part = 0;
  if (kind == 1) {
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
    if (join && kind == 2 && g.split > 1) {
      const int whole = in / g.split;
      r.part = in - whole * g.split;
      in = whole;
    }
    r.unit = in;
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
// The stages that a tile's sum has in each of the three products; the first of a part of it.
__device__ __forceinline__ int ns_stages(const NsShape& g, int op) {
  return (ns_depth(g, op) + kNsStep - 1) / kNsStep;
}
__device__ __forceinline__ int ns_stage(const NsShape& g, bool join, int op, int stages, int part) {
  if (!join || op != kNsGram || g.split == 1) return part * stages;
  return static_cast<int>(static_cast<int64_t>(stages) * part / g.split);
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
// A thread has a row of a chunk, 8 consecutive columns (16 bytes) at a time.
__device__ __forceinline__ uint8_t* ns_place(uint8_t* chunk, int row, int piece) {
  return chunk + row * 128 + ((piece ^ (row & 7)) << 4);
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
__device__ __forceinline__ void eight(const float* at, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(at), b = *reinterpret_cast<const float4*>(at + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
// What a tile's results are made with. (From the kernel's parameters, which lie in constant memory beyond
// what its cache holds: read again for every 8 columns they took 5000 clocks of a chunk.)
template <typename T>
__device__ __forceinline__ T held_in_register(T v) {
  if constexpr (std::is_same_v<T, float>) asm volatile("" : "+f"(v));
  else if constexpr (sizeof(T) == 8) asm volatile("" : "+l"(v));
  else asm volatile("" : "+r"(v));
  return v;
}
struct NsTask {
  int op, wide;
  int diagonal;     // a symmetric tile on it; the others go to their transposed place too
  float* diag_out;
  float a, b, c;
};
__device__ __forceinline__ void halves(const uint4& w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = unpack2(u[k], F16());
    v[2 * k] = f.x, v[2 * k + 1] = f.y;
  }
}
// A (gram) or B (poly) from the sums d; high, low: A's values, dp, diag: its diagonal at the row and at
// the columns (poly).
__device__ __forceinline__ void ns_symmetric(const NsTask& g, int p, int q, float dp, const float* diag,
                                             const uint4& high, const uint4& low, float (&d)[8]) {
  if (g.op == kNsGram) {
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = __fmul_rn(d[i], 1.0f / (kXScale * kXScale));
  } else {
    float x[8], l[8], dq[8];
    eight(diag, dq);
    halves(high, x);
    halves(low, l);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __fadd_rn(x[i], l[i]);
    if (!g.diagonal) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        d[i] = __fmaf_rn(g.c, __fmaf_rn(__fadd_rn(dp, dq[i]), x[i], d[i]), __fmul_rn(g.b, x[i]));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool on = p == q + i;  // (A' is 0 there)
        const float a = on ? dp : x[i], with = on ? dp : __fadd_rn(dp, dq[i]);
        d[i] = __fmaf_rn(g.c, __fmaf_rn(with, a, d[i]), __fmul_rn(g.b, a));
      }
    }
  }
  if (g.diagonal && p >= q && p < q + 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (p == q + i) g.diag_out[p] = d[i], d[i] = 0.0f;
  }
}
// a X + B X from B' X (d); high, low: X.
__device__ __forceinline__ void ns_applied(const NsTask& g, float diag_p, const float* diag, const uint4& high,
                                           const uint4& low, float (&d)[8]) {
  float x[8], l[8], e[8];
  if (g.wide) {
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = diag_p;
  } else {
    eight(diag, e);
  }
  halves(high, x);
  halves(low, l);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float w = __fadd_rn(x[i], l[i]);
    d[i] = __fmaf_rn(g.a, w, __fmaf_rn(e[i], w, d[i]));
  }
}
// 32 columns of a row from where the runs before left them, added to this run's.
__device__ __forceinline__ void add_run(const float* from, uint32_t (&v)[32]) {
  uint4 f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = *reinterpret_cast<const uint4*>(from + i * kNsSide * 4);
  const auto add = [](uint32_t a, uint32_t b) { return __float_as_uint(__fadd_rn(__uint_as_float(a), __uint_as_float(b))); };
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[4 * i] = add(f[i].x, v[4 * i]);
    v[4 * i + 1] = add(f[i].y, v[4 * i + 1]);
    v[4 * i + 2] = add(f[i].z, v[4 * i + 2]);
    v[4 * i + 3] = add(f[i].w, v[4 * i + 3]);
  }
}
// 8 columns of a row to their place in the transposed chunk: 64 rows of columns, twice 64 of the 128 rows. A
// warp's 32 rows lie side by side there.
__device__ __forceinline__ void ns_turn(uint8_t* chunk, int row, int col, const uint4& w) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  uint8_t* half = chunk + (row >> 6) * (kNsHalfChunk / 2) + (row & 7) * 2;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<uint16_t*>(half + (col + i) * 128 + ((((row >> 3) & 7) ^ ((col + i) & 7)) << 4)) =
        static_cast<uint16_t>(u[i >> 1] >> (16 * (i & 1)));
}
// A chunk of fp32 results, whose upper and lower 16 bits lie in its two parts, to where they go: a warp
// takes 32 rows, 8 of them at a time (so that as many loads are under way), two columns a lane.
template <typename L>
__device__ __forceinline__ void ns_result(const L& n, const NsShape& g, int matrix, int p0, int q0,
                                          const uint8_t* high, const uint8_t* low, int warp, int lane) {
  const NsResult& res = n.result[g.first_matrix + matrix];
  const int q = q0 + 2 * lane, left = g.cols - q, rows = g.rows - p0;
  if (left <= 0) return;
  const int64_t cols = g.cols;
  float* const param = res.param ? res.param + p0 * cols + q : nullptr;
  uint16_t* const out = res.out ? static_cast<uint16_t*>(res.out) + p0 * cols + q : nullptr;
  const bool pair = left >= 2 && (cols & 1) == 0;  // both columns by one access
  const bool param_pair = pair && (reinterpret_cast<uintptr_t>(param) & 7) == 0;
  const bool out_pair = pair && (reinterpret_cast<uintptr_t>(out) & 3) == 0;
  const float step = g.step, decay = n.decay;
  const bool f16 = n.out_kind == 0;
#pragma unroll 1
  for (int r0 = warp * 32; r0 < warp * 32 + 32 && r0 < rows; r0 += 8) {
    float2 old[8];
    if (param) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float* at = param + (r0 + i) * cols;
        if (r0 + i < rows) {
          if (param_pair) old[i] = *reinterpret_cast<const float2*>(at);
          else old[i] = make_float2(at[0], left >= 2 ? at[1] : 0.0f);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = r0 + i;
      if (row >= rows) break;
      const uint32_t at = row * 128 + (((lane >> 2) ^ (row & 7)) << 4) + (lane & 3) * 4;
      const uint32_t h = *reinterpret_cast<const uint32_t*>(high + at), l = *reinterpret_cast<const uint32_t*>(low + at);
      float x = __uint_as_float(__byte_perm(h, l, 0x1054u)), y = __uint_as_float(__byte_perm(h, l, 0x3276u));
      if (param) {
        x = __fmaf_rn(-step, x, __fmul_rn(old[i].x, decay));
        y = __fmaf_rn(-step, y, __fmul_rn(old[i].y, decay));
        float* to = param + row * cols;
        if (param_pair) {
          *reinterpret_cast<float2*>(to) = make_float2(x, y);
        } else {
          to[0] = x;
          if (left >= 2) to[1] = y;
        }
      }
      if (out) {
        uint16_t* to = out + row * cols;
        const uint32_t w = f16 ? pack2(x, y, F16()) : pack2(x, y, BF16());
        if (out_pair) {
          *reinterpret_cast<uint32_t*>(to) = w;
        } else {
          to[0] = static_cast<uint16_t>(w);
          if (left >= 2) to[1] = static_cast<uint16_t>(w >> 16);
        }
      }
    }
  }
}
// The old parameters of a row of a chunk, brought into L2 while its sums are made.
template <typename L>
__device__ __forceinline__ void ns_result_ahead(const L& n, const NsShape& g, int matrix, int p, int q0, int cols) {
  const float* param = n.result[g.first_matrix + matrix].param;
  if (!param) return;
  const float* at = param + static_cast<int64_t>(p) * g.cols + q0;
  const int left = g.cols - q0 < cols ? g.cols - q0 : cols;
  if (left > 0 && (reinterpret_cast<uintptr_t>(at) & 15) == 0 && left * 4 >= 16)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"(static_cast<uint32_t>(left * 4) & ~15u)
                 : "memory");
}

// The parts of the grams' sums, in their order, and what ns_symmetric makes of them: by every result warp, 32
// rows and 4 columns at a time.
template <int CTAS, typename L>
__device__ __forceinline__ void ns_join(const L& n, int warp, int lane) {
  constexpr int TILE = CTAS * kNsSide, ITEMS = (TILE / 4) * (TILE / 32);
  const int total = n.tiles[0] * ITEMS;
  for (int w = blockIdx.x * kResultWarps + warp; w < total; w += gridDim.x * kResultWarps) {
    const int t = w / ITEMS, item = w - t * ITEMS;
    const NsTile at = ns_tile(n, true, kNsPoly, t);
    const NsShape& g = n.shape[at.shape];
    if (g.split == 1) continue;
    const int cg = item / (TILE / 32), row = item % (TILE / 32) * 32 + lane;
    const int side = g.wide ? g.rows : g.cols, p = at.p * TILE + row, q = at.q * TILE + 4 * cg;
    if (p >= side || q >= side) continue;
    const int64_t unit = g.first_tile[2] + static_cast<int64_t>(at.unit) * g.split;
    const float* from = n.partial + unit * TILE * TILE + (cg * TILE + row) * 4;
    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k = 0; k < g.split; ++k) {
      const uint4 v = ld_after_v4(from + static_cast<int64_t>(k) * TILE * TILE);
      d[0] = __fadd_rn(d[0], __uint_as_float(v.x)), d[1] = __fadd_rn(d[1], __uint_as_float(v.y));
      d[2] = __fadd_rn(d[2], __uint_as_float(v.z)), d[3] = __fadd_rn(d[3], __uint_as_float(v.w));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      d[i] = __fmul_rn(d[i], 1.0f / (kXScale * kXScale));
      if (p == q + i) g.a_diag[static_cast<int64_t>(at.matrix) * g.diag_apart + p] = d[i], d[i] = 0.0f;
    }
    const uint32_t h[2] = {pack2(d[0], d[1], F16()), pack2(d[2], d[3], F16())};
    const float2 f0 = unpack2(h[0], F16()), f1 = unpack2(h[1], F16());
    const uint32_t l[2] = {pack2(__fsub_rn(d[0], f0.x), __fsub_rn(d[1], f0.y), F16()),
                           pack2(__fsub_rn(d[2], f1.x), __fsub_rn(d[3], f1.y), F16())};
    const int64_t base = at.matrix * g.a_apart, to = base + static_cast<int64_t>(p) * g.a_ld + q;
    st_v2(g.a_at + to, make_uint2(h[0], h[1]));
    st_v2(g.a_low_at + to, make_uint2(l[0], l[1]));
    if (at.p != at.q) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (q + i < side) {
          const int64_t turned = base + static_cast<int64_t>(q + i) * g.a_ld + p;
          g.a_at[turned] = static_cast<uint16_t>(h[i >> 1] >> (16 * (i & 1)));
          g.a_low_at[turned] = static_cast<uint16_t>(l[i >> 1] >> (16 * (i & 1)));
        }
    }
  }
}

// join: some shape's sums are split. (A kernel of its own: the others run 3 % slower with the code in it.)
template <int CTAS, bool join, typename L>
__global__ void __launch_bounds__(kTensorThreads, 1) k_newton_schulz(const __grid_constant__ L n) {
  constexpr int TILE = CTAS * kNsSide, HALF = TILE / 2;  // columns of a warp
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kNsBars);
  uint64_t* empty = full + kNsStages;
  uint64_t* summed = empty + kNsStages;
  uint64_t* taken = summed + kNsSlots;
  uint64_t* held = taken + kNsSlots;  // a half's chunk holds what its results need
  uint64_t* go = held + 2;  // the product before has ended everywhere
  uint64_t* drained = go + 1;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(drained + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CTAS == 2 ? cluster_rank() : 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kNsStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
    for (int i = 0; i < kNsSlots; ++i) mbar_init(&summed[i], 1), mbar_init(&taken[i], CTAS * kResultWarps);
    mbar_init(&held[0], 1);
    mbar_init(&held[1], 1);
    mbar_init(go, 1);
    mbar_init(drained, 1);
    mbar_init_fence();
  }
  __syncwarp();  // (what follows takes whole warps together)
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
  constexpr int per = join ? 4 : 3;
  const int ops = per * n.steps;
  bool alive = true;

  if (warp == kCopyWarp && lane == 0) {  // ----------------------------------- copies into the stages
    Ring<kNsStages> r;
    int64_t issued = 0;
    // The descriptors of a few shapes, at hand from the start (a first use waits for its own).
    for (int k = 0; k < n.shapes && k < 2; ++k) {
      const NsShape& g = n.shape[k];
      for (int i = 0; i < 2; ++i) {
        tma_prefetch(&g.x[i]);
        tma_prefetch(&g.xt[i]);
        tma_prefetch(&g.x_low[i]);
        tma_prefetch(&g.xt_low[i]);
      }
      tma_prefetch(&g.a);
      tma_prefetch(&g.b);
      tma_prefetch(&g.a_low);
      tma_prefetch(&g.b_low);
    }
    for (int at_op = 0; at_op < ops && alive; ++at_op) {
      const int op = ns_op(at_op, per), from = (at_op / per) & 1;
      const int tiles = op == kNsJoin ? 0 : held_in_register(n.tiles[ns_kind(op)]);
      NsTile next{};  // (looked up before the wait)
      if (first < tiles) next = ns_tile(n, join, op, first);
      ns_wait_grid(n.arrived, at_op * gridDim.x, alive);
      mbar_arrive(go);
      proxy_fence();
      for (int t = first; t < tiles && alive; t += apart) {
        const NsTile at = t == first ? next : ns_tile(n, join, op, t);
        const NsShape& g = n.shape[at.shape];
        const int p0 = at.p * TILE + rank * kNsSide, q0 = at.q * TILE + rank * kNsSide;
        const bool p_mn = ns_p_mn(g, op), q_mn = ns_q_mn(g, op);
        const int stages = ns_stages(g, op);
        const int begin = ns_stage(g, join, op, stages, at.part), end = ns_stage(g, join, op, stages, at.part + 1);
        // (the two small products first: each step cuts the running sum to fp32)
        for (int part = 0; part < kNsProducts && alive; ++part) {
          const bool p_low = part == 0, q_low = part == 1;
          const CUtensorMap *p, *q;
          if (op == kNsGram) {
            p = p_low ? &g.x_low[from] : &g.x[from], q = q_low ? &g.x_low[from] : &g.x[from];
          } else if (op == kNsPoly) {
            p = p_low ? &g.a_low : &g.a, q = q_low ? &g.a_low : &g.a;
          } else {
            p = p_low ? &g.b_low : &g.b, q = q_low ? &g.xt_low[from] : &g.xt[from];
            if (!g.wide) p = p_low ? &g.xt_low[from] : &g.xt[from], q = q_low ? &g.b_low : &g.b;
          }
          for (int k = begin * kNsStep; k < end * kNsStep; k += kNsStep) {
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
      const int op = ns_op(at_op, per), tiles = op == kNsJoin ? 0 : n.tiles[ns_kind(op)];
      for (int t = first; t < tiles && alive; t += apart) {
        const NsTile tile = ns_tile(n, join, op, t);
        const NsShape& g = n.shape[tile.shape];
        const bool p_mn = ns_p_mn(g, op), q_mn = ns_q_mn(g, op);
        const uint32_t instr = tc_instruction(TILE, TILE, 0, 0, p_mn, q_mn);
        const uint32_t base = smem_addr(smem);
        const uint64_t p_desc = ns_operand(base, p_mn), q_desc = ns_operand(base + kNsOperand, q_mn);
        const uint64_t p_step = p_mn ? 2048 >> 4 : 32 >> 4, q_step = q_mn ? 2048 >> 4 : 32 >> 4;
        const int whole = ns_stages(g, op),
                  each = ns_stage(g, join, op, whole, tile.part + 1) - ns_stage(g, join, op, whole, tile.part),
                  stages = kNsProducts * each;
        bool there = false;  // the stage has been seen already
        for (int run = 0, end; run < stages && alive; run = end) {
          end = min((run == 0 ? stages - each : run) + kNsRun, stages);
          const uint32_t to = tmem + s.at * TILE;
          tc_wait(&taken[s.at], s.phase ^ 1u, alive, &g_muon_fault, kMuonFault);
          for (int k = run; k < end; ++k) {
            // (the first copies of a product come when it begins)
            if (!there) tc_wait_long(&full[r.at], r.phase, alive, &g_muon_fault, kMuonFault, kGridWaitClocks);
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
                tc_mma_f16<CTAS>(to, p_desc + at + j * p_step, q_desc + at + j * q_step, instr, k > run || j > 0);
              tc_commit_to<CTAS>(use);
              if (k + 1 == end) tc_commit_to<CTAS>(&summed[s.at]);
            }
            __syncwarp();
          }
          s.next();
        }
      }
    }
    if (!alive) {
      bool wait = true;
      if (elect_one()) tc_commit_to<CTAS>(drained);
      __syncwarp();
      tc_wait(drained, 0, wait, &g_muon_fault, kMuonFault);
    }
  } else if (warp >= kFirstResultWarp) {  // ---------------------------------------------- the results
    const int half = (warp - kFirstResultWarp) >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21) + half * HALF;
    const uint32_t taken_at = CTAS == 2 ? cluster_addr(taken, 0) : 0;
    uint8_t* high = smem + kNsResults + half * 2 * kNsHalfChunk;
    uint8_t* low = high + kNsHalfChunk;
    float* diag_q = reinterpret_cast<float*>(smem + kNsDiag) + half * kNsChunk;
    const bool leader = row == 0;  // of the 4 warps of a half
    const bool skip = n.factor && !isfinite(ld_after_f32(n.factor));
    // this thread's place among the sums that runs leave: [columns / 4][rows][4] for a CTA
    float* const runs = n.runs + static_cast<int64_t>(blockIdx.x) * kNsSide * TILE + (half * (HALF / 4) * kNsSide + row) * 4;
    unsigned held_phase = 0;
    Ring<kNsSlots> s;
    for (int at_op = 0; at_op < ops; ++at_op) {
      const int op = ns_op(at_op, per), step = at_op / per, from = step & 1;
      const int tiles = op == kNsJoin ? 0 : n.tiles[ns_kind(op)];
      const bool last = op == kNsApply && step == n.steps - 1;
      NsTask task;
      task.op = op;
      task.a = held_in_register(n.coefficients[3 * step]);
      task.b = held_in_register(n.coefficients[3 * step + 1]);
      task.c = held_in_register(n.coefficients[3 * step + 2]);
      tc_wait_long(go, at_op & 1, alive, &g_muon_fault, kMuonFault, kGridWaitClocks);
      if (leader) proxy_fence();
      if (op == kNsJoin) ns_join<CTAS>(n, warp - kFirstResultWarp, lane);
      for (int t = first; t < tiles; t += apart) {
        const NsTile at = ns_tile(n, join, op, t);
        const NsShape& g = n.shape[at.shape];
        const int whole = ns_stages(g, op),
                  each = ns_stage(g, join, op, whole, at.part + 1) - ns_stage(g, join, op, whole, at.part);
        // All runs of a long sum but the last, added up.
        for (int run = kNsRun; run < each; run += kNsRun) {
          tc_wait_long(&summed[s.at], s.phase, alive, &g_muon_fault, kMuonFault, kGridWaitClocks);
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < HALF; c += 32) {
            uint32_t v[32];
            tmem_ld(lanes + s.at * TILE + c, v);
            tmem_ld_wait(v);
            float* to = runs + (c / 4) * kNsSide * 4;
            if (run > kNsRun) add_run(to, v);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4*>(to + i * kNsSide * 4) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if constexpr (CTAS == 2) mbar_arrive_cluster(taken_at + 8 * s.at);
            else mbar_arrive(&taken[s.at]);
          }
          s.next();
        }
        const bool more = each > kNsRun;
        if (join && op == kNsGram && g.split > 1) {  // a part of a tile's sums, as they are
          float* to = n.partial + static_cast<int64_t>(t) * TILE * TILE +
                      (half * (HALF / 4) * TILE + rank * kNsSide + row) * 4;
          tc_wait_long(&summed[s.at], s.phase, alive, &g_muon_fault, kMuonFault, kGridWaitClocks);
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < HALF; c += 32) {
            uint32_t v[32];
            tmem_ld(lanes + s.at * TILE + c, v);
            tmem_ld_wait(v);
            if (more) add_run(runs + (c / 4) * kNsSide * 4, v);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              st_v4(to + (c / 4 + i) * TILE * 4, make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if constexpr (CTAS == 2) mbar_arrive_cluster(taken_at + 8 * s.at);
            else mbar_arrive(&taken[s.at]);
          }
          s.next();
          continue;
        }
        task.wide = held_in_register(g.wide);
        const int side = held_in_register(task.wide ? g.rows : g.cols);
        task.diagonal = at.p == at.q;
        task.diag_out = held_in_register((op == kNsGram ? g.a_diag : g.b_diag) +
                                         static_cast<int64_t>(at.matrix) * g.diag_apart);
        const int rows = op == kNsApply ? held_in_register(g.rows) : side,
                  cols = op == kNsApply ? held_in_register(g.cols) : side;
        const bool turn = op != kNsApply && !task.diagonal;
        const CUtensorMap *turned = op == kNsGram ? &g.a_turned : &g.b_turned,
                          *turned_low = op == kNsGram ? &g.a_turned_low : &g.b_turned_low;
        const int p0 = at.p * TILE + rank * kNsSide, p = p0 + row;
        const CUtensorMap *in, *in_low, *out, *out_low;
        if (op == kNsApply) {
          in = g.wide ? &g.x[from] : &g.xt[from], in_low = g.wide ? &g.x_low[from] : &g.xt_low[from];
          out = g.wide ? &g.x[from ^ 1] : &g.xt[from ^ 1], out_low = g.wide ? &g.x_low[from ^ 1] : &g.xt_low[from ^ 1];
        } else {
          in = &g.a, in_low = &g.a_low;
          out = op == kNsGram ? &g.a : &g.b, out_low = op == kNsGram ? &g.a_low : &g.b_low;
        }
        // A's diagonal by rows and columns; B's by those of X that B is as wide as.
        const bool by_p = op == kNsPoly || (op == kNsApply && task.wide), by_q = op == kNsPoly || (op == kNsApply && !task.wide);
        const float* diag = (op == kNsApply ? g.b_diag : g.a_diag) + static_cast<int64_t>(at.matrix) * g.diag_apart;
        // Chunk k of this half: the copies that are under way from it end, and its inputs are fetched.
        const auto fetch = [&](int k) {
          const int q0 = at.q * TILE + half * HALF + k * kNsChunk;
          if (!leader || !alive || p0 >= rows || q0 >= cols) return;
          tma_store_wait_read();
          if (op == kNsGram) return;
          mbar_arrive_expect_tx(&held[half], 2 * kNsHalfChunk + (by_q ? kNsChunk * 4 : 0));
          tma_load(high, in, q0, p0, at.matrix, &held[half]);
          tma_load(low, in_low, q0, p0, at.matrix, &held[half]);
          if (by_q) bulk_load(diag_q, diag + q0, kNsChunk * 4, &held[half]);
        };
        float diag_p = 0.0f;
        if (by_p && p < rows) diag_p = ld_after_f32(diag + p);
        fetch(0);
        if (last && !skip && p < rows) ns_result_ahead(n, g, at.matrix, p, at.q * TILE + half * HALF, HALF);
        tc_wait_long(&summed[s.at], s.phase, alive, &g_muon_fault, kMuonFault, kGridWaitClocks);
        tc_fence_after();
#pragma unroll 1
        for (int k = 0; k < HALF / kNsChunk; ++k) {
          const int q0 = at.q * TILE + half * HALF + k * kNsChunk;
          const bool inside = p0 < rows && q0 < cols;  // the same for the half's 4 warps
          if (k > 0) fetch(k);
          if (inside && op != kNsGram) {
            tc_wait(&held[half], held_phase, alive, &g_muon_fault, kMuonFault);
            held_phase ^= 1u;
          }
          if (inside && op == kNsGram) named_barrier(2 + half, 128);  // (the chunk is free)
#pragma unroll
          for (int h = 0; h < kNsChunk; h += 32) {
            uint32_t v[32];
            tmem_ld(lanes + s.at * TILE + k * kNsChunk + h, v);
            tmem_ld_wait(v);
            if (k + 1 == HALF / kNsChunk && h + 32 == kNsChunk) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) {
                if constexpr (CTAS == 2) mbar_arrive_cluster(taken_at + 8 * s.at);
                else mbar_arrive(&taken[s.at]);
              }
            }
            if (more) add_run(runs + ((k * kNsChunk + h) / 4) * kNsSide * 4, v);
            if (inside && p < rows) {
              uint4 x[4], y[4];  // (all read before the first is written: they are places of one buffer)
              if (op != kNsGram) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  x[j] = *reinterpret_cast<const uint4*>(ns_place(high, row, h / 8 + j));
                  y[j] = *reinterpret_cast<const uint4*>(ns_place(low, row, h / 8 + j));
                }
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                float d[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) d[i] = __uint_as_float(v[8 * j + i]);
                uint4 w, l;
                if (op != kNsApply) {
                  ns_symmetric(task, p, q0 + h + 8 * j, diag_p, diag_q + h + 8 * j, x[j], y[j], d);
                  two_halves(d, w, l);
                } else {
                  ns_applied(task, diag_p, diag_q + h + 8 * j, x[j], y[j], d);
                  if (last) {
                    uint32_t u[4], f[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                      const uint32_t a = __float_as_uint(__fmul_rn(d[2 * i], 1.0f / kXScale)),
                                     b = __float_as_uint(__fmul_rn(d[2 * i + 1], 1.0f / kXScale));
                      u[i] = __byte_perm(a, b, 0x7632u), f[i] = __byte_perm(a, b, 0x5410u);
                    }
                    w = make_uint4(u[0], u[1], u[2], u[3]), l = make_uint4(f[0], f[1], f[2], f[3]);
                  } else {
                    two_halves(d, w, l);
                  }
                }
                *reinterpret_cast<uint4*>(ns_place(high, row, h / 8 + j)) = w;
                *reinterpret_cast<uint4*>(ns_place(low, row, h / 8 + j)) = l;
              }
            }
          }
          if (!inside) continue;
          if (last) {
            named_barrier(2 + half, 128);
            if (!skip) ns_result(n, g, at.matrix, p0, q0, high, low, warp & 3, lane);
            tma_store_fence();  // (read before the next copy into the chunk)
            named_barrier(2 + half, 128);
          } else {
            tma_store_fence();
            named_barrier(2 + half, 128);
            if (leader) {
              tma_store(out, q0, p0, at.matrix, high);
              tma_store(out_low, q0, p0, at.matrix, low);
              tma_store_commit();
            }
            if (turn) {  // the chunk once more, transposed where it lies: every thread takes its row out first
              if (leader) tma_store_wait_read();
              named_barrier(2 + half, 128);
#pragma unroll
              for (int of = 0; of < 2; ++of) {
                uint8_t* chunk = of == 0 ? high : low;
                uint4 x[kNsChunk / 8];
#pragma unroll
                for (int j = 0; j < kNsChunk / 8; ++j) x[j] = *reinterpret_cast<const uint4*>(ns_place(chunk, row, j));
                named_barrier(2 + half, 128);
#pragma unroll
                for (int j = 0; j < kNsChunk / 8; ++j) ns_turn(chunk, row, 8 * j, x[j]);
              }
              tma_store_fence();
              named_barrier(2 + half, 128);
              if (leader) {
                for (int i = 0; i < 2 && p0 + 64 * i < rows; ++i) {
                  tma_store(turned, p0 + 64 * i, q0, at.matrix, high + i * (kNsHalfChunk / 2));
                  tma_store(turned_low, p0 + 64 * i, q0, at.matrix, low + i * (kNsHalfChunk / 2));
                }
                tma_store_commit();
              }
            }
          }
        }
        s.next();
      }
      if (leader) tma_store_wait();
      named_barrier(1, kResultWarps * 32);
      if (threadIdx.x == kFirstResultWarp * 32) {
        proxy_fence();
        __threadfence();
        asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(n.arrived) : "memory");
      }
    }
  }
  __syncwarp();  // (as do the barrier and the release of tensor memory: the copies were one lane's)
  tc_fence_before();
  if constexpr (CTAS == 2) cluster_sync();
  else __syncthreads();
  if (warp == kCopyWarp) {
    tc_fence_after();
    tmem_free<CTAS>(tmem, TILE * kNsSlots);
  }
}

template <int CTAS, bool join, typename L>
static cudaError_t run_ns(const L& n, cudaStream_t s) {
  auto kern = k_newton_schulz<CTAS, join, L>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kNsCtas);
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
  int tiles = n.tiles[1];
  for (int i = 0; i < 3; ++i) tiles = n.tiles[i] > tiles ? n.tiles[i] : tiles;
  fit = fit < kNsCtas / CTAS ? fit : kNsCtas / CTAS;
  cfg.gridDim = dim3(static_cast<unsigned>((tiles < fit ? tiles : fit) * CTAS));
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, n);
}
template <typename L>
static cudaError_t run_ns(const L& n, int side, cudaStream_t s) {
  if (n.join) return side == 256 ? run_ns<2, true>(n, s) : run_ns<1, true>(n, s);
  return side == 256 ? run_ns<2, false>(n, s) : run_ns<1, false>(n, s);
}
cudaError_t launch_ns(const NsLaunch& n, int side, cudaStream_t s) {
  const NsShape& last = n.shape[n.shapes - 1];
  if (n.shapes > 2 || last.first_matrix + last.count > 32) return run_ns(n, side, s);
  NsLaunchFew few;  // (a launch's parameters are copied by the driver)
  few.steps = n.steps, few.shapes = n.shapes, few.join = n.join, few.partial = n.partial, few.runs = n.runs;
  for (int i = 0; i < 3; ++i) few.tiles[i] = n.tiles[i];
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
