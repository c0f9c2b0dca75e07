// muon.cu -- K12, K13 and the order of a Muon step:
//
//   m = mu m + (1 - mu) c g,  u = (1 - mu) c g + mu m (nesterov) or m,  X = u / max(|u|_F, eps)   (K12, K13)
//   the steps of K14, after the last one  p = p (1 - lr decay) - lr adjust X
//
// K12 reads the gradient and the momentum, writes the momentum and one partial sum of squares per
// CTA; K13 adds a matrix's partials in a fixed order, makes u again and writes X as two fp16. Both are bound by
// DRAM (10 bytes an element each with 16-bit gradients; 50 M elements 89 and 93 us, 5.6 TB/s); for small
// lists by their launches.
#include <algorithm>
#include <cmath>
#include <limits>
#include <vector>

#include "newton_schulz.cuh"
#include "zpp_overlap.cuh"
#include "zpp_tensor_map.h"

namespace zpp {

constexpr int kMuonPer = kThreads * 8;    // elements of a CTA's round
constexpr int kMuonPartials = 1024;       // of a matrix, at most
// Squares of what is below 2^-63 leave fp32's range, and an eps may be as small as 2^-126: a second sum takes values times
// 2^76, and counts where the first one is below 2^-60 (then none is above 2^-30, so the second one is finite; and
// above that, what the first one lost is some 2^-150 a value).
constexpr float kSmallScale = 75557863725914323419136.0f;  // 2^76
constexpr float kSmallBelow = 1.0f / 1152921504606846976.0f;  // 2^-60

struct MuonTable {
  int32_t count;
  bool nesterov;
  float mu, one_minus_mu, eps;
  int32_t x_kind;
  const float* factor;
  double* partial;
  uint32_t* arrived;  // K14's count, zeroed by K13
  ChunkHints hints;
  int32_t first[kMuonMatrices + 1];  // CTAs of the matrices before this one
  struct Item {
    const void* x;
    float* momentum;
    uint16_t *high, *low;
    int64_t n, per;       // elements, and those of a CTA (whole rounds)
    int32_t cols, ld;
  } item[kMuonMatrices];
};
static_assert(sizeof(MuonTable) <= 31 * 1024, "kernel parameter space");

// Elements i .. i + 7 of n, zeros behind the last. vec: x is 16-byte aligned.
template <int KIND>
__device__ __forceinline__ void load8(const void* x, int64_t i, int64_t n, bool vec, float (&v)[8]) {
  if (vec && i + 8 <= n) {
    const char* p = static_cast<const char*>(x) + i * (KIND == 2 ? 4 : 2);
#pragma unroll
    for (int h = 0; h < (KIND == 2 ? 2 : 1); ++h) {
      const uint4 w = ld_after_v4(p + 16 * h);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (KIND == 2) {
          v[4 * h + k] = __uint_as_float(u[k]);
        } else {
          const float2 f = KIND == 0 ? unpack2(u[k], F16()) : unpack2(u[k], BF16());
          v[2 * k] = f.x, v[2 * k + 1] = f.y;
        }
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[k] = 0.0f;
      if (i + k < n) {
        if constexpr (KIND == 2) v[k] = static_cast<const float*>(x)[i + k];
        else v[k] = KIND == 0 ? bits16_to_float(static_cast<const uint16_t*>(x)[i + k], F16())
                              : bits16_to_float(static_cast<const uint16_t*>(x)[i + k], BF16());
      }
    }
  }
}

// Brings what the CTA reads two rounds later into L2 (a line of 128 bytes by its first thread).
template <int KIND>
__device__ __forceinline__ void ahead(const void* x, int64_t i, int64_t n) {
  constexpr int SIZE = KIND == 2 ? 4 : 2;
  const int64_t to = i + 2 * kMuonPer;
  if ((threadIdx.x & (128 / (8 * SIZE) - 1)) == 0 && to < n)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(x) + to * SIZE));
}

__device__ __forceinline__ double cta_sum(double v, double* part) {  // valid in every thread
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
  for (int w = 0; w < kWarps; ++w) v += part[w];
  return v;
}

// K12 (SCALE false) and K13.
template <int KIND, bool SCALE>
__global__ void __launch_bounds__(kThreads) k_muon(const __grid_constant__ MuonTable t) {
  __shared__ double part[kWarps];
  grid_wait();
  grid_release();
  if (SCALE && blockIdx.x == 0 && threadIdx.x == 0) *t.arrived = 0u;
  const float factor = t.factor ? ld_after_f32(t.factor) : 1.0f;
  if (!isfinite(factor)) return;
  const int m = tensor_of(t.hints, t.first, static_cast<int>(blockIdx.x));
  const MuonTable::Item& it = t.item[m];
  const int cta = static_cast<int>(blockIdx.x) - t.first[m];
  const int64_t begin = cta * it.per, end = begin + it.per < it.n ? begin + it.per : it.n;
  float inv = 0.0f;
  if constexpr (SCALE) {
    double total = 0.0;
    for (int i = t.first[m] + static_cast<int>(threadIdx.x); i < t.first[m + 1]; i += kThreads)
      total += ld_after_f64(t.partial + i);
    total = cta_sum(total, part);
    const float norm = static_cast<float>(sqrt(total));
    // (a norm that is not a number passes through, and so does one that is infinite, as NaN)
    inv = norm <= 3.402823466e38f ? __fdiv_rn(1.0f, fmaxf(norm, t.eps)) : __int_as_float(0x7fc00000);
  }
  const bool x_vec = (reinterpret_cast<uintptr_t>(it.x) & 15) == 0;
  const bool m_vec = (reinterpret_cast<uintptr_t>(it.momentum) & 15) == 0;
  float sum = 0.0f, small = 0.0f;
#pragma unroll 2
  for (int64_t i = begin + threadIdx.x * 8; i < end; i += kMuonPer) {
    float x[8], u[8];
    load8<KIND>(it.x, i, it.n, x_vec, x);
    ahead<KIND>(it.x, i, it.n);
    if (it.momentum) {
      float mo[8];
      load8<2>(it.momentum, i, it.n, m_vec, mo);
      ahead<2>(it.momentum, i, it.n);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float g = __fmul_rn(t.one_minus_mu, __fmul_rn(x[k], factor));
        if constexpr (!SCALE) mo[k] = __fmaf_rn(t.mu, mo[k], g);
        u[k] = t.nesterov ? __fmaf_rn(t.mu, mo[k], g) : mo[k];
      }
      if constexpr (!SCALE) {
        if (m_vec && i + 8 <= it.n) {
          st_v4(it.momentum + i, make_uint4(__float_as_uint(mo[0]), __float_as_uint(mo[1]), __float_as_uint(mo[2]),
                                            __float_as_uint(mo[3])));
          st_v4(it.momentum + i + 4, make_uint4(__float_as_uint(mo[4]), __float_as_uint(mo[5]),
                                                __float_as_uint(mo[6]), __float_as_uint(mo[7])));
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (i + k < it.n) it.momentum[i + k] = mo[k];
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] = x[k];
    }
    if constexpr (!SCALE) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float up = __fmul_rn(u[k], kSmallScale);
        sum = __fmaf_rn(u[k], u[k], sum);
        small = __fmaf_rn(up, up, small);
      }
    } else {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = __fmul_rn(__fmul_rn(u[2 * k], inv), kXScale),
                    b = __fmul_rn(__fmul_rn(u[2 * k + 1], inv), kXScale);
        hi[k] = pack2(a, b, F16());
        const float2 f = unpack2(hi[k], F16());
        lo[k] = pack2(__fsub_rn(a, f.x), __fsub_rn(b, f.y), F16());
      }
      if (it.cols == it.ld) {  // the rows lie as the matrix's: n is a multiple of 8
        st_v4(it.high + i, make_uint4(hi[0], hi[1], hi[2], hi[3]));
        st_v4(it.low + i, make_uint4(lo[0], lo[1], lo[2], lo[3]));
      } else {
        int64_t row = i / it.cols;
        int col = static_cast<int>(i - row * it.cols);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (i + k < it.n) {
            it.high[row * it.ld + col] = static_cast<uint16_t>(hi[k >> 1] >> (16 * (k & 1)));
            it.low[row * it.ld + col] = static_cast<uint16_t>(lo[k >> 1] >> (16 * (k & 1)));
          }
          if (++col == it.cols) col = 0, ++row;
        }
      }
    }
  }
  if constexpr (!SCALE) {
    constexpr double back = 1.0 / (static_cast<double>(kSmallScale) * static_cast<double>(kSmallScale));
    const double all = cta_sum(sum < kSmallBelow ? static_cast<double>(small) * back : static_cast<double>(sum), part);
    if (threadIdx.x == 0) t.partial[blockIdx.x] = all;
  }
}

// ------------------------------------------------------------------------------------- the host's part
namespace {

struct Shape {
  int64_t rows, cols;
  int count = 0, first = 0;
  int64_t small() const { return std::min(rows, cols); }
  int64_t ld() const { return (cols + 15) / 16 * 16; }
  int64_t small_ld() const { return (small() + 15) / 16 * 16; }
  int64_t x_elems() const { return (rows * ld() + 63) / 64 * 64; }  // one matrix, 128-byte aligned
  int64_t a_elems() const { return (small() * small_ld() + 63) / 64 * 64; }
  int64_t diag_elems() const { return (small() + 63) / 64 * 64; }  // fp32
  bool wide() const { return rows <= cols; }
  // X twice, A and B, each in two fp16, and the diagonals
  int64_t bytes() const { return count * (4 * x_elems() * 2 + 4 * a_elems() * 2 + 2 * diag_elems() * 4); }
};

// Matrices that are worked on together, in the order of their shapes.
struct Batch {
  std::vector<Shape> shapes;
  std::vector<int> order;  // places in the list
  int64_t elems = 0;
};
// How K14 takes a batch: the side of its tiles, 256 by a pair of CTAs, or 128, which share themselves out more
// evenly; and into how many parts a gram's sum is split where its tiles leave most CTAs without work (worth
// the pass that joins them, 5 us, from 48 stages on: 100 x 6000 in five steps 460 us without).
// A stage takes either side about as long (0.3 us): counted are those of the slowest CTA.
struct Plan {
  int side = 128, share = 1;
  int64_t parts = 0;  // of tiles, in the gram
  bool join = false;
  bool runs = false;  // some sum takes more than one
};
int64_t stages_of(int64_t depth) { return kNsProducts * ((depth + 63) / 64); }
int64_t split_of(const Shape& s, const Plan& p) {
  return std::max<int64_t>(1, std::min<int64_t>(p.share, stages_of(std::max(s.rows, s.cols)) / 8));
}
Plan plan_of(const Batch& b) {
  Plan best;
  double least = 0.0;
  for (int pair = 0; pair < 2; ++pair) {
    Plan p;
    p.side = pair ? 256 : 128;
    const int64_t at_once = pair ? 76 : 152;
    double tiles[3] = {}, work[3] = {}, longest[3] = {};
    int64_t symmetric = 0, stages = 0;
    for (const Shape& s : b.shapes) {
      const int64_t small = s.small(), large = std::max(s.rows, s.cols);
      const int64_t m = (small + p.side - 1) / p.side, n = (large + p.side - 1) / p.side;
      for (int op = 0; op < 3; ++op) {
        const double t = static_cast<double>(s.count * (op == kNsApply ? m * n : m * (m + 1) / 2));
        const double depth = static_cast<double>(stages_of(op == kNsGram ? large : small));
        tiles[op] += t;
        work[op] += t * depth;
        longest[op] = std::max(longest[op], depth);
      }
      symmetric += s.count * (m * (m + 1) / 2);
      stages = std::max(stages, stages_of(large));
    }
    p.runs = stages > kNsProducts * kNsRun;
    if (2 * symmetric <= at_once && stages >= 48)
      p.share = static_cast<int>(std::min<int64_t>({at_once / symmetric, stages / 8, 16}));
    for (const Shape& s : b.shapes) {
      const int64_t m = (s.small() + p.side - 1) / p.side, split = split_of(s, p);
      p.parts += s.count * (m * (m + 1) / 2) * split;
      p.join |= split > 1;
    }
    double cost = 0.0;
    for (int op = 0; op < 3; ++op) {
      const double split = op == kNsGram ? p.share : 1;
      const double rounds = std::ceil(split * tiles[op] / static_cast<double>(at_once));
      cost += std::max(longest[op] / split, work[op] / split / tiles[op] * rounds);
    }
    if (p.join) cost += 16.0;
    if (pair == 0 || cost < least) best = p, least = cost;
  }
  return best;
}

int64_t bytes_of(const Batch& b) {
  int64_t n = 128;  // (the first ones count CTAs)
  for (const Shape& s : b.shapes) n += s.bytes();
  const Plan p = plan_of(b);
  if (p.join) n += p.parts * p.side * p.side * 4;
  if (p.runs) n += ns_run_floats(p.side) * 4;
  return n + static_cast<int64_t>(b.order.size()) * kMuonPartials * 8;
}
constexpr int64_t kBatchElems = int64_t{1} << 28;  // more than this starts another batch

// Calls each(batch) for the list's batches.
template <typename F>
auto batches(const MuonMatrix* list, int count, const F& each) {
  std::vector<std::vector<int>> of;
  Batch b;
  const auto flush = [&] {
    for (size_t k = 0; k < b.shapes.size(); ++k) {
      b.shapes[k].first = static_cast<int>(b.order.size());
      b.order.insert(b.order.end(), of[k].begin(), of[k].end());
    }
    const auto r = each(b);
    b = Batch{};
    of.clear();
    return r;
  };
  int held = 0;
  for (int i = 0; i < count; ++i) {
    const MuonMatrix& m = list[i];
    const int64_t n = m.rows * m.cols;
    if (n == 0) continue;
    size_t k = 0;
    while (k < b.shapes.size() && (b.shapes[k].rows != m.rows || b.shapes[k].cols != m.cols)) ++k;
    if (held == kMuonMatrices || (held > 0 && b.elems + n > kBatchElems) ||
        (k == b.shapes.size() && k == kMuonGroups)) {
      if (const auto r = flush(); r) return r;
      held = 0;
      k = 0;
    }
    if (k == b.shapes.size()) {
      Shape s;
      s.rows = m.rows, s.cols = m.cols;
      b.shapes.push_back(s);
      of.emplace_back();
    }
    ++b.shapes[k].count;
    of[k].push_back(i);
    b.elems += n;
    ++held;
  }
  return held ? flush() : decltype(each(b))(0);
}

float adjusted(const MuonArgs& a, int64_t rows, int64_t cols) {
  const double r = static_cast<double>(rows), c = static_cast<double>(cols);
  const double f = a.adjust == 0 ? std::sqrt(std::max(1.0, r / c)) : a.adjust == 1 ? 0.2 * std::sqrt(std::max(r, c)) : 1.0;
  return static_cast<float>(a.lr * f);
}

cudaError_t run_batch(const MuonMatrix* list, const Batch& b, const MuonArgs& a, uint8_t* workspace,
                      cudaStream_t s) {
  // ---- where things lie
  struct Place {
    uint16_t *x[2], *x_low[2], *a, *a_low, *b, *b_low;
    float *a_diag, *b_diag;
  };
  std::vector<Place> place(b.shapes.size());
  uint8_t* at = workspace + 128;  // (the first bytes count CTAs)
  for (size_t k = 0; k < b.shapes.size(); ++k) {
    const Shape& sh = b.shapes[k];
    const auto take = [&](int64_t elems, int size) {
      uint8_t* p = at;
      at += sh.count * elems * size;
      return p;
    };
    const auto half = [&](int64_t elems) { return reinterpret_cast<uint16_t*>(take(elems, 2)); };
    Place& p = place[k];
    for (int i = 0; i < 2; ++i) {
      p.x[i] = half(sh.x_elems());
      p.x_low[i] = half(sh.x_elems());
    }
    p.a = half(sh.a_elems());
    p.b = half(sh.a_elems());
    p.a_low = half(sh.a_elems());
    p.b_low = half(sh.a_elems());
    p.a_diag = reinterpret_cast<float*>(take(sh.diag_elems(), 4));
    p.b_diag = reinterpret_cast<float*>(take(sh.diag_elems(), 4));
  }
  // ---- K12, K13
  MuonTable t{};
  t.count = static_cast<int32_t>(b.order.size());
  t.nesterov = a.nesterov;
  t.mu = a.mu;
  t.one_minus_mu = a.one_minus_mu;
  t.eps = std::max(a.eps, std::numeric_limits<float>::min());
  t.x_kind = a.x_kind;
  t.factor = a.factor;
  t.partial = reinterpret_cast<double*>(at);
  at += static_cast<int64_t>(b.order.size()) * kMuonPartials * 8;
  float* parts = reinterpret_cast<float*>(at);  // of K14's split sums
  t.arrived = reinterpret_cast<uint32_t*>(workspace);
  t.first[0] = 0;
  // Rounds of a CTA: as few as 8 CTAs an SM leave (each adds up its matrix's partials in K13).
  const int64_t enough = std::max<int64_t>(1, b.elems / (int64_t{152} * 8 * kMuonPer));
  for (size_t k = 0, i = 0; k < b.shapes.size(); ++k) {
    const Shape& sh = b.shapes[k];
    for (int j = 0; j < sh.count; ++j, ++i) {
      const MuonMatrix& m = list[b.order[i]];
      MuonTable::Item& it = t.item[i];
      it.x = m.x;
      it.momentum = m.momentum;
      it.high = place[k].x[0] + j * sh.x_elems();
      it.low = place[k].x_low[0] + j * sh.x_elems();
      it.n = sh.rows * sh.cols;
      it.cols = static_cast<int32_t>(sh.cols);
      it.ld = static_cast<int32_t>(sh.ld());
      const int64_t rounds = (it.n + kMuonPer - 1) / kMuonPer;
      const int64_t each = std::max((rounds + kMuonPartials - 1) / kMuonPartials, enough);
      it.per = each * kMuonPer;
      t.first[i + 1] = t.first[i] + static_cast<int32_t>((rounds + each - 1) / each);
    }
  }
  t.hints.fill(t.first, t.count);
  const int grid = t.first[t.count];
  const auto prepare = [&](auto first, auto second) {
    const cudaError_t e = launch_overlapped(first, grid, kThreads, s, t);
    return e != cudaSuccess ? e : launch_overlapped(second, grid, kThreads, s, t);
  };
  cudaError_t e = a.x_kind == 2   ? prepare(k_muon<2, false>, k_muon<2, true>)
                  : a.x_kind == 1 ? prepare(k_muon<1, false>, k_muon<1, true>)
                                  : prepare(k_muon<0, false>, k_muon<0, true>);
  if (e != cudaSuccess) return e;

  // ---- K14
  NsLaunch n{};
  const Plan plan = plan_of(b);
  const int side = plan.side;
  n.join = plan.join;
  n.steps = a.steps;
  n.shapes = static_cast<int32_t>(b.shapes.size());
  n.out_kind = a.out_kind;
  n.decay = a.decay;
  n.factor = a.factor;
  n.arrived = t.arrived;
  n.partial = parts;
  n.runs = parts + (plan.join ? plan.parts * side * side : 0);
  for (int i = 0; i < 3 * a.steps; ++i) n.coefficients[i] = static_cast<float>(a.coefficients[i]);
  for (size_t i = 0; i < b.order.size(); ++i) n.result[i] = NsResult{list[b.order[i]].param, list[b.order[i]].out};
  for (size_t k = 0; k < b.shapes.size(); ++k) {
    const Shape& sh = b.shapes[k];
    const Place& pl = place[k];
    NsShape& g = n.shape[k];
    g.rows = static_cast<int32_t>(sh.rows), g.cols = static_cast<int32_t>(sh.cols);
    g.diag_apart = static_cast<int32_t>(sh.diag_elems());
    g.wide = sh.wide();
    g.count = sh.count, g.first_matrix = sh.first;
    g.side_tiles = static_cast<int32_t>((sh.small() + side - 1) / side);
    g.row_tiles = static_cast<int32_t>((sh.rows + side - 1) / side);
    g.col_tiles = static_cast<int32_t>((sh.cols + side - 1) / side);
    g.split = static_cast<int32_t>(split_of(sh, plan));
    g.a_at = pl.a, g.a_low_at = pl.a_low, g.a_ld = static_cast<int32_t>(sh.small_ld()), g.a_apart = sh.a_elems();
    for (int i = 0; i < 3; ++i) g.first_tile[i] = n.tiles[i];
    n.tiles[2] += sh.count * g.side_tiles * (g.side_tiles + 1) / 2 * g.split;
    n.tiles[0] += sh.count * g.side_tiles * (g.side_tiles + 1) / 2;
    n.tiles[1] += sh.count * g.row_tiles * g.col_tiles;
    g.step = adjusted(a, sh.rows, sh.cols);
    g.a_diag = pl.a_diag, g.b_diag = pl.b_diag;
    const auto map = [&](const uint16_t* p, bool of_x, bool mn, CUtensorMap* to) {
      if (e == cudaSuccess)
        e = make_tensor_map(to, p, 2, of_x ? sh.cols : sh.small(), of_x ? sh.rows : sh.small(),
                            (of_x ? sh.ld() : sh.small_ld()) * 2, sh.count,
                            (of_x ? sh.x_elems() : sh.a_elems()) * 2, mn ? 64 : 128);
    };
    for (int i = 0; i < 2; ++i) {
      map(pl.x[i], true, !sh.wide(), &g.x[i]);
      map(pl.x[i], true, sh.wide(), &g.xt[i]);
      map(pl.x_low[i], true, !sh.wide(), &g.x_low[i]);
      map(pl.x_low[i], true, sh.wide(), &g.xt_low[i]);
    }
    map(pl.a, false, false, &g.a);
    map(pl.b, false, false, &g.b);
    map(pl.a, false, true, &g.a_turned);
    map(pl.b, false, true, &g.b_turned);
    map(pl.a_low, false, false, &g.a_low);
    map(pl.b_low, false, false, &g.b_low);
    map(pl.a_low, false, true, &g.a_turned_low);
    map(pl.b_low, false, true, &g.b_turned_low);
  }
  return e != cudaSuccess ? e : launch_ns(n, side, s);
}

}  // namespace

int64_t muon_workspace(const MuonMatrix* list, int count) {
  int64_t most = 0;
  batches(list, count, [&](const Batch& b) {
    most = std::max(most, bytes_of(b));
    return 0;
  });
  return most;
}

cudaError_t launch_muon(const MuonMatrix* list, int count, const MuonArgs& a, uint8_t* workspace,
                        cudaStream_t s) {
  return batches(list, count, [&](const Batch& b) { return run_batch(list, b, a, workspace, s); });
}

}  // namespace zpp
