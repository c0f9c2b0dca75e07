// newton_schulz.cuh -- the products of K14: what a launch is told (internal to the Muon step).
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "zpp_launch.h"

namespace zpp {

// X is held times 2^10, so that fp16 keeps its 11 bits down to elements of 2^-24; what rounding it
// to fp16 lost is held in a second fp16.
constexpr float kXScale = 1024.0f;
// Matrices whose smaller side is at most this are worked on with products of both fp16.
constexpr int kNsExactSide = 128;

enum NsOp : int32_t {
  kNsGram = 0,   // A = X X^T (or X^T X): the smaller of the two, symmetric
  kNsPoly = 1,   // B = b A + c A A, symmetric
  kNsApply = 2,  // X = a X + B X (or X B)
  kNsLast = 3,   // the same, written as the result
};

// The matrices of one shape in a launch: D[rows][cols] = P Q^T, the sum over `depth`. parts 3: P and Q
// are sums of two fp16, and D = P Q^T + P Qlow^T + Plow Q^T.
struct NsGroup {
  CUtensorMap p, q, p_low, q_low;
  int32_t parts;
  int32_t p_mn, q_mn;        // the operand's rows are steps of the sum
  int32_t rows, cols, depth;
  int32_t p_tiles, q_tiles;  // symmetric: q_tiles == p_tiles, tiles on and above the diagonal
  int32_t per_matrix;        // tiles of one matrix
  int32_t first_tile;        // of the group in the launch
  int32_t first_matrix;      // of the group in the batch
  int32_t ld;                // of in, low and out (elements)
  int64_t apart;             // elements between matrices of in, low and out
  const uint16_t *in, *in_low;  // A (poly) or X (apply), fp16 and what that lost (or null)
  uint16_t *out, *out_low;
  const float* diag_in;      // of A (poly), B (apply); the fp16 matrices hold zeros there
  float* diag_out;
  int32_t diag_apart;        // between matrices
  float step;                // last, Muon: the learning rate of the shape
};
struct NsResult {  // last: where a matrix's result goes
  float* param;
  void* out;
};
struct NsLaunch {
  int32_t op, groups, tiles;
  int32_t side;  // of a tile: 128, or 256 by a pair of CTAs
  float a, b, c;
  int32_t early;  // apply: three steps or more follow
  float decay;
  int32_t out_kind;
  const float* factor;
  NsResult result[kMuonMatrices];
  NsGroup group[kMuonGroups];
};
static_assert(sizeof(NsLaunch) <= 31 * 1024, "kernel parameter space");

cudaError_t launch_ns(const NsLaunch& n, cudaStream_t s);

}  // namespace zpp
