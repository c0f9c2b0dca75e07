// newton_schulz.cuh -- K14: what its launch is told (internal to the Muon step).
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "zpp_launch.h"

namespace zpp {

// X is held times 2^10, so that fp16 keeps its 11 bits down to elements of 2^-24; what rounding it
// to fp16 lost is held in a second fp16.
constexpr float kXScale = 1024.0f;

constexpr int kNsProducts = 3;  // of two factors in two fp16 each: all but that of what both lost
// Stages of the product of first parts that the matrix unit adds up in a row, at most. It cuts the running sum to
// fp32 in each of a stage's four steps, by up to 2^-23 of it, and a gram's diagonal, a sum of squares, falls short by
// as much; the steps multiply that by ten. So the sums of several runs are added by the warps that take them, in the
// workspace, rounded to nearest. (4096 x 16384, normal values, against 64 bits: 9.9e-6 of the result and 9.2 ms, fp32
// products leave 9.1e-6; 1e-4 and 8.8 ms in one run; runs of 16 7.4e-6 and 9.5 ms, of 64 1.7e-5 and 8.85.) The products
// with second parts are small and go with the first run.
constexpr int kNsRun = 32;
constexpr int kNsCtas = 152;  // at most
constexpr int64_t ns_run_floats(int side) { return int64_t{kNsCtas} * 128 * side; }  // of all CTAs' tiles

// The products of a step, in their order.
enum NsOp : int32_t {
  kNsGram = 0,   // A = X X^T (or X^T X): the smaller of the two, symmetric
  kNsPoly = 1,   // B = b A + c A A, symmetric
  kNsApply = 2,  // X = a X + B X (or X B); of the last step the result
  kNsJoin = 3,   // after a gram whose sums were split: the parts added up
};
constexpr int kNsMaxSteps = 100;

// The matrices of one shape. Matrices of fp16 come in pairs: the nearest values and (`low`) what those lost.
struct NsShape {
  CUtensorMap x[2], x_low[2];    // X as the gram reads it: rows along the sum if wide, else across it
  CUtensorMap xt[2], xt_low[2];  // X as the apply reads it: the other way round
  CUtensorMap a, a_low, b, b_low;
  CUtensorMap a_turned, a_turned_low, b_turned, b_turned_low;  // for a tile's transposed place: boxes of 64 rows
  uint16_t *a_at, *a_low_at;     // as a_ld and a_apart: for the join
  float *a_diag, *b_diag;        // fp32; the fp16 matrices hold zeros there
  int32_t rows, cols, diag_apart;
  int32_t wide;                  // rows <= cols
  int32_t count, first_matrix;   // in the batch
  int32_t side_tiles;            // of A's side
  int32_t row_tiles, col_tiles;  // of X
  int32_t split;                 // parts of a gram's sum
  int32_t a_ld;
  int64_t a_apart;
  int32_t first_tile[3];         // of the shape: in the poly, in the apply, and parts of tiles in the gram
  float step;                    // Muon: the learning rate of the shape
};
struct NsResult {  // where a matrix's result goes
  float* param;
  void* out;
};
// A launch: all steps of a batch, the GPU's CTAs waiting for each other between two products.
template <int SHAPES, int MATRICES>
struct NsLaunchOf {
  int32_t steps, shapes, tiles[3];  // of the poly, of the apply, and parts of tiles of the gram
  int32_t join;                     // some shape's sums are split
  float* partial;                   // [parts of tiles][columns / 4][rows][4], where they are
  float* runs;                      // ns_run_floats(), where a sum takes more than one run
  int32_t out_kind;
  float decay;
  const float* factor;
  uint32_t* arrived;                // zero before: CTAs that have ended a product
  float coefficients[3 * kNsMaxSteps];
  NsResult result[MATRICES];
  NsShape shape[SHAPES];
};
using NsLaunch = NsLaunchOf<kMuonGroups, kMuonMatrices>;
using NsLaunchFew = NsLaunchOf<2, 32>;
static_assert(sizeof(NsLaunch) <= 31 * 1024, "kernel parameter space");

// side: of a tile, 128 or 256 (by a pair of CTAs).
cudaError_t launch_ns(const NsLaunch& n, int side, cudaStream_t s);

}  // namespace zpp
