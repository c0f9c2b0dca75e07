// zpp_launch.h -- host-side launchers of the sm_103a kernels (internal to libzpp).
// The C ABI in zpp_abi.cu validates arguments and then calls exactly one of these.
#pragma once

#include <cuda_runtime_api.h>
#include <stdint.h>

namespace zpp {

// K1: block quantisation of n fp16 (is_bf16 = 0) or bf16 values.
cudaError_t launch_quant(const void* x, int is_bf16, int64_t n, int block, int bits,
                         void* codes, float* scales, cudaStream_t s);

// K2: dequantisation into fp16 (out_kind 0), bf16 (1) or fp32 (2).
cudaError_t launch_dequant(const void* codes, const float* scales, int64_t n, int block,
                           int bits, void* y, int out_kind, cudaStream_t s);

// The qgZ launchers cover the hop-1 chunks / receivers with local index l in
// [l_begin, l_end) (the whole exchange is [0, M)).
// K3: slice reorder + block quantisation of `ranks` consecutive ranks of E elements each
// (all W = N*M ranks of the virtual layout, or the one rank of a real device).
cudaError_t launch_reorder_quant(const void* grads, int is_bf16, int64_t E, int block, int bits,
                                 int N, int M, int l_begin, int l_end, int ranks, void* codes,
                                 float* scales, cudaStream_t s);

// K3 over a bucket given as tensors (the flatten fused in; whole exchange only). Tensor t
// holds the W ranks' copies back to back, rank r's at ptr[t] + r * len_t, len_t =
// offs[t+1] - offs[t]; offs[0] = 0, offs[count] = E. Passed by value in the kernel's
// parameter space (about 16 KB), so no device table is needed.
constexpr int kMaxTensors = 1024;  // = ZPP_MAX_TENSORS
struct TensorTable {
  const uint16_t* ptr[kMaxTensors];
  int64_t offs[kMaxTensors + 1];
  int32_t count;
};
cudaError_t launch_reorder_quant_tensors(const TensorTable& tab, int is_bf16, int64_t E, int block,
                                         int bits, int N, int M, void* codes, float* scales,
                                         cudaStream_t s);
// The same per input type (v8: every tensor pointer is 32-byte aligned).
cudaError_t launch_reorder_quant_tensors_f16(const TensorTable& tab, int64_t E, int block,
                                             int bits, int N, int M, bool v8, void* codes,
                                             float* scales, cudaStream_t s);
cudaError_t launch_reorder_quant_tensors_bf16(const TensorTable& tab, int64_t E, int block,
                                              int bits, int N, int M, bool v8, void* codes,
                                              float* scales, cudaStream_t s);

// K4: intra-node fused dequantise -> fp32 sum over M sources -> requantise. Receiver
// (n, l), n < N, reads C elements at offset l*C of sources n*M .. n*M+M-1, which lie E
// elements apart, and writes C codes at receiver offset (n*M + l)*C. The virtual layout
// has C = E / M; one real rank's received chunks are N = 1, l = 0 and E = C.
cudaError_t launch_dequant_reduce_requant(const void* codes, const float* scales, int64_t E,
                                          int64_t C, int block, int bits, int N, int M,
                                          int l_begin, int l_end, void* out_codes,
                                          float* out_scales, cudaStream_t s);

// K5: inter-node dequantise -> fp32 sum over N slices, times post_scale, stored as fp16
// (out_kind 0), bf16 (1) or fp32 (2). Receiver (n, l), n < nz, reads S elements at offset
// n*S of the N hop-1 outputs of ranks (n', l), which are C elements long and M outputs
// apart, and writes S outputs at (n*M + l)*S. The virtual layout has S = E / W, C = E / M,
// nz = N; one real rank's received slices are S = C, M = 1, nz = 1, l = 0.
cudaError_t launch_dequant_reduce(const void* codes, const float* scales, int64_t S, int64_t C,
                                  int block, int bits, int N, int M, int l_begin, int l_end,
                                  int nz, float post_scale, void* out, int out_kind,
                                  cudaStream_t s);

// The device fault word: bits set by kernels whose bounded waits ran out (1: a producer
// wait of the INT8 K4 ring, 2: a consumer wait of that ring, 4: the wait self-test).
// Synchronous: copies the word of the current device to *flags, then zeroes it if clear.
cudaError_t read_device_fault(unsigned* flags, bool clear);

// A kernel that waits, bounded by limit_ns, on a barrier nothing completes (sets bit 4).
cudaError_t launch_wait_selftest(unsigned long long limit_ns, cudaStream_t s);

// K6: 256-bit device copy (the same-run HBM reference).
cudaError_t launch_copy(const void* src, void* dst, int64_t bytes, cudaStream_t s);

// Which tensor of a list a CTA belongs to: the tensors of a launch have first[0] .. first[count]
// CTAs before them, and every 2^shift-th CTA's tensor is written down, so that a CTA searches a
// few entries (from kernel parameters, each step a dependent load) and not all.
struct ChunkHints {
  static constexpr int kBuckets = 64;
  int32_t shift;
  uint16_t at[kBuckets + 1];
  void fill(const int32_t* first, int count) {  // count >= 1
    const int32_t grid = first[count];
    for (shift = 0; (grid - 1) >> shift >= kBuckets;) ++shift;
    int t = 0;
    for (int b = 0; b <= kBuckets; ++b) {
      while (t + 1 < count && first[t + 1] <= static_cast<int64_t>(b) << shift) ++t;
      at[b] = static_cast<uint16_t>(t);
    }
  }
};
#ifdef __CUDACC__
__device__ __forceinline__ int tensor_of(const ChunkHints& hints, const int32_t* first, int cta) {
  int lo = hints.at[cta >> hints.shift], hi = hints.at[(cta >> hints.shift) + 1] + 1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= cta) lo = mid;
    else hi = mid;
  }
  return lo;
}
#endif

// K7: sums of squares over a list of tensors (one partial per CTA into `workspace`), then
// norm and clip factor. The list travels in the kernel's parameter space.
constexpr int kNormChunk = 16384;  // elements per CTA
template <int CAP>
struct NormTableOf {
  const void* ptr[CAP];
  int64_t n[CAP];
  int32_t first[CAP + 1];  // CTAs of the tensors before this one
  int32_t count;
  ChunkHints hints;
};
using NormTable = NormTableOf<kMaxTensors>;
// A launch's parameters are copied by the driver: up to this many tensors travel in a small
// table (a call with one tensor costs the host 3 us less than with the full one).
constexpr int kFewTensors = 16;
inline int64_t norm_chunks(int64_t n) { return (n + kNormChunk - 1) / kNormChunk; }
// What a counted optimiser step keeps on the device (= zpp_adamw_record), and what its factors
// are made of.
struct StepRecord {
  int64_t step, reserved;
  float factor, step_size, inv_root_bc2;
  uint32_t key;
  double beta[2], power[2];
};
struct StepCount {
  double lr, beta[2];
  double power[2];                // known > 0: beta^known, and
  float step_size, inv_root_bc2;  // the factors of that step
  int64_t known;                  // the step's number; 0: one more than the record's
  uint32_t seed;
  StepRecord* record;  // null: nothing is counted
};
// count: the factor `out[1]` is that of an optimiser step, whose record is written.
cudaError_t launch_grad_norm(NormTable& tab, int g_kind, float pre_scale, float max_norm,
                             float* workspace, float* out, const StepCount& count, cudaStream_t s);

// K8: one AdamW step over a list of tensors; at most kAdamwTensors per launch (their
// descriptors travel in the kernel's parameter space).
constexpr int kAdamwTensors = 432;
constexpr int kStateBlock = 256;   // = ZPP_STATE_BLOCK
struct AdamwTensor {
  float* param;
  const void* grad;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  void* weight;
  int64_t n;
};
struct AdamwArgs {
  float beta1, one_minus_beta1, beta2, one_minus_beta2;
  float step_size;      // lr / (1 - beta1^t)
  float inv_root_bc2;   // 1 / sqrt(1 - beta2^t)
  float eps, decay;     // decay = lr * weight_decay
  uint32_t key;         // of the rounding hash
  const float* grad_scale;
  StepRecord* record;      // its factors replace those above (counted), or it is told `step`
  int64_t step;            // > 0 with a record: the step's number, known on the host
  int32_t g_kind, w_kind;  // zpp_dtype of grad and weight
};
template <int CAP>
struct AdamwTableOf {
  AdamwArgs a;
  int64_t first_block;     // state blocks of the tensors of earlier launches
  ChunkHints hints;
  int32_t count;
  int32_t first[CAP + 1];  // chunks of the tensors before this one
  int32_t block0[CAP];     // state blocks of the tensors before this one
  AdamwTensor t[CAP];
};
using AdamwTable = AdamwTableOf<kAdamwTensors>;
// The parameter space is said to hold 32,764 bytes, but a build of k_adamw whose hints lay at its byte
// 32,264 (behind 448 tensors, with fp32 states) stepped the first tensor of every list only; the
// same code with the hints in front steps all. So the table ends before 31 KB, the tensors last.
static_assert(sizeof(AdamwTable) <= 31 * 1024, "kernel parameter space");
constexpr int adamw_warp_blocks(int state_bits) { return state_bits == 8 ? 2 : 1; }
constexpr int adamw_chunk(int state_bits) {  // elements per CTA of 8 warps
  return 8 * adamw_warp_blocks(state_bits) * kStateBlock;
}
inline int64_t adamw_chunks(int64_t n, int state_bits) {
  return (n + adamw_chunk(state_bits) - 1) / adamw_chunk(state_bits);
}
cudaError_t launch_adamw(AdamwTable& tab, int state_bits, cudaStream_t s);
// Writes count.record for a step by the factor *grad_scale (null: 1).
cudaError_t launch_step_count(const StepCount& count, const float* grad_scale, cudaStream_t s);

// K9: y = x W^T (+ bias) from block-quantised codes. x_bf16: x and bias are bf16, else fp16;
// y_kind as a zpp_dtype.
struct MatvecArgs {
  const uint8_t* codes;
  const float* scales;
  int64_t rows, cols;
  int32_t block, bits;
  const uint16_t* x;
  int32_t x_bf16;
  int64_t vecs, x_stride;
  const uint16_t* bias;
  void* y;
  int32_t y_kind;
  int64_t y_stride;
};
cudaError_t launch_matvec(const MatvecArgs& a, cudaStream_t s);

// K10: y = a b^T (+ bias) of e4m3 matrices with a scale per block of 128 along the sum.
struct MatmulOperand {
  const uint8_t* codes;
  int64_t rows, stride;  // stride in bytes
  const float* scales;
  int64_t scale_row, scale_block;
  int32_t tile;          // rows that share a scale: 1 or 128
};
struct MatmulArgs {
  MatmulOperand a, b;
  int64_t depth;  // of the sum
  const void* bias;
  void* y;
  int32_t y_kind;  // zpp_dtype of y and bias
  int64_t y_stride;
};
cudaError_t launch_matmul_fp8(const MatmulArgs& a, cudaStream_t s);
cudaError_t read_matmul_fault(unsigned* flags, bool clear);

// K11: e4m3 codes and power-of-two scales of a matrix, and of its transpose (codes_t null: not).
struct QuantFp8Args {
  const void* x;
  int32_t x_kind;
  int64_t rows, cols, x_stride;
  int32_t tile;
  uint8_t* codes;
  int64_t codes_stride;
  float* scales;
  int64_t scale_row, scale_block;
  uint8_t* codes_t;
  int64_t codes_t_stride;
  float* scales_t;  // tile 1 only
  int64_t scale_t_row, scale_t_block;
};
cudaError_t launch_quant_fp8(const QuantFp8Args& a, cudaStream_t s);

// K12 .. K14: Newton-Schulz products over a list of matrices, with the Muon step around them.
constexpr int kMuonMatrices = 256;  // of a batch
constexpr int kMuonGroups = 12;     // shapes of a batch
struct MuonMatrix {
  const void* x;     // the gradient, or the matrix itself
  float* momentum;   // null: x itself is what becomes orthogonal
  float* param;      // Muon: updated; else null
  void* out;         // the result in 16 bits, or the updated parameter in 16 bits (may be null)
  int64_t rows, cols;
};
struct MuonArgs {
  float mu, one_minus_mu;
  bool nesterov;
  float decay;           // 1 - lr * weight_decay
  double lr;
  int32_t adjust;        // 0: sqrt(max(1, rows / cols)), 1: 0.2 sqrt(max(rows, cols)), 2: 1
  float eps;
  int32_t steps;
  const double* coefficients;  // [steps][3], HOST
  int32_t x_kind, out_kind;
  const float* factor;   // device, or null
};
// Bytes of workspace; the list is taken in batches, one after the other.
int64_t muon_workspace(const MuonMatrix* list, int count);
cudaError_t launch_muon(const MuonMatrix* list, int count, const MuonArgs& a, uint8_t* workspace,
                        cudaStream_t s);
cudaError_t read_muon_fault(unsigned* flags, bool clear);

// Grid size when every CTA owns `per_cta` consecutive tiles and exits (no grid-stride
// loop): on GB300 a streaming kernel launched this way sustains more HBM bandwidth than
// a persistent grid sized to the SM count.
inline int tile_grid(int64_t tiles, int per_cta) {
  int64_t g = (tiles + per_cta - 1) / per_cta;
  return static_cast<int>(g > 0 ? g : 1);
}

}  // namespace zpp
