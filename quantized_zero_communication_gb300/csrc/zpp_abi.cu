// zpp_abi.cu -- the extern "C" boundary of libzpp: argument checks (before any launch),
// kernel selection, status codes, and the same-run 256-bit copy kernel.
#include <zpp.h>

#include <algorithm>
#include <cmath>
#include <cstddef>
#include <limits>

#include "zpp_device.cuh"
#include "zpp_launch.h"

namespace zpp {

// K6: streaming copy. Each CTA copies 4 x 256 consecutive 32-byte vectors (all loads
// in flight before the stores) and exits.
__global__ void __launch_bounds__(kThreads) k_copy(const U8x32* __restrict__ src,
                                                   U8x32* __restrict__ dst, int64_t nvec) {
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kThreads * 4 + threadIdx.x;
  U8x32 r[4];
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (base + u * kThreads < nvec) r[u] = ld_stream_v8(src + base + u * kThreads);
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (base + u * kThreads < nvec) st_v8(dst + base + u * kThreads, r[u]);
}

cudaError_t launch_copy(const void* src, void* dst, int64_t bytes, cudaStream_t s) {
  const int64_t nvec = bytes / 32;
  const int grid = tile_grid(nvec, kThreads * 4);
  k_copy<<<grid, kThreads, 0, s>>>(static_cast<const U8x32*>(src), static_cast<U8x32*>(dst), nvec);
  return cudaGetLastError();
}

}  // namespace zpp

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool valid_block(int32_t block) {
  return block >= ZPP_MIN_BLOCK && block <= ZPP_MAX_BLOCK && (block & (block - 1)) == 0;
}

bool valid_bits(int32_t bits) { return bits == 4 || bits == 8; }

zpp_status from_cuda(cudaError_t e) { return e == cudaSuccess ? ZPP_OK : ZPP_ERR_CUDA; }

// Shared checks of the three qgZ entry points; on success W is set.
zpp_status check_topology(int64_t E, int32_t block, int32_t bits, zpp_topology t, int64_t* W) {
  if (!valid_bits(bits) || !valid_block(block)) return ZPP_ERR_INVALID_ARG;
  if (t.num_nodes < 1 || t.gpus_per_node < 1) return ZPP_ERR_INVALID_ARG;
  const int64_t w = static_cast<int64_t>(t.num_nodes) * t.gpus_per_node;
  if (w > 65535) return ZPP_ERR_INVALID_ARG;  // ranks index grid dimensions
  if (E < 0 || E >= (int64_t{1} << 31)) return ZPP_ERR_INVALID_ARG;
  if (E % (w * block) != 0) return ZPP_ERR_INVALID_ARG;
  if (w * E > ZPP_MAX_ELEMS) return ZPP_ERR_INVALID_ARG;
  *W = w;
  return ZPP_OK;
}

bool valid_range(zpp_local_range r, zpp_topology t) {
  return r.begin >= 0 && r.begin <= r.end && r.end <= t.gpus_per_node;
}

zpp_local_range full_range(zpp_topology t) { return zpp_local_range{0, t.gpus_per_node}; }

}  // namespace

extern "C" {

int64_t zpp_code_bytes(int64_t n, int32_t bits) {
  if (n < 0 || !valid_bits(bits)) return -1;
  return bits == 8 ? n : (n + 1) / 2;
}

int64_t zpp_num_scales(int64_t n, int32_t block) {
  if (n < 0 || block <= 0) return -1;
  return (n + block - 1) / block;
}

const char* zpp_status_string(zpp_status s) {
  switch (s) {
    case ZPP_OK: return "ZPP_OK";
    case ZPP_ERR_INVALID_ARG: return "ZPP_ERR_INVALID_ARG: invalid argument";
    case ZPP_ERR_MISALIGNED: return "ZPP_ERR_MISALIGNED: pointer alignment rule broken";
    case ZPP_ERR_UNSUPPORTED: return "ZPP_ERR_UNSUPPORTED: unsupported dtype combination";
    case ZPP_ERR_CUDA: return "ZPP_ERR_CUDA: CUDA runtime error at launch";
  }
  return "unknown zpp_status";
}

zpp_status zpp_quant_blockwise(const void* x, zpp_dtype x_dt, int64_t n, int32_t block,
                               int32_t bits, void* codes, float* scales, cudaStream_t stream) {
  if (!valid_bits(bits) || !valid_block(block) || n < 0 || n > ZPP_MAX_ELEMS)
    return ZPP_ERR_INVALID_ARG;
  if (x_dt != ZPP_F16 && x_dt != ZPP_BF16 && x_dt != ZPP_F32) return ZPP_ERR_INVALID_ARG;
  if (n == 0) return ZPP_OK;
  if (!x || !codes || !scales) return ZPP_ERR_INVALID_ARG;
  if (x_dt == ZPP_F32) return ZPP_ERR_UNSUPPORTED;
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return ZPP_ERR_MISALIGNED;
  return from_cuda(zpp::launch_quant(x, x_dt == ZPP_BF16, n, block, bits, codes, scales, stream));
}

zpp_status zpp_dequant_blockwise(const void* codes, const float* scales, int64_t n, int32_t block,
                                 int32_t bits, void* y, zpp_dtype y_dt, cudaStream_t stream) {
  if (!valid_bits(bits) || !valid_block(block) || n < 0 || n > ZPP_MAX_ELEMS)
    return ZPP_ERR_INVALID_ARG;
  if (y_dt != ZPP_F16 && y_dt != ZPP_BF16 && y_dt != ZPP_F32) return ZPP_ERR_INVALID_ARG;
  if (n == 0) return ZPP_OK;
  if (!codes || !scales || !y) return ZPP_ERR_INVALID_ARG;
  if (!aligned(codes, 16) || !aligned(y, 16) || !aligned(scales, 4)) return ZPP_ERR_MISALIGNED;
  return from_cuda(zpp::launch_dequant(codes, scales, n, block, bits, y, static_cast<int>(y_dt), stream));
}

zpp_status zpp_qgz_reorder_quant_range(const void* grads, zpp_dtype g_dt, int64_t elems_per_rank,
                                       int32_t block, int32_t bits, zpp_topology topo,
                                       zpp_local_range range, void* codes, float* scales,
                                       cudaStream_t stream) {
  int64_t W = 0;
  zpp_status st = check_topology(elems_per_rank, block, bits, topo, &W);
  if (st != ZPP_OK) return st;
  if (g_dt != ZPP_F16 && g_dt != ZPP_BF16 && g_dt != ZPP_F32) return ZPP_ERR_INVALID_ARG;
  if (!valid_range(range, topo)) return ZPP_ERR_INVALID_ARG;
  if (elems_per_rank == 0 || range.begin == range.end) return ZPP_OK;
  if (!grads || !codes || !scales) return ZPP_ERR_INVALID_ARG;
  if (g_dt == ZPP_F32) return ZPP_ERR_UNSUPPORTED;
  if (!aligned(grads, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return ZPP_ERR_MISALIGNED;
  return from_cuda(zpp::launch_reorder_quant(grads, g_dt == ZPP_BF16, elems_per_rank, block, bits,
                                             topo.num_nodes, topo.gpus_per_node, range.begin,
                                             range.end, static_cast<int>(W), codes, scales,
                                             stream));
}

zpp_status zpp_qgz_reorder_quant(const void* grads, zpp_dtype g_dt, int64_t elems_per_rank,
                                 int32_t block, int32_t bits, zpp_topology topo, void* codes,
                                 float* scales, cudaStream_t stream) {
  return zpp_qgz_reorder_quant_range(grads, g_dt, elems_per_rank, block, bits, topo,
                                     full_range(topo), codes, scales, stream);
}

zpp_status zpp_qgz_reorder_quant_tensors(const void* const* tensors, const int64_t* sizes,
                                         int32_t num_tensors, zpp_dtype g_dt, int32_t block,
                                         int32_t bits, zpp_topology topo, void* codes,
                                         float* scales, cudaStream_t stream) {
  static_assert(zpp::kMaxTensors == ZPP_MAX_TENSORS, "tensor table size");
  if (!tensors || !sizes || num_tensors < 1 || num_tensors > ZPP_MAX_TENSORS)
    return ZPP_ERR_INVALID_ARG;
  int64_t E = 0;
  for (int32_t t = 0; t < num_tensors; ++t) {
    if (sizes[t] < 0 || sizes[t] >= (int64_t{1} << 31)) return ZPP_ERR_INVALID_ARG;
    E += sizes[t];
    if (E >= (int64_t{1} << 31)) return ZPP_ERR_INVALID_ARG;
  }
  int64_t W = 0;
  zpp_status st = check_topology(E, block, bits, topo, &W);
  if (st != ZPP_OK) return st;
  if (g_dt != ZPP_F16 && g_dt != ZPP_BF16 && g_dt != ZPP_F32) return ZPP_ERR_INVALID_ARG;
  if (E == 0) return ZPP_OK;
  if (!codes || !scales) return ZPP_ERR_INVALID_ARG;
  for (int32_t t = 0; t < num_tensors; ++t)
    if (sizes[t] > 0 && !tensors[t]) return ZPP_ERR_INVALID_ARG;
  if (g_dt == ZPP_F32) return ZPP_ERR_UNSUPPORTED;
  for (int32_t t = 0; t < num_tensors; ++t)
    if (sizes[t] % 16 != 0 || (sizes[t] > 0 && !aligned(tensors[t], 16))) return ZPP_ERR_MISALIGNED;
  if (!aligned(codes, 16) || !aligned(scales, 4)) return ZPP_ERR_MISALIGNED;
  zpp::TensorTable tab;
  tab.count = num_tensors;
  tab.offs[0] = 0;
  for (int32_t t = 0; t < num_tensors; ++t) {
    tab.ptr[t] = static_cast<const uint16_t*>(tensors[t]);
    tab.offs[t + 1] = tab.offs[t] + sizes[t];
  }
  return from_cuda(zpp::launch_reorder_quant_tensors(tab, g_dt == ZPP_BF16, E, block, bits,
                                                     topo.num_nodes, topo.gpus_per_node, codes,
                                                     scales, stream));
}

zpp_status zpp_dequant_reduce_requant_range(const void* codes, const float* scales,
                                            int64_t elems_per_rank, int32_t block, int32_t bits,
                                            zpp_topology topo, zpp_local_range range,
                                            void* out_codes, float* out_scales,
                                            cudaStream_t stream) {
  int64_t W = 0;
  zpp_status st = check_topology(elems_per_rank, block, bits, topo, &W);
  if (st != ZPP_OK) return st;
  if (!valid_range(range, topo)) return ZPP_ERR_INVALID_ARG;
  if (elems_per_rank == 0 || range.begin == range.end) return ZPP_OK;
  if (!codes || !scales || !out_codes || !out_scales) return ZPP_ERR_INVALID_ARG;
  if (!aligned(codes, 16) || !aligned(out_codes, 16) || !aligned(scales, 4) ||
      !aligned(out_scales, 4))
    return ZPP_ERR_MISALIGNED;
  return from_cuda(zpp::launch_dequant_reduce_requant(
      codes, scales, elems_per_rank, elems_per_rank / topo.gpus_per_node, block, bits,
      topo.num_nodes, topo.gpus_per_node, range.begin, range.end, out_codes, out_scales, stream));
}

zpp_status zpp_dequant_reduce_requant(const void* codes, const float* scales,
                                      int64_t elems_per_rank, int32_t block, int32_t bits,
                                      zpp_topology topo, void* out_codes, float* out_scales,
                                      cudaStream_t stream) {
  return zpp_dequant_reduce_requant_range(codes, scales, elems_per_rank, block, bits, topo,
                                          full_range(topo), out_codes, out_scales, stream);
}

zpp_status zpp_dequant_reduce_scaled_range(const void* codes, const float* scales,
                                           int64_t elems_per_rank, int32_t block, int32_t bits,
                                           zpp_topology topo, zpp_local_range range,
                                           float post_scale, void* out, zpp_dtype out_dt,
                                           cudaStream_t stream) {
  int64_t W = 0;
  zpp_status st = check_topology(elems_per_rank, block, bits, topo, &W);
  if (st != ZPP_OK) return st;
  if (out_dt != ZPP_F16 && out_dt != ZPP_BF16 && out_dt != ZPP_F32) return ZPP_ERR_INVALID_ARG;
  if (!(post_scale == post_scale) || post_scale - post_scale != 0.0f) return ZPP_ERR_INVALID_ARG;
  if (!valid_range(range, topo)) return ZPP_ERR_INVALID_ARG;
  if (elems_per_rank == 0 || range.begin == range.end) return ZPP_OK;
  if (!codes || !scales || !out) return ZPP_ERR_INVALID_ARG;
  if (!aligned(codes, 16) || !aligned(out, 16) || !aligned(scales, 4)) return ZPP_ERR_MISALIGNED;
  return from_cuda(zpp::launch_dequant_reduce(
      codes, scales, elems_per_rank / W, elems_per_rank / topo.gpus_per_node, block, bits,
      topo.num_nodes, topo.gpus_per_node, range.begin, range.end, topo.num_nodes, post_scale, out,
      static_cast<int>(out_dt), stream));
}

zpp_status zpp_dequant_reduce_scaled(const void* codes, const float* scales,
                                     int64_t elems_per_rank, int32_t block, int32_t bits,
                                     zpp_topology topo, float post_scale, void* out,
                                     zpp_dtype out_dt, cudaStream_t stream) {
  return zpp_dequant_reduce_scaled_range(codes, scales, elems_per_rank, block, bits, topo,
                                         full_range(topo), post_scale, out, out_dt, stream);
}

zpp_status zpp_dequant_reduce(const void* codes, const float* scales, int64_t elems_per_rank,
                              int32_t block, int32_t bits, zpp_topology topo, float* out,
                              cudaStream_t stream) {
  return zpp_dequant_reduce_scaled_range(codes, scales, elems_per_rank, block, bits, topo,
                                         full_range(topo), 1.0f, out, ZPP_F32, stream);
}

zpp_status zpp_qgz_reorder_quant_local(const void* grads, zpp_dtype g_dt, int64_t elems_per_rank,
                                       int32_t block, int32_t bits, zpp_topology topo,
                                       zpp_local_range range, void* codes, float* scales,
                                       cudaStream_t stream) {
  int64_t W = 0;
  zpp_status st = check_topology(elems_per_rank, block, bits, topo, &W);
  if (st != ZPP_OK) return st;
  if (g_dt != ZPP_F16 && g_dt != ZPP_BF16 && g_dt != ZPP_F32) return ZPP_ERR_INVALID_ARG;
  if (!valid_range(range, topo)) return ZPP_ERR_INVALID_ARG;
  if (elems_per_rank == 0 || range.begin == range.end) return ZPP_OK;
  if (!grads || !codes || !scales) return ZPP_ERR_INVALID_ARG;
  if (g_dt == ZPP_F32) return ZPP_ERR_UNSUPPORTED;
  if (!aligned(grads, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return ZPP_ERR_MISALIGNED;
  return from_cuda(zpp::launch_reorder_quant(grads, g_dt == ZPP_BF16, elems_per_rank, block, bits,
                                             topo.num_nodes, topo.gpus_per_node, range.begin,
                                             range.end, 1, codes, scales, stream));
}

namespace {
// Checks shared by the two calls on received chunks: `len` elements per source, a
// multiple of the block, `sources` of them.
zpp_status check_received(int64_t len, int32_t block, int32_t bits, int32_t sources) {
  if (!valid_bits(bits) || !valid_block(block)) return ZPP_ERR_INVALID_ARG;
  if (sources < 1 || sources > 65535) return ZPP_ERR_INVALID_ARG;
  if (len < 0 || len >= (int64_t{1} << 31) || len % block != 0) return ZPP_ERR_INVALID_ARG;
  if (len * sources > ZPP_MAX_ELEMS) return ZPP_ERR_INVALID_ARG;
  return ZPP_OK;
}
}  // namespace

zpp_status zpp_dequant_reduce_requant_local(const void* codes, const float* scales, int64_t chunk,
                                            int32_t block, int32_t bits, int32_t sources,
                                            void* out_codes, float* out_scales,
                                            cudaStream_t stream) {
  const zpp_status st = check_received(chunk, block, bits, sources);
  if (st != ZPP_OK) return st;
  if (chunk == 0) return ZPP_OK;
  if (!codes || !scales || !out_codes || !out_scales) return ZPP_ERR_INVALID_ARG;
  if (!aligned(codes, 16) || !aligned(out_codes, 16) || !aligned(scales, 4) ||
      !aligned(out_scales, 4))
    return ZPP_ERR_MISALIGNED;
  // one receiver (N = 1, l = 0) whose sources are the received chunks, `chunk` apart
  return from_cuda(zpp::launch_dequant_reduce_requant(codes, scales, chunk, chunk, block, bits, 1,
                                                      sources, 0, 1, out_codes, out_scales,
                                                      stream));
}

zpp_status zpp_dequant_reduce_local(const void* codes, const float* scales, int64_t slice,
                                    int32_t block, int32_t bits, int32_t sources,
                                    float post_scale, void* out, zpp_dtype out_dt,
                                    cudaStream_t stream) {
  const zpp_status st = check_received(slice, block, bits, sources);
  if (st != ZPP_OK) return st;
  if (out_dt != ZPP_F16 && out_dt != ZPP_BF16 && out_dt != ZPP_F32) return ZPP_ERR_INVALID_ARG;
  if (!(post_scale == post_scale) || post_scale - post_scale != 0.0f) return ZPP_ERR_INVALID_ARG;
  if (slice == 0) return ZPP_OK;
  if (!codes || !scales || !out) return ZPP_ERR_INVALID_ARG;
  if (!aligned(codes, 16) || !aligned(out, 16) || !aligned(scales, 4)) return ZPP_ERR_MISALIGNED;
  // one receiver (n = 0, l = 0) whose N sources are the received slices, `slice` apart
  return from_cuda(zpp::launch_dequant_reduce(codes, scales, slice, slice, block, bits, sources, 1,
                                              0, 1, 1, post_scale, out, static_cast<int>(out_dt),
                                              stream));
}

namespace {
bool valid_dtype(zpp_dtype t) { return t == ZPP_F16 || t == ZPP_BF16 || t == ZPP_F32; }
bool is_finite(double v) { return v - v == 0.0; }
}  // namespace

int64_t zpp_grad_norm_workspace(int64_t total_elems, int32_t num_tensors) {
  if (total_elems < 0 || num_tensors < 0) return -1;
  // every tensor rounds up to whole chunks; one float more for an empty list
  return total_elems / zpp::kNormChunk + num_tensors + 1;
}

zpp_status zpp_grad_norm(const void* const* grads, const int64_t* sizes, int32_t num_tensors,
                         zpp_dtype g_dt, float pre_scale, float max_norm, float* workspace,
                         float* out, cudaStream_t stream) {
  if (num_tensors < 0 || num_tensors > ZPP_MAX_TENSORS || !valid_dtype(g_dt))
    return ZPP_ERR_INVALID_ARG;
  if (num_tensors > 0 && (!grads || !sizes)) return ZPP_ERR_INVALID_ARG;
  if (!is_finite(pre_scale) || !(max_norm > 0.0f)) return ZPP_ERR_INVALID_ARG;
  if (!workspace || !out) return ZPP_ERR_INVALID_ARG;
  int64_t total = 0;
  for (int32_t t = 0; t < num_tensors; ++t) {
    if (sizes[t] < 0 || sizes[t] > ZPP_MAX_ELEMS) return ZPP_ERR_INVALID_ARG;
    total += sizes[t];
    if (total > ZPP_MAX_ELEMS) return ZPP_ERR_INVALID_ARG;
    if (sizes[t] > 0 && !grads[t]) return ZPP_ERR_INVALID_ARG;
  }
  for (int32_t t = 0; t < num_tensors; ++t)
    if (sizes[t] > 0 && !aligned(grads[t], 16)) return ZPP_ERR_MISALIGNED;
  if (!aligned(workspace, 4) || !aligned(out, 4)) return ZPP_ERR_MISALIGNED;
  zpp::NormTable tab;
  tab.count = num_tensors;
  tab.first[0] = 0;
  for (int32_t t = 0; t < num_tensors; ++t) {
    tab.ptr[t] = grads[t];
    tab.n[t] = sizes[t];
    tab.first[t + 1] = tab.first[t] + static_cast<int32_t>(zpp::norm_chunks(sizes[t]));
  }
  return from_cuda(zpp::launch_grad_norm(tab, static_cast<int>(g_dt), pre_scale, max_norm,
                                         workspace, out, zpp::StepCount{}, stream));
}

namespace {

// The arguments that both forms of the step share. step_min: the smallest number of a step.
zpp_status check_adamw(const zpp_adamw_tensor* tensors, int32_t num_tensors, zpp_dtype g_dt,
                       zpp_dtype w_dt, int32_t state_bits, const zpp_adamw_params* hp,
                       int64_t step_min, const float* grad_scale) {
  static_assert(zpp::kStateBlock == ZPP_STATE_BLOCK, "state block");
  if (num_tensors < 0 || num_tensors > ZPP_MAX_TENSORS || (num_tensors > 0 && !tensors) || !hp)
    return ZPP_ERR_INVALID_ARG;
  if (!valid_dtype(g_dt) || !valid_dtype(w_dt) || (state_bits != 8 && state_bits != 32))
    return ZPP_ERR_INVALID_ARG;
  if (!is_finite(hp->lr) || !is_finite(hp->weight_decay) || !is_finite(hp->eps) || hp->eps < 0.0 ||
      !(hp->beta1 >= 0.0 && hp->beta1 < 1.0) || !(hp->beta2 >= 0.0 && hp->beta2 < 1.0) ||
      hp->step < step_min)
    return ZPP_ERR_INVALID_ARG;
  int64_t total = 0;
  bool any_weight = false;
  for (int32_t i = 0; i < num_tensors; ++i) {
    const zpp_adamw_tensor& t = tensors[i];
    if (t.n < 0 || t.n > ZPP_MAX_ELEMS) return ZPP_ERR_INVALID_ARG;
    total += t.n;
    if (total > ZPP_MAX_ELEMS) return ZPP_ERR_INVALID_ARG;
    if (t.n == 0) continue;
    if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq) return ZPP_ERR_INVALID_ARG;
    if (state_bits == 8 && (!t.exp_avg_scale || !t.exp_avg_sq_scale)) return ZPP_ERR_INVALID_ARG;
    any_weight |= t.weight != nullptr;
  }
  if (any_weight && w_dt == ZPP_F32) return ZPP_ERR_UNSUPPORTED;
  for (int32_t i = 0; i < num_tensors; ++i) {
    const zpp_adamw_tensor& t = tensors[i];
    if (t.n == 0) continue;
    if (!aligned(t.param, 16) || !aligned(t.grad, 16) || !aligned(t.exp_avg, 16) ||
        !aligned(t.exp_avg_sq, 16) || !aligned(t.weight, 16))
      return ZPP_ERR_MISALIGNED;
    if (state_bits == 8 && (!aligned(t.exp_avg_scale, 4) || !aligned(t.exp_avg_sq_scale, 4)))
      return ZPP_ERR_MISALIGNED;
  }
  return aligned(grad_scale, 4) ? ZPP_OK : ZPP_ERR_MISALIGNED;
}

// beta^step and the factors made from it, in 64 bits, rounded once.
struct StepFactors {
  double power[2];
  float step_size, inv_root_bc2;
  explicit StepFactors(const zpp_adamw_params& hp) {
    const double t = static_cast<double>(hp.step);
    power[0] = std::pow(hp.beta1, t);
    power[1] = std::pow(hp.beta2, t);
    step_size = static_cast<float>(hp.lr / (1.0 - power[0]));
    inv_root_bc2 = static_cast<float>(1.0 / std::sqrt(1.0 - power[1]));
  }
};

// record: null, or the step's record: told hp->step where that is known, read where it is 0.
zpp_status run_adamw(const zpp_adamw_tensor* tensors, int32_t num_tensors, zpp_dtype g_dt,
                     zpp_dtype w_dt, int32_t state_bits, const zpp_adamw_params* hp,
                     const float* grad_scale, zpp_adamw_record* record, cudaStream_t stream) {
  zpp::AdamwTable tab;
  zpp::AdamwArgs& a = tab.a;
  a.beta1 = static_cast<float>(hp->beta1);
  a.one_minus_beta1 = static_cast<float>(1.0 - hp->beta1);
  a.beta2 = static_cast<float>(hp->beta2);
  a.one_minus_beta2 = static_cast<float>(1.0 - hp->beta2);
  if (hp->step > 0) {
    const StepFactors f(*hp);
    a.step_size = f.step_size;
    a.inv_root_bc2 = f.inv_root_bc2;
  }
  // The denominator's reciprocal takes a subnormal for zero, and 0 / eps has to stay 0.
  a.eps = hp->eps > 0.0 ? std::max(static_cast<float>(hp->eps), std::numeric_limits<float>::min()) : 0.0f;
  a.decay = static_cast<float>(hp->lr * hp->weight_decay);
  a.key = (hp->seed * 0x9E3779B9u) ^ (static_cast<uint32_t>(hp->step) * 0x510E527Fu);
  a.grad_scale = grad_scale;
  a.record = reinterpret_cast<zpp::StepRecord*>(record);
  a.step = hp->step;
  a.g_kind = static_cast<int32_t>(g_dt);
  a.w_kind = static_cast<int32_t>(w_dt);
  tab.first_block = 0;
  int64_t blocks = 0;
  for (int32_t i = 0; i < num_tensors;) {  // one launch per kAdamwTensors non-empty tensors
    tab.count = 0;
    tab.first[0] = 0;
    tab.first_block = blocks;
    for (; i < num_tensors && tab.count < zpp::kAdamwTensors; ++i) {
      const zpp_adamw_tensor& s = tensors[i];
      if (s.n == 0) continue;
      const int32_t c = tab.count++;
      tab.t[c] = zpp::AdamwTensor{s.param,         s.grad,             s.exp_avg, s.exp_avg_sq,
                                  s.exp_avg_scale, s.exp_avg_sq_scale, s.weight,  s.n};
      tab.first[c + 1] = tab.first[c] + static_cast<int32_t>(zpp::adamw_chunks(s.n, state_bits));
      tab.block0[c] = static_cast<int32_t>(blocks - tab.first_block);
      blocks += (s.n + ZPP_STATE_BLOCK - 1) / ZPP_STATE_BLOCK;
    }
    if (tab.count == 0) break;
    const zpp_status st = from_cuda(zpp::launch_adamw(tab, state_bits, stream));
    if (st != ZPP_OK) return st;
  }
  return ZPP_OK;
}

}  // namespace

zpp_status zpp_adamw_step(const zpp_adamw_tensor* tensors, int32_t num_tensors, zpp_dtype g_dt,
                          zpp_dtype w_dt, int32_t state_bits, const zpp_adamw_params* hp,
                          const float* grad_scale, cudaStream_t stream) {
  const zpp_status st =
      check_adamw(tensors, num_tensors, g_dt, w_dt, state_bits, hp, 1, grad_scale);
  if (st != ZPP_OK) return st;
  return run_adamw(tensors, num_tensors, g_dt, w_dt, state_bits, hp, grad_scale, nullptr, stream);
}

zpp_status zpp_adamw_step_counted(const zpp_adamw_tensor* tensors, int32_t num_tensors,
                                  zpp_dtype g_dt, zpp_dtype w_dt, int32_t state_bits,
                                  const zpp_adamw_params* hp, const float* grad_scale,
                                  const zpp_adamw_clip* clip, zpp_adamw_record* record,
                                  cudaStream_t stream) {
  static_assert(sizeof(zpp_adamw_record) == sizeof(zpp::StepRecord) &&
                    offsetof(zpp_adamw_record, factor) == offsetof(zpp::StepRecord, factor) &&
                    offsetof(zpp_adamw_record, power) == offsetof(zpp::StepRecord, power) &&
                    offsetof(zpp::StepRecord, factor) % 16 == 0,
                "the record's layout");
  zpp_status st = check_adamw(tensors, num_tensors, g_dt, w_dt, state_bits, hp, 0, grad_scale);
  if (st != ZPP_OK) return st;
  if (!record || (clip && grad_scale)) return ZPP_ERR_INVALID_ARG;
  if (clip) {
    if (!is_finite(clip->pre_scale) || !(clip->max_norm > 0.0f) || !clip->workspace || !clip->out)
      return ZPP_ERR_INVALID_ARG;
    if (!aligned(clip->workspace, 4) || !aligned(clip->out, 4)) return ZPP_ERR_MISALIGNED;
  }
  if (!aligned(record, 16)) return ZPP_ERR_MISALIGNED;

  bool elements = false;
  for (int32_t i = 0; i < num_tensors; ++i) elements |= tensors[i].n > 0;
  // A step whose number the host knows and that cannot be skipped leaves its number as it runs.
  if (hp->step > 0 && !clip && !grad_scale && elements)
    return run_adamw(tensors, num_tensors, g_dt, w_dt, state_bits, hp, nullptr, record, stream);

  zpp::StepCount count{};
  count.lr = hp->lr;
  count.beta[0] = hp->beta1;
  count.beta[1] = hp->beta2;
  count.known = hp->step;
  count.seed = hp->seed;
  count.record = reinterpret_cast<zpp::StepRecord*>(record);
  if (hp->step > 0) {
    const StepFactors f(*hp);
    count.power[0] = f.power[0];
    count.power[1] = f.power[1];
    count.step_size = f.step_size;
    count.inv_root_bc2 = f.inv_root_bc2;
  }
  if (clip) {
    zpp::NormTable tab;
    tab.count = num_tensors;
    tab.first[0] = 0;
    for (int32_t i = 0; i < num_tensors; ++i) {
      tab.ptr[i] = tensors[i].grad;
      tab.n[i] = tensors[i].n;
      tab.first[i + 1] = tab.first[i] + static_cast<int32_t>(zpp::norm_chunks(tensors[i].n));
    }
    st = from_cuda(zpp::launch_grad_norm(tab, static_cast<int>(g_dt), clip->pre_scale, clip->max_norm,
                                         clip->workspace, clip->out, count, stream));
  } else {
    st = from_cuda(zpp::launch_step_count(count, grad_scale, stream));
  }
  if (st != ZPP_OK) return st;
  zpp_adamw_params recorded = *hp;
  recorded.step = 0;
  return run_adamw(tensors, num_tensors, g_dt, w_dt, state_bits, &recorded, nullptr, record, stream);
}

zpp_status zpp_matvec_blockwise(const void* codes, const float* scales, int64_t rows, int64_t cols,
                                int32_t block, int32_t bits, const void* x, zpp_dtype x_dt,
                                int64_t vecs, int64_t x_stride, const void* bias, void* y,
                                zpp_dtype y_dt, int64_t y_stride, cudaStream_t stream) {
  if (!valid_bits(bits) || !valid_block(block)) return ZPP_ERR_INVALID_ARG;
  if (!valid_dtype(x_dt) || !valid_dtype(y_dt)) return ZPP_ERR_INVALID_ARG;
  constexpr int64_t kDim = int64_t{1} << 31;
  if (rows < 0 || rows >= kDim || cols < 1 || cols >= kDim || vecs < 0 || vecs > 65535)
    return ZPP_ERR_INVALID_ARG;
  if (rows > ZPP_MAX_ELEMS / cols) return ZPP_ERR_INVALID_ARG;
  if (x_stride < cols || x_stride > ZPP_MAX_ELEMS || y_stride < rows || y_stride > ZPP_MAX_ELEMS)
    return ZPP_ERR_INVALID_ARG;
  if (rows == 0 || vecs == 0) return ZPP_OK;
  if (!codes || !scales || !x || !y) return ZPP_ERR_INVALID_ARG;
  if (x_dt == ZPP_F32) return ZPP_ERR_UNSUPPORTED;
  if (!aligned(codes, 16) || !aligned(x, 16) || !aligned(y, 16) || !aligned(scales, 4) ||
      !aligned(bias, 2))
    return ZPP_ERR_MISALIGNED;
  zpp::MatvecArgs a;
  a.codes = static_cast<const uint8_t*>(codes);
  a.scales = scales;
  a.rows = rows;
  a.cols = cols;
  a.block = block;
  a.bits = bits;
  a.x = static_cast<const uint16_t*>(x);
  a.x_bf16 = x_dt == ZPP_BF16;
  a.vecs = vecs;
  a.x_stride = x_stride;
  a.bias = static_cast<const uint16_t*>(bias);
  a.y = y;
  a.y_kind = static_cast<int32_t>(y_dt);
  a.y_stride = y_stride;
  return from_cuda(zpp::launch_matvec(a, stream));
}

zpp_status zpp_device_fault(uint32_t* flags, int32_t clear) {
  if (!flags) return ZPP_ERR_INVALID_ARG;
  unsigned v = 0;
  const zpp_status st = from_cuda(zpp::read_device_fault(&v, clear != 0));
  *flags = st == ZPP_OK ? v : 0u;
  return st;
}

zpp_status zpp_wait_selftest(uint64_t limit_ns, cudaStream_t stream) {
  if (limit_ns == 0 || limit_ns > 10000000000ull) return ZPP_ERR_INVALID_ARG;
  return from_cuda(zpp::launch_wait_selftest(limit_ns, stream));
}

zpp_status zpp_device_copy(const void* src, void* dst, int64_t bytes, cudaStream_t stream) {
  if (bytes < 0 || bytes % 32 != 0) return ZPP_ERR_INVALID_ARG;
  if (bytes == 0) return ZPP_OK;
  if (!src || !dst) return ZPP_ERR_INVALID_ARG;
  if (!aligned(src, 32) || !aligned(dst, 32)) return ZPP_ERR_MISALIGNED;
  return from_cuda(zpp::launch_copy(src, dst, bytes, stream));
}

}  // extern "C"
