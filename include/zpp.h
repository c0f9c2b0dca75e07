/*
 * zpp.h -- C ABI of the GB300 (sm_103a) ZeRO++ block-quantisation hot path.
 *
 * Pages cited (by title; the section follows the label):
 *   [ZeRO++ summary]  "ZeRO++: Extremely Efficient Collective Communication for Large
 *                      Model Training" (atlas.scime.ai summary)
 *   [ZeRO++ abstract] "ZeRO++: Extremely Efficient Collective Communication for Giant
 *                      Model Training" (mlsanity.com record, arXiv abstract)
 *   [LIT-102]         "LIT-102: ZeRO++: Extremely Efficient Collective Communication
 *                      for Giant Model Training" (anthology-of-the-sota record)
 *
 * What the calls compute (the pages fix the structure, not the formula; this is the
 * reading every entry point implements, bit for bit):
 *   per block of `block` consecutive elements (the last block may be shorter):
 *     amax  = max |x|;  scale = fp32(amax / qmax);  inv = fp32(qmax / amax)
 *     q     = clamp(rint_to_even(x * inv), -qmax, qmax),  qmax = 2^(bits-1) - 1,
 *             the product x * inv taken exactly (rounded once, to an integer)
 *     amax == 0 or inv not finite  ->  scale = 0 and every q = 0
 *   dequantise: y = fp32((float)q * scale), then round-to-nearest-even into y's type.
 *   reduce (the qgZ hops): sum = fma(q, scale, sum) per received chunk -- one rounding
 *   per term -- starting from +0.0f, sources in ascending order.
 *
 * Storage: INT8 codes are two's-complement bytes; INT4 codes are two's-complement
 * nibbles, element 2i in the LOW nibble of byte i and 2i+1 in the high nibble (an odd
 * trailing element leaves the high nibble 0). Scales are a separate fp32 array, one
 * per block, in block order.
 *
 * Virtual topology (qgZ): N nodes x M GPUs per node, W = N*M ranks, rank r = n*M + l.
 * Ranks are HBM buffers laid out back to back ([W][...]); the all-to-all exchanges are
 * index maps over them, no data is moved between the steps.
 *   E = elements per rank, S = E / W (the slice each rank owns), C = N*S (hop-1 chunk).
 *
 * Conventions for every entry point:
 *   - All buffer pointers are DEVICE pointers owned by the caller. The library
 *     allocates nothing, never synchronises, and only enqueues kernels on `stream`
 *     (0 = the legacy default stream). The stream's device has to be the current one.
 *   - Inputs and outputs must not overlap.
 *   - Arguments are checked on the host before any launch; on an error nothing is
 *     launched and nothing is written.
 *   - Alignment: element and code buffers (x, y, grads, codes, out, and the tensors of
 *     zpp_qgz_reorder_quant_tensors) must be 16-byte aligned; scale arrays 4-byte
 *     aligned. Element buffers that are also 32-byte aligned take 256-bit vector accesses,
 *     16-byte aligned ones 128-bit accesses; the results are the same bits.
 *   - n == 0 (or a zero-sized topology payload) returns ZPP_OK and launches nothing.
 *   - A launch failure is reported as ZPP_ERR_CUDA (from cudaGetLastError); an
 *     asynchronous fault surfaces at the caller's next synchronisation.
 *   - Inputs must be finite; NaN or Inf inputs give unspecified codes.
 */
#ifndef ZPP_H
#define ZPP_H

#include <stdint.h>
#include <cuda_runtime_api.h>

#if defined(__GNUC__)
#define ZPP_API __attribute__((visibility("default")))
#else
#define ZPP_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum zpp_status {
  ZPP_OK = 0,
  ZPP_ERR_INVALID_ARG = 1, /* bad bits / block / size / topology / null pointer */
  ZPP_ERR_MISALIGNED = 2,  /* a pointer breaks the alignment rule above */
  ZPP_ERR_UNSUPPORTED = 3, /* a valid but unimplemented dtype combination */
  ZPP_ERR_CUDA = 4         /* the CUDA runtime reported an error at launch */
} zpp_status;

typedef enum zpp_dtype { ZPP_F16 = 0, ZPP_BF16 = 1, ZPP_F32 = 2 } zpp_dtype;

typedef struct zpp_topology {
  int32_t num_nodes;     /* N >= 1 */
  int32_t gpus_per_node; /* M >= 1 */
} zpp_topology;

/* A range [begin, end) of local GPU indices l (0 <= begin <= end <= M). The qgZ exchange
 * splits exactly by l: hop-1 chunk l of every rank feeds only the receivers with local
 * index l, whose hop-1 outputs feed only the hop-2 receivers with local index l. So the
 * three qgZ steps restricted to one range form an independent sub-pipeline, and the
 * ranges of a partition of [0, M) may run on different streams (the pipelining of the
 * intra- and inter-node hops, on one GPU). */
typedef struct zpp_local_range {
  int32_t begin;
  int32_t end;
} zpp_local_range;

/* Limits checked by every entry point. */
#define ZPP_MIN_BLOCK 64
#define ZPP_MAX_BLOCK 4096
#define ZPP_MAX_ELEMS (((int64_t)1) << 38)
#define ZPP_MAX_TENSORS 1024 /* tensors per bucket in zpp_qgz_reorder_quant_tensors */

/*
 * qwZ step 1 -- block-wise symmetric quantisation of a weight shard before the forward
 * all-gather ([ZeRO++ summary] Approach: block-wise INT8 weight quantisation;
 * [ZeRO++ abstract]: block-quantisation based all-gather; [LIT-102] Key takeaways:
 * block-wise rather than per-tensor). Also the INT4 gradient quantiser of qgZ.
 *   x      : [n] elements of x_dt (ZPP_F16 or ZPP_BF16; ZPP_F32 -> ZPP_ERR_UNSUPPORTED)
 *   n      : element count, 0 <= n <= ZPP_MAX_ELEMS
 *   block  : power of two in [64, 4096]
 *   bits   : 8 or 4
 *   codes  : out, zpp_code_bytes(n, bits) bytes
 *   scales : out, zpp_num_scales(n, block) floats
 * Shards whose sizes are multiples of `block` can be quantised in one call over their
 * concatenation: the result is identical to one call per shard.
 */
ZPP_API zpp_status zpp_quant_blockwise(const void* x, zpp_dtype x_dt, int64_t n, int32_t block,
                               int32_t bits, void* codes, float* scales, cudaStream_t stream);

/*
 * qwZ step 2 -- dequantisation of the gathered codes after the all-gather
 * ([ZeRO++ summary] Approach; [ZeRO++ abstract]: block-quantisation based all-gather).
 *   codes  : [zpp_code_bytes(n, bits)] bytes; scales: [zpp_num_scales(n, block)] floats
 *   y      : out, [n] elements of y_dt (ZPP_F16, ZPP_BF16 or ZPP_F32)
 * Other arguments as in zpp_quant_blockwise.
 */
ZPP_API zpp_status zpp_dequant_blockwise(const void* codes, const float* scales, int64_t n,
                                 int32_t block, int32_t bits, void* y, zpp_dtype y_dt,
                                 cudaStream_t stream);

/*
 * qgZ step 1 -- tensor-slice reordering plus block quantisation of every rank's
 * gradient before the 2-hop all-to-all ([ZeRO++ summary] Approach: slices reordered
 * so each reduced slice lands on its owner; INT4 gradient reduction).
 * Each rank's E elements are W slices of S; original slice j = n_d*M + l_d (owned by
 * rank j) is written at position p = l_d*N + n_d, so the reordered buffer is M chunks
 * of C = N*S, chunk l going to local peer l in hop 1. Quantisation then runs over the
 * reordered buffer (blocks never straddle slices).
 *   grads          : [W][E] elements of g_dt (ZPP_F16 or ZPP_BF16)
 *   elems_per_rank : E, a multiple of W*block, E < 2^31
 *   bits           : 4 (the pages' INT4); 8 is accepted as an extension
 *   codes          : out, [W][zpp_code_bytes(E, bits)]
 *   scales         : out, [W][E/block]
 */
ZPP_API zpp_status zpp_qgz_reorder_quant(const void* grads, zpp_dtype g_dt, int64_t elems_per_rank,
                                 int32_t block, int32_t bits, zpp_topology topo,
                                 void* codes, float* scales, cudaStream_t stream);

/*
 * qgZ step 1 with the bucket flatten fused in. A rank's gradient bucket is usually the
 * concatenation of many parameter gradients; this call reads them where they are
 * instead of from a flattened copy, and writes exactly (bit for bit) what
 * zpp_qgz_reorder_quant writes for the bucket whose rank r holds, in order, its copies of
 * tensors 0..num_tensors-1 ([ZeRO++ summary] Approach: slices reordered for correct
 * placement). The flattening copy -- a full read and write of the bucket -- is saved.
 *   tensors     : HOST array [num_tensors] of device pointers; tensor t holds the W ranks'
 *                 copies back to back ([W][sizes[t]] elements of g_dt), 16-byte aligned
 *   sizes       : HOST array [num_tensors], elements per rank of tensor t: a multiple of
 *                 16 (else ZPP_ERR_MISALIGNED), 0 allowed (its pointer is then not read)
 *   num_tensors : 1 .. ZPP_MAX_TENSORS
 * E = the sum of sizes must satisfy the rules of zpp_qgz_reorder_quant (a multiple of
 * W*block, E < 2^31); codes and scales are as there. Tensors of one rank may cross slice
 * and block boundaries freely. Both host arrays are read during the call only.
 */
ZPP_API zpp_status zpp_qgz_reorder_quant_tensors(const void* const* tensors, const int64_t* sizes,
                                                 int32_t num_tensors, zpp_dtype g_dt,
                                                 int32_t block, int32_t bits, zpp_topology topo,
                                                 void* codes, float* scales, cudaStream_t stream);

/*
 * qgZ step 2 -- the fused kernel of the intra-node hop: every receiver (n, l)
 * dequantises chunk l of the M ranks of its node, sums them in fp32 (l' ascending) and
 * requantises the sums by blocks for the inter-node hop ([ZeRO++ summary] Approach:
 * dequantise before reduction; Measured effects table: fusion kernel; [LIT-102] Key
 * takeaways: reduce locally in higher precision). K = M chunks are read once.
 *   codes, scales  : the outputs of zpp_qgz_reorder_quant
 *   out_codes      : out, [W][zpp_code_bytes(C, bits)]
 *   out_scales     : out, [W][C/block]
 */
ZPP_API zpp_status zpp_dequant_reduce_requant(const void* codes, const float* scales,
                                      int64_t elems_per_rank, int32_t block, int32_t bits,
                                      zpp_topology topo, void* out_codes, float* out_scales,
                                      cudaStream_t stream);

/*
 * qgZ step 3 -- the inter-node hop's final dequantise-reduce: receiver (n, l)
 * dequantises slice n of the hop-1 output of rank (n', l) for n' = 0..N-1 and sums in
 * fp32 (n' ascending). The result is the SUM over all W ranks of the receiver's own
 * slice; scaling by 1/W for an average is left to the caller ([ZeRO++ summary]
 * Approach; [ZeRO++ abstract]: quantised gradient averaging).
 *   codes, scales  : the outputs of zpp_dequant_reduce_requant
 *   out            : out, [W][S] fp32
 */
ZPP_API zpp_status zpp_dequant_reduce(const void* codes, const float* scales, int64_t elems_per_rank,
                              int32_t block, int32_t bits, zpp_topology topo, float* out,
                              cudaStream_t stream);

/*
 * qgZ step 3 with the average folded in ([ZeRO++ abstract]: the gradient step averages
 * the ranks' gradients). Computes the same sums as zpp_dequant_reduce, multiplies each by
 * post_scale (one fp32 rounding; pass 1/W for the average, exact when W is a power of
 * two) and stores the result as out_dt with round-to-nearest-even.
 *   post_scale : finite, else ZPP_ERR_INVALID_ARG
 *   out        : out, [W][S] elements of out_dt (ZPP_F16, ZPP_BF16 or ZPP_F32)
 * Other arguments as in zpp_dequant_reduce.
 */
ZPP_API zpp_status zpp_dequant_reduce_scaled(const void* codes, const float* scales,
                                             int64_t elems_per_rank, int32_t block, int32_t bits,
                                             zpp_topology topo, float post_scale, void* out,
                                             zpp_dtype out_dt, cudaStream_t stream);

/*
 * The three qgZ steps restricted to the local indices of `range` ([ZeRO++ summary]
 * Approach: overlapped intra- and inter-node pipelining). Buffers have the full layouts
 * of the unrestricted calls; only the parts that belong to the range are read or written:
 *   zpp_qgz_reorder_quant_range     writes chunks l in range of every rank's codes/scales
 *   zpp_dequant_reduce_requant_range writes the hop-1 output of receivers (n, l), l in range
 *   zpp_dequant_reduce_scaled_range  writes the owner slices of ranks (n, l), l in range
 * An empty range returns ZPP_OK and launches nothing; a range outside [0, M] is
 * ZPP_ERR_INVALID_ARG. Results are bit-identical to the unrestricted calls.
 */
ZPP_API zpp_status zpp_qgz_reorder_quant_range(const void* grads, zpp_dtype g_dt,
                                               int64_t elems_per_rank, int32_t block,
                                               int32_t bits, zpp_topology topo,
                                               zpp_local_range range, void* codes,
                                               float* scales, cudaStream_t stream);
ZPP_API zpp_status zpp_dequant_reduce_requant_range(const void* codes, const float* scales,
                                                    int64_t elems_per_rank, int32_t block,
                                                    int32_t bits, zpp_topology topo,
                                                    zpp_local_range range, void* out_codes,
                                                    float* out_scales, cudaStream_t stream);
ZPP_API zpp_status zpp_dequant_reduce_scaled_range(const void* codes, const float* scales,
                                                   int64_t elems_per_rank, int32_t block,
                                                   int32_t bits, zpp_topology topo,
                                                   zpp_local_range range, float post_scale,
                                                   void* out, zpp_dtype out_dt,
                                                   cudaStream_t stream);

/*
 * The three qgZ steps as one real rank runs them, on its own buffers, with the two
 * all-to-all exchanges between them left to the caller's collectives ([ZeRO++ summary]
 * Approach: 2-hop all-to-all; the virtual-layout calls above run the same kernels with the
 * exchanges as index maps). For rank r = n*M + l of topology {N, M}, W = N*M, S = E/W,
 * C = N*S:
 *
 * zpp_qgz_reorder_quant_local -- step 1 on this rank's E gradient elements: exactly row r
 *   of what zpp_qgz_reorder_quant writes (the reorder does not depend on r). Chunk l' (C
 *   elements at offset l'*C) of the result is what goes to local peer l' in hop 1; only
 *   the chunks l' in `range` are written ({0, M}: all), so each can be produced just before
 *   its send.
 *   grads : [E] elements of g_dt; codes: out, [zpp_code_bytes(E, bits)]; scales: out, [E/block]
 *   Rules as for zpp_qgz_reorder_quant_range.
 *
 * zpp_dequant_reduce_requant_local -- the fused intra-node hop on the chunks this rank
 *   received: chunk l of each of its node's M ranks, in local-index order, `sources` = M
 *   chunks of `chunk` = C elements back to back. Writes exactly row r of what
 *   zpp_dequant_reduce_requant writes.
 *   codes : [sources][zpp_code_bytes(chunk, bits)]; scales: [sources][chunk/block]
 *   out_codes : out, [zpp_code_bytes(chunk, bits)]; out_scales: out, [chunk/block]
 *
 * zpp_dequant_reduce_local -- the final inter-node hop on the slices this rank received:
 *   slice n of the hop-1 output of ranks (n', l), n' = 0..N-1 ascending, `sources` = N
 *   slices of `slice` = S elements back to back. Writes exactly row r of what
 *   zpp_dequant_reduce_scaled writes (post_scale 1 and fp32 out: zpp_dequant_reduce).
 *   codes : [sources][zpp_code_bytes(slice, bits)]; scales: [sources][slice/block]
 *   out   : out, [slice] elements of out_dt; post_scale: finite
 *
 * For the last two: block a power of two in [64, 4096], bits 4 or 8, 1 <= sources <= 65535,
 * chunk (slice) a multiple of block below 2^31 (0: ZPP_OK, nothing launched), else
 * ZPP_ERR_INVALID_ARG. Alignment and ownership as for every call.
 */
ZPP_API zpp_status zpp_qgz_reorder_quant_local(const void* grads, zpp_dtype g_dt,
                                               int64_t elems_per_rank, int32_t block, int32_t bits,
                                               zpp_topology topo, zpp_local_range range,
                                               void* codes, float* scales, cudaStream_t stream);
ZPP_API zpp_status zpp_dequant_reduce_requant_local(const void* codes, const float* scales,
                                                    int64_t chunk, int32_t block, int32_t bits,
                                                    int32_t sources, void* out_codes,
                                                    float* out_scales, cudaStream_t stream);
ZPP_API zpp_status zpp_dequant_reduce_local(const void* codes, const float* scales, int64_t slice,
                                            int32_t block, int32_t bits, int32_t sources,
                                            float post_scale, void* out, zpp_dtype out_dt,
                                            cudaStream_t stream);

/*
 * The optimiser step and the product with quantised weights: what happens to a weight on
 * either side of the collectives (no counterpart in the pages, which take both from the
 * training framework around them). The three calls below obey the conventions above; every
 * sum, state and norm is fp32 or wider inside.
 */

/* Global gradient norm and clip factor over a list of tensors, on the device:
 *   norm = |pre_scale| * sqrt(sum over all tensors and elements of g^2)
 *   coef = pre_scale * (norm > max_norm ? max_norm / norm : 1)
 * coef is what zpp_adamw_step takes as grad_scale, so a step needs no host round trip.
 * When the norm is not finite (an element is Inf or NaN, or the sum of squares leaves fp32's
 * range) coef is NaN, which makes zpp_adamw_step skip the step.
 *   grads       : HOST array [num_tensors] of device pointers, 16-byte aligned, each to
 *                 sizes[t] contiguous elements of g_dt (ZPP_F16, ZPP_BF16 or ZPP_F32)
 *   sizes       : HOST array [num_tensors], 0 allowed (its pointer is then not read); the
 *                 sum at most ZPP_MAX_ELEMS. Read during the call only, as grads.
 *   num_tensors : 0 .. ZPP_MAX_TENSORS (0: norm 0)
 *   pre_scale   : finite (e.g. 1 / loss scale); max_norm: > 0, +Inf for no clipping
 *   workspace   : device floats, at least zpp_grad_norm_workspace(sum of sizes, num_tensors);
 *                 not shared with another stream's call in flight
 *   out         : device, out[0] = norm, out[1] = coef
 * The sums run in a fixed order (no atomics): the same input gives the same bits.
 */
ZPP_API zpp_status zpp_grad_norm(const void* const* grads, const int64_t* sizes,
                                 int32_t num_tensors, zpp_dtype g_dt, float pre_scale,
                                 float max_norm, float* workspace, float* out,
                                 cudaStream_t stream);

/* Floats of workspace for zpp_grad_norm; -1 on a negative argument. */
ZPP_API int64_t zpp_grad_norm_workspace(int64_t total_elems, int32_t num_tensors);

/* One tensor of an AdamW step; all pointers are device pointers. */
typedef struct zpp_adamw_tensor {
  float* param;            /* [n] fp32 master weights, updated */
  const void* grad;        /* [n] of g_dt */
  void* exp_avg;           /* m: [n] fp32, or [n] e4m3 codes with state_bits 8; updated */
  void* exp_avg_sq;        /* v: [n] fp32, or [n] e4m3 codes of sqrt(v); updated */
  float* exp_avg_scale;    /* state_bits 8: [ceil(n / ZPP_STATE_BLOCK)], updated; else unused */
  float* exp_avg_sq_scale; /* as above, for sqrt(v) */
  void* weight;            /* out, NULL or [n] of w_dt: the updated weights rounded */
  int64_t n;               /* elements, 0 allowed (the pointers are then not read) */
} zpp_adamw_tensor;

typedef struct zpp_adamw_params {
  double lr, beta1, beta2, eps, weight_decay;
  int64_t step;  /* 1 for the first step (bias correction) */
  uint32_t seed; /* state_bits 8: seeds the stochastic rounding */
} zpp_adamw_params;

#define ZPP_STATE_BLOCK 256 /* elements per fp8 state scale */

/*
 * One AdamW step (decoupled weight decay) over a list of tensors. With c = *grad_scale (1
 * when NULL) and t = step, per element:
 *   g = c * grad;  m = beta1 m + (1 - beta1) g;  v = beta2 v + (1 - beta2) g^2
 *   param = param (1 - lr weight_decay)
 *           - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 *   weight = param rounded to nearest even into w_dt (the shard zpp_quant_blockwise reads)
 * If c is not finite the whole step is skipped: nothing is written.
 *
 * state_bits 8: m and r = sqrt(v) are held as e4m3 codes with one fp32 scale per
 * ZPP_STATE_BLOCK consecutive elements of a tensor (the last block may be shorter; amax over
 * its finite values),
 *   scale = amax * fl(1/448), inv = 448 * fl(1/amax), value = code * scale
 *   (inv not finite: scale 0, codes 0)
 * The step itself uses the unrounded m and v. Rounding is stochastic: with x = value * inv and
 * h the e4m3 spacing at |x|, the code is floor(|x| / h + u) h with u = (k + 1/2) / 65536, k 16
 * bits of a hash of (seed, step, element number): the low ones for m, the high ones for r. So a
 * running average moves in expectation even where its change is far below h (round to
 * nearest would freeze it), and equal inputs give equal bits. r > 0 keeps at least the
 * smallest code, so a denominator never collapses. Element numbers count blocks through the
 * list: tensor t's element i has ZPP_STATE_BLOCK * (blocks of tensors 0..t-1) + i. An Inf or NaN
 * gradient, or one whose square overflows, makes its own element NaN, no other's. A v below
 * 2^-126 (|grad| below some 1e-18) may count as smaller than it is.
 *   hash: all mod 2^32, key = (seed * 0x9E3779B9) ^ (step * 0x510E527F), i split in lo, hi:
 *     x = lo * 0x9E3779B9 + hi * 0xA54FF53B + key;  x = (x ^ x >> 16) * 0xBB67AE85 + key
 *     x = (x ^ x >> 15) * 0x9B05688D;               bits = x ^ x >> 16
 *
 *   tensors     : HOST array [num_tensors], read during the call only; the n sum to at most
 *                 ZPP_MAX_ELEMS; param, grad, exp_avg, exp_avg_sq, weight 16-byte aligned
 *   num_tensors : 0 .. ZPP_MAX_TENSORS
 *   g_dt        : ZPP_F16, ZPP_BF16 or ZPP_F32; w_dt: ZPP_F16 or ZPP_BF16 (ZPP_F32 with a
 *                 non-NULL weight: ZPP_ERR_UNSUPPORTED)
 *   state_bits  : 32 or 8
 *   hp          : HOST, read during the call: lr and weight_decay finite, 0 <= beta1, beta2 < 1,
 *                 eps >= 0 and finite (one below 2^-126 counts as 2^-126; with 0 an element that
 *                 never had a gradient is 0 / 0), step >= 1
 *   grad_scale  : device, 4-byte aligned, or NULL
 */
ZPP_API zpp_status zpp_adamw_step(const zpp_adamw_tensor* tensors, int32_t num_tensors,
                                  zpp_dtype g_dt, zpp_dtype w_dt, int32_t state_bits,
                                  const zpp_adamw_params* hp, const float* grad_scale,
                                  cudaStream_t stream);

/* A run's step count on the device, 16-byte aligned. The caller sets `step` (0 for a new run) and
 * zeroes the rest, which zpp_adamw_step_counted keeps: the factors of the step in hand, and
 * beta^step, so that the next step's power is one product. */
typedef struct zpp_adamw_record {
  int64_t step; /* number of the last step that was taken */
  int64_t reserved;
  float factor, step_size, inv_root_bc2;
  uint32_t key;
  double beta[2], power[2]; /* power[k] = beta[k]^step, for beta1 and beta2 */
} zpp_adamw_record;

/* Clipping by the norm of the step's own gradients, as zpp_grad_norm. */
typedef struct zpp_adamw_clip {
  float pre_scale, max_norm;
  float* workspace; /* zpp_grad_norm_workspace(sum of n, num_tensors) floats */
  float* out;       /* (norm, factor) */
} zpp_adamw_clip;

/*
 * zpp_adamw_step, counted: a step that a non-finite factor skips has no number, so bias
 * corrections and rounding bits go on from the last step that was taken. Nobody on the host
 * needs to know which ones were, and a captured step is the next one each time it is replayed.
 *   hp->step    : 0: this step is number record->step + 1, read in the stream's order; >= 1: its
 *                 number, where the caller knows it
 *   grad_scale  : as above; clip: NULL, or the factor comes from the norm of the gradients, left
 *                 in clip->out (HOST struct, read during the call; then grad_scale is NULL)
 *   record      : device; afterwards record->step is this step's number, or one less if it was
 *                 skipped (a list without elements counts too)
 * Every argument is checked before the first launch. The rest as zpp_adamw_step.
 */
ZPP_API zpp_status zpp_adamw_step_counted(const zpp_adamw_tensor* tensors, int32_t num_tensors,
                                          zpp_dtype g_dt, zpp_dtype w_dt, int32_t state_bits,
                                          const zpp_adamw_params* hp, const float* grad_scale,
                                          const zpp_adamw_clip* clip, zpp_adamw_record* record,
                                          cudaStream_t stream);

/*
 * y = x W^T (+ bias) for a few vectors x, straight from the codes of a [rows][cols] matrix
 * quantised row-major by zpp_quant_blockwise (blocks may run across rows):
 *   y[j][r] = sum_c q[r][c] * scales[(r * cols + c) / block] * x[j][c]  (+ bias[r])
 * Products and sums are fp32 (code times x is exact), y is rounded once. A scale multiplies the sum
 * of its block's products, or of a part of them: an infinite one gives infinity of that sum's sign,
 * or NaN where the sum is 0.
 *   codes, scales : as zpp_quant_blockwise writes them for n = rows * cols <= ZPP_MAX_ELEMS
 *   rows, cols    : 0 <= rows < 2^31, 1 <= cols < 2^31; block, bits as in zpp_quant_blockwise
 *   x             : [vecs] rows of cols elements of x_dt (ZPP_F16 or ZPP_BF16; ZPP_F32 ->
 *                   ZPP_ERR_UNSUPPORTED), row j at x + j * x_stride, x_stride >= cols
 *   vecs          : 0 .. 65535. Meant for a handful (decoding): the codes are read once for 16 vectors,
 *                   so for many vectors dequantise and use a matrix product
 *   bias          : NULL or [rows] of x_dt
 *   y             : out, row j at y + j * y_stride, y_stride >= rows, of y_dt (any zpp_dtype)
 * x and y must be 16-byte aligned, bias 2-byte; the strides (in elements) may be any.
 */
ZPP_API zpp_status zpp_matvec_blockwise(const void* codes, const float* scales, int64_t rows,
                                        int64_t cols, int32_t block, int32_t bits, const void* x,
                                        zpp_dtype x_dt, int64_t vecs, int64_t x_stride,
                                        const void* bias, void* y, zpp_dtype y_dt,
                                        int64_t y_stride, cudaStream_t stream);

/*
 * Matrices of e4m3 codes with a scale per block, and their products: the arithmetic of a linear layer
 * that trains or answers in 8 bits (no counterpart in the pages). value = code * scale.
 */
#define ZPP_FP8_BLOCK 128 /* columns that share a scale */

/* A matrix of codes, row-major; all pointers are device pointers. */
typedef struct zpp_fp8_matrix {
  void* codes;         /* 16-byte aligned; row r at codes + r * stride */
  float* scales;       /* of element (r, c): scales[(r / tile) * scale_row + (c / 128) * scale_block] */
  int64_t rows, cols;  /* 0 <= rows < 2^31, 1 <= cols < 2^31, rows * cols <= ZPP_MAX_ELEMS */
  int64_t stride;      /* bytes between rows: a multiple of 16, cols <= stride <= ZPP_MAX_ELEMS */
  int64_t scale_row, scale_block; /* >= 0, at most ZPP_MAX_ELEMS */
  int32_t tile;        /* rows that share a scale: 1 or 128 */
} zpp_fp8_matrix;

/*
 * A matrix to codes, and its transpose with it: a backward pass multiplies along the other index.
 * Per block (128 columns of `tile` rows; those at the edges are smaller), amax over finite values:
 *   scale = the smallest 2^e, e >= -126, with amax <= 448 * 2^e  (amax 0: scale 0, codes 0)
 *   code  = x / scale rounded to nearest even (exact but for that: the scale is a power of two)
 * An infinite or NaN value has the code NaN (0x7f or 0xff).
 *   x            : [rows][cols] of x_dt (any zpp_dtype), row r at x + r * x_stride elements,
 *                  cols <= x_stride <= ZPP_MAX_ELEMS, aligned to its elements
 *   out          : HOST struct, read during the call; bytes between cols and stride are left as they were
 *   transposed   : HOST struct or NULL; rows and cols are out's cols and rows, tile is out's. With tile 1
 *                  its blocks are 128 rows of a column of x. With tile 128 a tile's scale is also that
 *                  of its transpose: scales is not written (read out's with the strides exchanged).
 */
ZPP_API zpp_status zpp_quant_fp8(const void* x, zpp_dtype x_dt, int64_t x_stride,
                                 const zpp_fp8_matrix* out, const zpp_fp8_matrix* transposed,
                                 cudaStream_t stream);

/*
 * y = a b^T (+ bias): y[m][n] = sum_k a[m][k] b[n][k] (+ bias[n]) of the values that the codes stand
 * for. Sums are fp32: of the codes within a block of 128, then of the blocks times both scales, in
 * ascending order; y is rounded once. Where there are few tiles of y the blocks are taken in up to 8
 * parts, each in ascending order, and the parts added in theirs: as the sizes of the call say, so that
 * the same call gives the same bits, and a row of a may get others beside another number of rows. The product
 * of two scales may be rounded to fp32 first, or that of a block's sum and one of them. NaN codes and non-finite
 * scales give what such values give.
 *   a, b : HOST structs, read during the call; cols is the same in both. One may be the other
 *   bias : NULL or [b.rows] of y_dt
 *   y    : out, [a.rows][b.rows] of y_dt (any zpp_dtype), row m at y + m * y_stride elements,
 *          b.rows <= y_stride <= ZPP_MAX_ELEMS; y and bias are aligned to their elements
 * The products run on the tensor cores (waits inside: see zpp_device_fault). The call takes its
 * kernel by the sizes: for few rows of a it is bound by reading b.
 */
ZPP_API zpp_status zpp_matmul_fp8(const zpp_fp8_matrix* a, const zpp_fp8_matrix* b, const void* bias,
                                  void* y, zpp_dtype y_dt, int64_t y_stride, cudaStream_t stream);

/*
 * Updates of matrices whose singular values are made nearly equal (no counterpart in the pages): beside
 * the AdamW step for what is not a matrix.
 *
 * Newton-Schulz steps on a matrix x: X = x / max(|x|, eps), |x| the root of the sum of squares, then
 * for each step k with (a, b, c) = coefficients[k]:
 *   A = X X^T,  B = b A + c A A,  X = a X + B X
 * (for a matrix with more rows than columns the same of its transpose). Every value is held in two fp16
 * (the second one what the first lost), sums and the diagonals of A and B in fp32. After the usual five
 * steps 2e-6 (256 x 1024) to 1e-5 (4096 x 16384) of the result's norm is error, as with fp32 products.
 * Singular values have to stay below 8 through the steps and coefficients below 15 (the usual ones keep to 1.3). Elements
 * whose squares leave fp32's range upwards (above 1.8e19) give NaN; small ones count whatever their squares are.
 */
typedef struct zpp_newton_schulz {
  const double* coefficients; /* HOST [steps][3], finite */
  int32_t steps;              /* 1 .. 100 */
  double eps;                 /* > 0, finite; one below 2^-126 counts as 2^-126 */
} zpp_newton_schulz;

#define ZPP_MAX_SIDE (((int64_t)1) << 30) /* rows and columns of a matrix below */

typedef struct zpp_matrix {
  const void* x;      /* [rows][cols] of x_dt, device, aligned to its elements */
  void* out;          /* out, [rows][cols] of out_dt; may be x where the types are one */
  int64_t rows, cols; /* 0 .. ZPP_MAX_SIDE, rows * cols <= ZPP_MAX_ELEMS; 0: no pointer is read */
} zpp_matrix;

/*
 * The steps on a list of matrices; those of one shape share each launch's tiles.
 *   list      : HOST array [num], read during the call only; num 0 .. ZPP_MAX_TENSORS
 *   x_dt      : any zpp_dtype; out_dt: ZPP_F16 or ZPP_BF16 (ZPP_F32 -> ZPP_ERR_UNSUPPORTED)
 *   workspace : device, 128-byte aligned, zpp_orthogonalize_workspace(list, num) bytes; not shared with
 *               another stream's call in flight, nor by two captured graphs that may run at once
 */
ZPP_API zpp_status zpp_orthogonalize(const zpp_matrix* list, int32_t num, zpp_dtype x_dt,
                                     zpp_dtype out_dt, const zpp_newton_schulz* ns, void* workspace,
                                     cudaStream_t stream);

/* Bytes of workspace; -1 on sizes that the call refuses. Only sizes are read, no pointers. */
ZPP_API int64_t zpp_orthogonalize_workspace(const zpp_matrix* list, int32_t num);

/* One matrix of a Muon step; all pointers are device pointers, aligned to their elements. */
typedef struct zpp_muon_tensor {
  float* param;       /* [rows][cols] fp32 master weights, updated */
  const void* grad;   /* [rows][cols] of g_dt */
  float* momentum;    /* [rows][cols], updated */
  void* weight;       /* out, NULL or [rows][cols] of w_dt: the updated weights rounded */
  int64_t rows, cols; /* as zpp_matrix */
} zpp_muon_tensor;

typedef struct zpp_muon_params {
  double lr, momentum, weight_decay;
  int32_t nesterov; /* 0 or 1 */
  int32_t adjust;   /* ZPP_MUON_ORIGINAL, ZPP_MUON_MATCH_RMS_ADAMW or ZPP_MUON_NONE */
  zpp_newton_schulz ns;
} zpp_muon_params;

#define ZPP_MUON_ORIGINAL 0        /* adj = sqrt(max(1, rows / cols)) */
#define ZPP_MUON_MATCH_RMS_ADAMW 1 /* adj = 0.2 sqrt(max(rows, cols)) */
#define ZPP_MUON_NONE 2            /* adj = 1 */

/*
 * One Muon step over a list of matrices. With c = *grad_scale (1 when NULL) and mu = momentum:
 *   g = c * grad;  m = mu m + (1 - mu) g;  u = nesterov ? (1 - mu) g + mu m : m
 *   param = param (1 - lr weight_decay) - lr adj X,  X = the Newton-Schulz steps on u
 *   weight = param rounded to nearest even into w_dt
 * If c is not finite the whole step is skipped: nothing is written. (zpp_grad_norm's factor is one.)
 *   tensors   : HOST array [num], read during the call only; num 0 .. ZPP_MAX_TENSORS
 *   g_dt      : any zpp_dtype; w_dt: ZPP_F16 or ZPP_BF16 (ZPP_F32 with a non-NULL weight:
 *               ZPP_ERR_UNSUPPORTED)
 *   hp        : HOST, read during the call: lr and weight_decay finite, 0 <= momentum < 1
 *   grad_scale: device, 4-byte aligned, or NULL
 *   workspace : as zpp_orthogonalize's, zpp_muon_workspace(tensors, num) bytes
 */
ZPP_API zpp_status zpp_muon_step(const zpp_muon_tensor* tensors, int32_t num, zpp_dtype g_dt,
                                 zpp_dtype w_dt, const zpp_muon_params* hp, const float* grad_scale,
                                 void* workspace, cudaStream_t stream);
ZPP_API int64_t zpp_muon_workspace(const zpp_muon_tensor* tensors, int32_t num);

/* Bytes of packed codes for n elements: n for INT8, ceil(n/2) for INT4; -1 on bad bits. */
ZPP_API int64_t zpp_code_bytes(int64_t n, int32_t bits);

/* Number of scales for n elements: ceil(n / block); -1 on a bad block. */
ZPP_API int64_t zpp_num_scales(int64_t n, int32_t block);

/* Static, never-NULL description of a status code. */
ZPP_API const char* zpp_status_string(zpp_status status);

/*
 * Fault word of the current device (no counterpart in the pages). Kernels that wait for
 * data in flight (the INT8 fused-hop kernel waits on shared-memory barriers completed by
 * bulk copies) bound every wait to about a second; a wait that runs out sets a bit here,
 * the kernel still ends, and its outputs are unspecified. Bits: 1 and 2 -- a wait of the
 * INT8 fused hop ran out; 4 -- zpp_wait_selftest ran out (as it always does); 8 -- a wait of
 * zpp_matmul_fp8; 16 -- a wait of zpp_orthogonalize or zpp_muon_step.
 *   flags : out, the word (0 when nothing ran out since the last clear)
 *   clear : nonzero -> zero the word after reading it
 * Unlike the other calls this one synchronises with the device (it copies the word back);
 * call it after the work it should cover has been synchronised.
 */
ZPP_API zpp_status zpp_device_fault(uint32_t* flags, int32_t clear);

/*
 * Diagnostic (no counterpart in the pages): launches one warp that waits on a
 * shared-memory barrier nothing completes, bounded by limit_ns nanoseconds (1 ns .. 10 s,
 * else ZPP_ERR_INVALID_ARG), then sets bit 4 of the fault word and ends. It exercises the
 * bounded wait and the fault report on the device without a fault of any kind.
 */
ZPP_API zpp_status zpp_wait_selftest(uint64_t limit_ns, cudaStream_t stream);

/*
 * Measurement helper (no counterpart in the pages): a 256-bit streaming device copy
 * used as the same-run HBM reference next to the kernels above.
 *   src, dst : 32-byte aligned device buffers; bytes: a multiple of 32.
 */
ZPP_API zpp_status zpp_device_copy(const void* src, void* dst, int64_t bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ZPP_H */
