/*
 * qlinear.h -- C ABI of the group-wise affine W4 g64 quantized linear layer (sm_100a),
 * with its W8 g64 variant (qlinear8_*, at the end).
 *
 * The packed format (aimarketly "Ideogram-4-IQ4_M", intro: one f16 scale and one
 * f16 bias per 64 weights on top of 4-bit codes, 4.5 bits per weight;
 * huggingface "SceneWorks/ideogram-4-mlx", Versions: group-wise affine, group
 * size 64) and its uniform affine grid w = scale * q + bias (aimarketly
 * "Ideogram-4-IQ4_M", "What IQ4 means here").
 *
 * Layout of every tensor (all row-major, dense, no padding):
 *   x       bf16     [M][K]      activations
 *   codes   uint32   [N][K/8]    code (n, k) = (codes[n][k/8] >> 4*(k%8)) & 0xF, low nibble first
 *   scales  f16      [N][K/64]   group scale  s(n, k/64)
 *   biases  f16      [N][K/64]   group bias   b(n, k/64)
 *   y       bf16     [M][N]      y[m][n] = sum_k x[m][k] * (s * q(n, k) + b)
 * W is logically [N][K] (a PyTorch Linear weight): y = x . W^T.
 *
 * Conventions shared by every entry point:
 *   - Ownership: the caller owns every buffer.  Tensor arguments are DEVICE
 *     pointers on the current CUDA device.  The library allocates no device
 *     memory; scratch comes from the caller's workspace.
 *   - Asynchrony: work is enqueued on `stream` (0 = legacy default stream).
 *     QL_OK means "validated and launched"; launch failures return QL_ERR_CUDA.
 *     Faults detected inside kernels (non-finite pack input, a bounded wait that
 *     expired) are recorded in a per-device status word read by
 *     qlinear_get_device_status().
 *   - Validation happens before any launch; on any error nothing is launched.
 *     Required: group == 64 (else QL_ERR_UNSUPPORTED); K % 64 == 0, N % 8 == 0,
 *     M >= 1, K >= 64, N >= 8, non-null tensors (else QL_ERR_INVALID_ARG); every
 *     pointer 16-byte aligned (else QL_ERR_ALIGNMENT); outputs must not overlap
 *     inputs (else QL_ERR_INVALID_ARG).
 *   - Non-finite activations or parameters propagate through the arithmetic
 *     IEEE-style.
 *   - Thread safety: calls are reentrant; the last-dispatch record is
 *     thread-local.
 */
#ifndef QLINEAR_H
#define QLINEAR_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#if defined(__GNUC__)
#define QL_API __attribute__((visibility("default")))
#else
#define QL_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    QL_OK = 0,
    QL_ERR_INVALID_ARG = 1,     /* bad size, null pointer, overlap, non-finite pack input */
    QL_ERR_ALIGNMENT = 2,       /* a pointer is not 16-byte aligned */
    QL_ERR_UNSUPPORTED = 3,     /* group != 64, or a feature not built (see each call) */
    QL_ERR_WORKSPACE = 4,       /* workspace missing or smaller than qlinear_workspace_size() */
    QL_ERR_CUDA = 5,            /* a CUDA runtime call or kernel launch failed */
    QL_ERR_DEVICE_TIMEOUT = 6,  /* a bounded wait inside a kernel expired; the kernel returned early */
    QL_ERR_BOUNDS = 7           /* a kernel's own index check failed (debug builds) */
} ql_status;

typedef enum { QL_F32 = 0, QL_BF16 = 1 } ql_dtype;

/* Kernel paths of qlinear_forward, for qlinear_forward_config() and qlinear_last_dispatch(). */
typedef enum {
    QL_PATH_AUTO = 0,       /* per-shape choice of the dispatcher */
    QL_PATH_GEMV = 1,       /* CUDA-core split-K weight streaming (any M; meant for M <= 4) */
    QL_PATH_TC_SKINNY = 2,  /* tcgen05 weight streaming for small M: stream-K over K, fp32 partials
                               reduced in a fixed order; the dispatcher uses it for M <= 32, forced it
                               runs M <= 64 (QL_ERR_UNSUPPORTED above) */
    QL_PATH_TC_FUSED = 3    /* tcgen05 fused-dequant GEMM for large M */
    /* Both tcgen05 paths multiply f16 operands with fp32 accumulation in tensor memory: each
     * weight is rounded once, RN_f16(s * q + b), and each activation row is scaled by a power of
     * two into f16 (exact for entries above 2^-28 of the row's largest magnitude) and scaled back
     * after the accumulation.  QL_PATH_GEMV multiplies the exact codes in fp32. */
} ql_path;

/*
 * Bytes of device workspace qlinear_forward() needs for this shape (0 is
 * possible).  Returns (size_t)-1 when the shape is invalid.
 */
QL_API size_t qlinear_workspace_size(int64_t M, int64_t K, int64_t N, int32_t group);

/*
 * y = x . W^T for the packed W (the layer the pages describe: bf16
 * activations, fp32 accumulation, bf16 output).  Preconditions and errors as in
 * the conventions above; additionally `workspace` must hold at least
 * qlinear_workspace_size(M, K, N, group) bytes (QL_ERR_WORKSPACE otherwise)
 * and must not overlap any tensor.  The dispatcher picks the kernel path from
 * (M, K, N); qlinear_last_dispatch() reports the choice.
 */
QL_API ql_status qlinear_forward(const void* x, const uint32_t* codes, const void* scales,
                          const void* biases, void* y, int64_t M, int64_t K, int64_t N,
                          int32_t group, void* workspace, size_t workspace_bytes,
                          cudaStream_t stream);

/*
 * qlinear_forward with the path and split-K factor forced (testing and tuning).
 * path: a ql_path; split_k: 0 = the dispatcher's choice, else the number of K
 * slices, 1 <= split_k <= K/64 (and <= 1024 on the fused path; QL_ERR_INVALID_ARG otherwise); slice z covers the
 * groups [z*G/split_k, (z+1)*G/split_k), G = K/64.
 * out_dtype: QL_BF16 = the layer's output; QL_F32 writes y as fp32 [M][N]
 * (the same arithmetic without the final rounding, for numerical tests).
 * Split-K: QL_PATH_GEMV and QL_PATH_TC_FUSED take split_k > 1 (the fused path then writes one fp32
 * partial per slice into the workspace and sums them in slice order, for shapes with fewer output
 * tiles than SMs); QL_PATH_TC_SKINNY balances K itself and returns QL_ERR_UNSUPPORTED for it.
 * A path that cannot run the shape returns QL_ERR_UNSUPPORTED.
 */
QL_API ql_status qlinear_forward_config(const void* x, const uint32_t* codes, const void* scales,
                                 const void* biases, void* y, ql_dtype out_dtype,
                                 int64_t M, int64_t K, int64_t N, int32_t group,
                                 int32_t path, int32_t split_k,
                                 void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Workspace bytes for qlinear_forward_config() with the same path and split_k. */
QL_API size_t qlinear_workspace_size_config(int64_t M, int64_t K, int64_t N, int32_t group,
                                     int32_t path, int32_t split_k);

/*
 * Standalone dequantization: out[n][k] = RN_fp32(s * q + b), rounded once more
 * to bf16 (nearest even) when out_dtype == QL_BF16.  Bit-exact by definition:
 * s*q + b is formed with one fused multiply-add.  out is [N][K] of out_dtype.
 */
QL_API ql_status qlinear_dequant(const uint32_t* codes, const void* scales, const void* biases,
                          int64_t K, int64_t N, int32_t group, void* out, ql_dtype out_dtype,
                          cudaStream_t stream);

/*
 * Quantize fp32 w [N][K] into codes/scales/biases.
 * imatrix == NULL: min/max round-to-nearest (MLX's own solution, candidate 0
 * of the search in aimarketly "Ideogram-4-IQ4_M", "What IQ4 means here"):
 * per group of 64, s = RN32(RN32(max-min)/15), scale = RN_f16(s),
 * bias = RN_f16(min), q = clamp(rint(RN32(RN32(w-bias)/scale)), 0, 15)
 * (ties to even), q = 0 when scale == 0.  Deterministic: equal inputs give
 * equal bytes.
 * imatrix != NULL: importance-weighted fit.  imatrix is fp32 [K], the per-channel
 * E[x^2] of the layer's activations (device memory, read only).  Per group the
 * candidates are the RTN triple, then 80 range shrinks (lo = min + a r,
 * hi = max - c r, a, c in {0, 0.025, ..., 0.2}), each refined by up to two
 * weighted least-squares refits of (scale, bias) with the codes fixed; the
 * triple with the lowest sum_j imp_j (w_j - RN32(s q_j + b))^2 (float64,
 * imp = imatrix + 1e-6 * mean(imatrix)) wins, ties to the earliest, so the fit
 * is never worse than RTN on that objective.  Deterministic: every float64 sum
 * is taken in index order with correctly rounded operations.  A negative or
 * non-finite imatrix entry is an argument error reported through the device
 * status word (all groups written as zeros).
 * A group holding a non-finite value or |w| > 65504 is written as codes 0,
 * scale 0, bias 0, and the device status word records QL_ERR_INVALID_ARG.
 */
QL_API ql_status qlinear_pack(const float* w, const float* imatrix, int64_t K, int64_t N, int32_t group,
                       uint32_t* codes, void* scales, void* biases, cudaStream_t stream);

/*
 * Synchronizes `stream`, then reads and clears the current device's status word
 * (the first error a kernel recorded since the last read).  Returns QL_OK when
 * no kernel recorded anything, QL_ERR_CUDA if the synchronization fails.
 */
QL_API ql_status qlinear_get_device_status(cudaStream_t stream);

/*
 * Writes a NUL-terminated description of the calling thread's last
 * qlinear_forward dispatch, e.g. "path=tc_fused bits=4 tile=256w x 192t x 64k stages=x5/c2x4/a2
 * ctas=148 splitk=1 launches=3 why=auto:M>64,split:9x72" (stages: activation, code x K-steps per
 * code stage, tensor-memory weight stages; launches = kernels that call enqueued; why = the rule or
 * the caller's forced path behind the choice),
 * truncated to len bytes.  QL_ERR_INVALID_ARG if buf is NULL or len == 0.
 */
QL_API ql_status qlinear_last_dispatch(char* buf, size_t len);

/*
 * Test hook of the checked build (libqlinear_bounds.so, compiled with QL_BOUNDS_CHECK); the pages have no
 * counterpart.  kernel_mask bit 0 holds back the code producer of the fused tensor-core kernel
 * (QL_PATH_TC_FUSED), bit 1 that of the weight-streaming kernel (QL_PATH_TC_SKINNY): they issue no code
 * or parameter load; bit 2 the row copies of qlinear_norm_residual's ring (D > 512 and more than two rows per
 * SM); bit 3 the copies of the kernel in front of QL_PATH_TC_FUSED that does the adapters' first product.  The
 * kernel's other roles then wait until the limit, record QL_ERR_DEVICE_TIMEOUT and
 * unwind (nothing of theirs in flight, tensor memory freed).  wait_limit_ns replaces the one-second
 * limit of every bounded wait in the library's kernels (> 0); call with kernel_mask 0 and 1000000000
 * to restore the defaults.  Synchronous (two small host-to-device copies on the legacy stream).
 * The shipped library returns QL_ERR_UNSUPPORTED and changes nothing; QL_ERR_INVALID_ARG for an
 * unknown bit or a zero limit.
 */
QL_API ql_status qlinear_test_stall(int32_t kernel_mask, uint64_t wait_limit_ns);

/*
 * Test hook of the checked build (libqlinear_bounds.so); the pages have no counterpart.  Selects the ring
 * depths of the fused tensor-core kernel that later 4-bit, bf16-output, unsplit qlinear_forward calls
 * (QL_PATH_TC_FUSED or the dispatcher's choice of it) launch on this process: variant 0 is the shipped
 * configuration, variants 1 .. QL_TEST_RING_VARIANTS-1 other (activation stages, code stages, epilogue
 * staging blocks per warp) triples.  Every ring position is a function of the step count alone, so the
 * output must be the same bytes for every variant.  The shipped library returns QL_ERR_UNSUPPORTED;
 * QL_ERR_INVALID_ARG for a variant out of range; QL_ERR_CUDA if the variant's shared-memory size
 * cannot be set on the current device.
 */
#define QL_TEST_RING_VARIANTS 7
QL_API ql_status qlinear_test_ring_depth(int32_t variant);

/*
 * Test hook of the checked build (libqlinear_bounds.so); the pages have no counterpart.  Holds back the
 * roles of the tensor-core kernels in role_mask at their start, each CTA's and warp's by a different part
 * (0/7 .. 7/7) of max_ns, so that every hand-off between roles (TMA rings, tensor-memory stages,
 * accumulators, partials) meets other orders of arrival; the output must not change.  Bits: 1 the
 * activation producer, 2 the code producer, 4 the dequantizers, 8 the MMA issuers, 16 the epilogue or
 * drain warps; in the adapters' first product above 64 rows 1 the conversion, 2 the tiles' adapter lists, 8 the
 * product; in the norms' ring 1 the row copies, 16 the warps.  role_mask 0 turns it off.  Synchronous (two
 * small host-to-device copies on the legacy stream).  The shipped library returns QL_ERR_UNSUPPORTED;
 * QL_ERR_INVALID_ARG for an unknown bit or max_ns above 1 ms.
 */
QL_API ql_status qlinear_test_delay(int32_t role_mask, uint64_t max_ns);

/*
 * Test hook of the checked build (libqlinear_bounds.so); the pages have no counterpart.  Takes the last `cut` elements off
 * every extent that a kernel checks an index against, so that right accesses of them are recorded as QL_ERR_BOUNDS and
 * skipped: which arrays' accesses are checked can be tested without a wrong one.  0 turns it off.  Synchronous (a small
 * host-to-device copy on the legacy stream).  The shipped library returns QL_ERR_UNSUPPORTED; QL_ERR_INVALID_ARG for a
 * negative cut.
 */
QL_API ql_status qlinear_test_extent(int64_t cut);

/*
 * Allocation-free forward for small M.  The pages have no counterpart of this
 * call; it exists for callers that cannot allocate device memory where they
 * run the layer (a plugin living inside another engine's fixed memory pool, a
 * serving loop that must not allocate after start-up, a runtime that passes
 * only inputs and outputs and no workspace).
 *
 * Same arithmetic and arguments as qlinear_forward (bf16 y), restricted to
 * M <= QL_NOALLOC_MAX_M (QL_ERR_UNSUPPORTED above), and it allocates nothing:
 * its split-K partials live in a fixed scratch array of
 * QL_NOALLOC_SCRATCH_BYTES compiled into the library, which every GPU that
 * loads the library holds until the process exits.  A shape whose partials
 * would not fit returns QL_ERR_WORKSPACE.  The first call on a device looks up
 * that device's address of the array (cudaGetSymbolAddress with the device
 * current), so make the first call on each device before any stream capture.
 * All calls share the one array and it keeps the last call's contents: calls
 * that overlap on the GPU (other streams or host threads) race and must be
 * serialized by the caller.  No cudaMalloc, cudaFree or allocating library
 * routine is called.  The cached address is that of the context current at
 * the first call: do not use this entry point across cudaDeviceReset.  A
 * launch error already pending on the calling thread when the call is made
 * returns QL_ERR_CUDA before anything is launched and is left pending.
 * It runs the CUDA-core split-K path (QL_PATH_GEMV), whose cost grows with M
 * (each 4-row block of activations streams the weights again).
 */
#define QL_NOALLOC_SCRATCH_BYTES (4u << 20)
#define QL_NOALLOC_MAX_M 64
QL_API ql_status qlinear_forward_noalloc(const void* x, const uint32_t* codes, const void* scales,
                                         const void* biases, void* y, int64_t M, int64_t K, int64_t N,
                                         int32_t group, cudaStream_t stream);

/*
 * Measurement hook.  While set (both non-NULL), every qlinear_forward* call
 * made by the calling thread records `start` on its stream immediately before
 * its main kernel (the tensor-core GEMM or the weight-streaming kernel) and
 * `stop` immediately after it, so the main kernel can be timed alone.  The
 * caller owns both events; NULL, NULL turns the hook off.  Thread-local.
 */
QL_API ql_status qlinear_set_profile_events(cudaEvent_t start, cudaEvent_t stop);

/*
 * W8 g64: the 8-bit variant of the same format.  The pages ship an 8-bit pack beside the 4-bit one
 * (huggingface "SceneWorks/ideogram-4-mlx", Versions: Q8) and keep the modulation and conditioning
 * projections at 8 bits (aimarketly "Ideogram-4-IQ4_M", Conversion); the scale and bias stay one f16
 * pair per 64 weights, so a weight costs 8.5 bits.
 *
 *   codes   uint32   [N][K/4]    code (n, k) = (codes[n][k/4] >> 8*(k%4)) & 0xFF, low byte first
 *   scales, biases, x, y          as for the 4-bit calls; w = s * q + b with q in [0, 255]
 *
 * Each qlinear8_* call has the arguments, preconditions, errors and arithmetic of the 4-bit call of
 * the same name, with the code tensor above in place of the 4-bit one:
 *   qlinear8_forward / _config   y = x . W^T; the same kernel paths (QL_PATH_GEMV multiplies exact
 *                                codes in fp32; both tcgen05 paths multiply RN_f16(s * q + b) by f16
 *                                activations scaled per row by a power of two, fp32 accumulation)
 *   qlinear8_workspace_size[_config]
 *   qlinear8_dequant             out = RN_fp32(s * q + b) (bf16: rounded once more), bit-exact
 *   qlinear8_pack                min/max round-to-nearest with 255 levels:
 *                                s = RN32(RN32(max-min)/255), scale = RN_f16(s), bias = RN_f16(min),
 *                                q = clamp(rint(RN32(RN32(w-bias)/scale)), 0, 255) (ties to even),
 *                                q = 0 when scale == 0; imatrix must be NULL (QL_ERR_UNSUPPORTED
 *                                otherwise: the importance-weighted fit is built for 4-bit codes)
 */
QL_API size_t qlinear8_workspace_size(int64_t M, int64_t K, int64_t N, int32_t group);
QL_API size_t qlinear8_workspace_size_config(int64_t M, int64_t K, int64_t N, int32_t group,
                                             int32_t path, int32_t split_k);
QL_API ql_status qlinear8_forward(const void* x, const uint32_t* codes, const void* scales,
                                  const void* biases, void* y, int64_t M, int64_t K, int64_t N,
                                  int32_t group, void* workspace, size_t workspace_bytes,
                                  cudaStream_t stream);
QL_API ql_status qlinear8_forward_config(const void* x, const uint32_t* codes, const void* scales,
                                         const void* biases, void* y, ql_dtype out_dtype,
                                         int64_t M, int64_t K, int64_t N, int32_t group,
                                         int32_t path, int32_t split_k,
                                         void* workspace, size_t workspace_bytes, cudaStream_t stream);
QL_API ql_status qlinear8_dequant(const uint32_t* codes, const void* scales, const void* biases,
                                  int64_t K, int64_t N, int32_t group, void* out, ql_dtype out_dtype,
                                  cudaStream_t stream);
QL_API ql_status qlinear8_pack(const float* w, const float* imatrix, int64_t K, int64_t N, int32_t group,
                               uint32_t* codes, void* scales, void* biases, cudaStream_t stream);

/*
 * SwiGLU up/gate pair in one call: h = silu(x . W_gate^T) * (x . W_up^T) elementwise, with
 * silu(z) = z / (1 + e^-z) (the DiT block's MLP is a SwiGLU of three Linears, jimmysue "Ideogram 4"
 * notes, sec. 2.1 and 2.8; this call covers the first two and the gating, the third is an ordinary
 * qlinear_forward of h).
 *
 *   x                                   bf16 [M][K]
 *   gate_codes / up_codes               uint32 [I][K/8], 4-bit codes as above
 *   gate_scales, gate_biases, up_...    f16 [I][K/64]
 *   h                                   [M][I], bf16 (QL_BF16) or fp32 (QL_F32, for numerical tests)
 *
 * Arithmetic of the tcgen05 path (QL_PATH_TC_FUSED): g and u accumulate in fp32 from f16 operands
 * (weights RN_f16(s * q + b), activations scaled per row by a power of two), then
 * h = g / (1 + expf(-g)) * u in fp32, rounded once to the output type.  One GEMM computes both: each
 * tile holds 128 rows of the gate weight and the same 128 rows of the up weight, so g and u of an
 * output element meet in the epilogue and never travel through memory.
 * Preconditions as for qlinear_forward with N = I (I % 8 == 0), all eight tensors 16-byte aligned,
 * h overlapping no input and the workspace overlapping nothing; `workspace` must hold
 * qlinear_swiglu_workspace_size(M, K, I, group) bytes (QL_ERR_WORKSPACE otherwise).
 */
QL_API size_t qlinear_swiglu_workspace_size(int64_t M, int64_t K, int64_t I, int32_t group);
QL_API ql_status qlinear_swiglu_forward(const void* x, const uint32_t* gate_codes, const void* gate_scales,
                                        const void* gate_biases, const uint32_t* up_codes,
                                        const void* up_scales, const void* up_biases, void* h,
                                        ql_dtype out_dtype, int64_t M, int64_t K, int64_t I, int32_t group,
                                        void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * y[i] = sum_{z=0}^{S-1} partials[z][i], summed in z order in fp32 and rounded once to out_dtype.
 * partials is fp32 [S][count] (device, read only), y is [count] of out_dtype; count % 4 == 0.
 * This is the combination step of a K-sharded (row-parallel) layer: the ranks' fp32 partial
 * outputs (qlinear_forward_config with QL_F32), gathered in rank order, reduce to the same bytes on
 * every rank.  Errors: QL_ERR_INVALID_ARG (null pointer, S < 1, count not a positive multiple of 4,
 * y overlapping partials, bad out_dtype), QL_ERR_ALIGNMENT (a pointer not 16-byte aligned).
 */
QL_API ql_status qlinear_reduce_partials(const float* partials, int32_t S, int64_t count, void* y,
                                         ql_dtype out_dtype, cudaStream_t stream);

/*
 * Low-rank adapters of many requests beside a packed projection:
 *   t[m][j] = s[a] * sum_k x[m][k] * A[a][j][k],   a = adapter_ids[m]
 *   y[m][n] = sum_k x[m][k] * W[n][k] + sum_j t[m][j] * B[a][n][j]
 * x, codes, scales, biases, y and the arithmetic of the packed product as in qlinear_forward (QL_F32: y in fp32);
 * the adapters' products accumulate in fp32 too and y is rounded once.
 *
 *   lora_a        bf16 [L][r][K]     the L loaded adapters' down projections
 *   lora_b        bf16 [L][N][r]     their up projections
 *   lora_scale    fp32 [L]           s (e.g. alpha / rank); NULL: 1
 *   adapter_ids   int32 [M]          on the device: each row's adapter; -1: none, the row is qlinear_forward's.  Rows
 *                                    may carry their ids in any order.  An id outside [-1, L) counts as -1 and the
 *                                    device status word records QL_ERR_INVALID_ARG.
 *
 * Adapters of a lower rank than r are padded with zeros.  Preconditions and errors as in qlinear_forward, and L >= 1
 * and non-null lora_a, lora_b, adapter_ids (else QL_ERR_INVALID_ARG); r % 8 == 0 and r <= 128 (else
 * QL_ERR_UNSUPPORTED); lora_a and lora_b 16-byte, lora_scale and adapter_ids 4-byte aligned; y and the workspace
 * overlap no adapter tensor.  `workspace` holds qlinear_lora_workspace_size(M, K, N, group, L, r) bytes.
 * Non-finite activations and entries of lora_a reach the outputs of their own rows only.  A non-finite entry of
 * lora_b counts as zero and is recorded as QL_ERR_INVALID_ARG in the device status word: rows of several adapters
 * share a tensor-core tile, where it would reach the others' outputs.
 * Above 64 rows t is held as two bf16 terms (2^-16 relative) of t over the row's power of two; an adapter that makes t
 * more than 2^110 times its row's largest activation gives infinities there.
 *
 * Up to 64 rows the weights are streamed as in qlinear_forward and the adapters are added where the partial sums
 * meet; above, they are extra K-steps of the fused kernel, one 64-column step per 32 / r distinct adapters of each
 * 192-row tile, so rows of one adapter are best kept together (tokens in no order also have their t copied in
 * smaller pieces: 4608 rows of 30 adapters, r = 16, K = N = 4608 take 385 us against 205 in order).
 */
QL_API size_t qlinear_lora_workspace_size(int64_t M, int64_t K, int64_t N, int32_t group, int32_t L, int32_t r);
QL_API ql_status qlinear_lora_forward(const void* x, const uint32_t* codes, const void* scales, const void* biases,
                                      const void* lora_a, const void* lora_b, const float* lora_scale,
                                      const int32_t* adapter_ids, void* y, ql_dtype out_dtype, int64_t M, int64_t K,
                                      int64_t N, int32_t group, int32_t L, int32_t r, void* workspace,
                                      size_t workspace_bytes, cudaStream_t stream);
/* The same with 8-bit codes (uint32 [N][K/4], as qlinear8_forward). */
QL_API size_t qlinear8_lora_workspace_size(int64_t M, int64_t K, int64_t N, int32_t group, int32_t L, int32_t r);
QL_API ql_status qlinear8_lora_forward(const void* x, const uint32_t* codes, const void* scales, const void* biases,
                                       const void* lora_a, const void* lora_b, const float* lora_scale,
                                       const int32_t* adapter_ids, void* y, ql_dtype out_dtype, int64_t M, int64_t K,
                                       int64_t N, int32_t group, int32_t L, int32_t r, void* workspace,
                                       size_t workspace_bytes, cudaStream_t stream);

/*
 * The SwiGLU pair with adapters: h = silu(g) * u, where g and u are the projections of x by the gate and the up
 * weight, each with its own down and up projection of row m's adapter (one id and one scale for both):
 *   gate_lora_a, up_lora_a   bf16 [L][r][K]        gate_lora_b, up_lora_b   bf16 [L][I][r]
 * Everything else as in qlinear_swiglu_forward and qlinear_lora_forward.
 */
QL_API size_t qlinear_swiglu_lora_workspace_size(int64_t M, int64_t K, int64_t I, int32_t group, int32_t L, int32_t r);
QL_API ql_status qlinear_swiglu_lora_forward(const void* x, const uint32_t* gate_codes, const void* gate_scales,
                                             const void* gate_biases, const uint32_t* up_codes, const void* up_scales,
                                             const void* up_biases, const void* gate_lora_a, const void* gate_lora_b,
                                             const void* up_lora_a, const void* up_lora_b, const float* lora_scale,
                                             const int32_t* adapter_ids, void* h, ql_dtype out_dtype, int64_t M,
                                             int64_t K, int64_t I, int32_t group, int32_t L, int32_t r, void* workspace,
                                             size_t workspace_bytes, cudaStream_t stream);

/*
 * The norms after and before a block, fused with its gate and the residual update between them:
 *   v = sum_{z<S} y[z]                                  the block's output, partials summed in z order
 *   v = v / sqrt(mean_d v^2 + eps) * post_weight        when post_norm != 0
 *   r = residual_scale * x + branch_scale * gate[seg] * v
 *   h = r / sqrt(mean_d r^2 + eps) * pre_weight * (1 + scale[seg]) + shift[seg]       when h != NULL
 * with seg = segment_ids[m] and the means over the D entries of row m.  All of it in fp32; r and h are rounded once
 * each, h from the unrounded r.
 *
 *   x              [M][D] of x_dtype (QL_BF16 or QL_F32), the residual stream
 *   y              y_dtype QL_BF16: bf16 [M][D] (S = 1); QL_F32: fp32 [S][M][D], e.g. the gathered partial outputs of
 *                  a row-parallel projection, which this call then combines as qlinear_reduce_partials does.
 *                  NULL: r is x itself, only h is written (out must be NULL; S, y_dtype, post_*, gate are not looked at)
 *   out            [M][D] of x_dtype: r.  May be x (the update in place); other overlaps are refused
 *   h              bf16 [M][D], or NULL (no pre norm; pre_weight, scale and shift must then be NULL)
 *   post_weight, pre_weight   [D] of param_dtype; NULL: 1 (post_weight needs post_norm)
 *   gate           [T][D] of param_dtype; NULL: 1
 *   scale, shift   [T][D] of param_dtype; NULL: 0
 *   segment_ids    int32 [M] on the device; NULL: segment 0 for every row.  A row with a negative segment is padding:
 *                  it is not read, and its rows of out and h are left as they were.  A row with a segment >= T is
 *                  left alone too, and the device status word records QL_ERR_INVALID_ARG.
 *
 * Required (QL_ERR_INVALID_ARG): M >= 1, D >= 8, D % 8 == 0, T >= 1, S >= 1 (S == 1 for bf16 y), eps >= 0 and finite,
 * at least one output.  D <= QL_NORM_MAX_D (QL_ERR_UNSUPPORTED above).  All pointers 16-byte aligned except
 * segment_ids (4).  No workspace.  The mean squares are fp32 sums: a row whose sum of squares leaves fp32's range
 * normalizes by infinity, and one whose squares fall below it (entries under about 2^-63) by sqrt(eps) alone, so
 * with eps = 0 its result is infinite or NaN.
 */
#define QL_NORM_MAX_D 32768
QL_API ql_status qlinear_norm_residual(const void* x, ql_dtype x_dtype, const void* y, ql_dtype y_dtype, int32_t S,
                                       int32_t post_norm, const void* post_weight, const void* gate,
                                       float residual_scale, float branch_scale, const void* pre_weight,
                                       const void* scale, const void* shift, ql_dtype param_dtype,
                                       const int32_t* segment_ids, int32_t T, float eps, void* out, void* h,
                                       int64_t M, int64_t D, cudaStream_t stream);

/*
 * A packed projection with bias, activation, gate and residual in its epilogue:
 *   z[m][n] = sum_k x[m][k] * W[n][k] + bias[n]
 *   y[m][n] = residual[m][n] + gate[seg][n] * act(z[m][n]),   seg = segment_ids[m]
 * x, codes, scales, biases and the arithmetic of the packed product as in qlinear_forward; everything behind it in
 * fp32, y rounded once.  An activation errs by at most (20 + 8 E) 2^-24 of its value, where e^-E is the exponential
 * in it (E = |z|, z^2 / 2, 2 |u|), far in its tail too; values under 2^-120 may come out as zero.
 *
 *   bias          [N] of param_dtype (QL_BF16 or QL_F32); NULL: 0
 *   activation    a ql_activation: z; silu z / (1 + e^-z); gelu z Phi(z); its tanh form
 *                 z / 2 (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3)))
 *   gate          [T][N] of param_dtype; NULL: 1
 *   residual      [M][N] of out_dtype; may be y (the update in place; other overlaps are refused); NULL: 0
 *   segment_ids   int32 [M] on the device; NULL: segment 0 for every row.  A row with a negative segment is padding: its
 *                 row of y is left as it was.  A row with a segment >= T is left alone too, and the device status word
 *                 records QL_ERR_INVALID_ARG.
 *   y             [M][N] of out_dtype (QL_BF16 or QL_F32)
 *
 * Preconditions and errors as in qlinear_forward, and T >= 1, a known activation and types (else QL_ERR_INVALID_ARG);
 * bias, gate and residual 16-byte, segment_ids 4-byte aligned; y and the workspace overlap none of them (but y the
 * residual, as said).  `workspace` holds qlinear_epilogue_workspace_size(M, K, N, group) bytes (0: it may be NULL).
 *
 * Above 64 rows the epilogue is the fused kernel's (or, where its K-steps are split, that of their sum), up to 64 the
 * streaming path's reduction.  Up to 8 rows of a weight of at most 32 MiB of codes, 16 of 16 and 32 of 4 (of 8-bit codes
 * 8 and 2) may be one launch without a workspace, which multiplies exact codes, offset by 128, by the bf16 activations in
 * fp32: activations beyond 2^110 may overflow there, and an infinite one makes its row NaN.  Weights of 4-bit codes over
 * two thirds of these sizes and wider than N = 8192 (above 8 rows 4096) are faster on the streaming path: the workspace
 * size is that path's for them, and without such a workspace they are one launch like the others.
 */
typedef enum { QL_ACT_NONE = 0, QL_ACT_SILU = 1, QL_ACT_GELU = 2, QL_ACT_GELU_TANH = 3 } ql_activation;
QL_API size_t qlinear_epilogue_workspace_size(int64_t M, int64_t K, int64_t N, int32_t group);
QL_API ql_status qlinear_epilogue_forward(const void* x, const uint32_t* codes, const void* scales, const void* biases,
                                          const void* bias, int32_t activation, const void* gate, ql_dtype param_dtype,
                                          const void* residual, const int32_t* segment_ids, int32_t T, void* y,
                                          ql_dtype out_dtype, int64_t M, int64_t K, int64_t N, int32_t group,
                                          void* workspace, size_t workspace_bytes, cudaStream_t stream);
/* The same with 8-bit codes (uint32 [N][K/4], as qlinear8_forward). */
QL_API size_t qlinear8_epilogue_workspace_size(int64_t M, int64_t K, int64_t N, int32_t group);
QL_API ql_status qlinear8_epilogue_forward(const void* x, const uint32_t* codes, const void* scales, const void* biases,
                                           const void* bias, int32_t activation, const void* gate, ql_dtype param_dtype,
                                           const void* residual, const int32_t* segment_ids, int32_t T, void* y,
                                           ql_dtype out_dtype, int64_t M, int64_t K, int64_t N, int32_t group,
                                           void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * Rotation of heads by positions of several axes (time, height, width, as in the DiT's rotary embedding: jimmysue
 * "Ideogram 4" notes, MRoPE), alone or in the same pass as the norms of queries and keys head by head:
 *   n[m][h][d] = x[m][h][d] / sqrt(mean_d x[m][h][d]^2 + eps) * weight[d]       (qlinear_qk_norm_rotary)
 *   the first 2 P elements of every head are P pairs (a, b): elements i and i + P, or 2 i and 2 i + 1 (adjacent != 0);
 *   pair i turns by the angle 2 pi turns[i] positions[axes[i]][m]:  (a, b) <- (a cos - b sin, b cos + a sin)
 * All of it in fp32 but the angle, whose whole turns are dropped in 64 bits; outputs are rounded once.
 *
 * A ql_heads names one tensor of heads, [M][heads][D] with a stride per token and per head (in elements; a head's D
 * elements lie side by side), e.g. the queries or the keys inside a packed QKV projection's output, or one kept head
 * by head:
 *   in, in_token, in_head      what is read
 *   out, out_token, out_head   what is written: `in` itself with the same strides (in place), or memory that meets no
 *                              input.  No two elements of it may share a place.
 *   weight                     [D] of weight_dtype; NULL: 1 (NULL without norms)
 * The queries and the keys may have different numbers of heads and lie in one buffer.
 *
 *   dtype          QL_BF16 or QL_F32, of every tensor of heads
 *   positions      [A][M] of pos_type on the device: one row per axis.  NULL (with P == 0): norms without rotation
 *   turns          double [P] on the device: pair i's turns per unit of position, its frequency / 2 pi
 *   axes           int32 [P] on the device: the axis whose position pair i takes.  A pair with an axis outside [0, A) is
 *                  not turned, and the device status word records QL_ERR_INVALID_ARG.
 *   segment_ids    int32 [M] on the device or NULL: a row with a negative one is padding, it is not read and its heads of
 *                  `out` are left as they were
 *
 * Required (QL_ERR_INVALID_ARG): M >= 1, D >= 8, D % 8 == 0, heads >= 1, 0 <= 2 P <= D, eps >= 0 and finite,
 * A <= QL_HEAD_MAX_D, strides from 0 to 2^56 / max(M, heads).  P % 8 == 0 and D <= QL_HEAD_MAX_D (QL_ERR_UNSUPPORTED
 * otherwise).  Heads, weights and strides 16-byte aligned, the rest by their element.  k may be NULL (queries alone).  No
 * workspace.  Sums of squares leave fp32's range, above and below, as in qlinear_norm_residual.
 */
#define QL_HEAD_MAX_D 512
typedef enum { QL_POS_I32 = 0, QL_POS_I64 = 1, QL_POS_F32 = 2 } ql_pos_type;
typedef struct {
    const void* in;
    void* out;
    int64_t in_token, in_head, out_token, out_head;
    const void* weight;
    int32_t heads;
} ql_heads;
QL_API ql_status qlinear_rotary_axes(const ql_heads* x, ql_dtype dtype, const void* positions, ql_pos_type pos_type,
                                     int32_t A, const double* turns, const int32_t* axes, int32_t P, int32_t adjacent,
                                     const int32_t* segment_ids, int64_t M, int64_t D, cudaStream_t stream);
QL_API ql_status qlinear_qk_norm_rotary(const ql_heads* q, const ql_heads* k, ql_dtype dtype, ql_dtype weight_dtype,
                                        float eps, const void* positions, ql_pos_type pos_type, int32_t A,
                                        const double* turns, const int32_t* axes, int32_t P, int32_t adjacent,
                                        const int32_t* segment_ids, int64_t M, int64_t D, cudaStream_t stream);

/*
 * Self-test of the bounded waits inside the library's kernels.  Enqueues one small kernel that waits
 * on a barrier nothing ever completes, with the same bounded wait every pipeline role uses: it gives
 * up after the library's wait limit (about one second), records QL_ERR_DEVICE_TIMEOUT in the device
 * status word and returns, leaving the context usable.  A following qlinear_get_device_status()
 * therefore returns QL_ERR_DEVICE_TIMEOUT.  Returns QL_ERR_CUDA if the launch fails.
 */
QL_API ql_status qlinear_selftest_bounded_wait(cudaStream_t stream);

/* Static, human-readable name of a status code. */
QL_API const char* qlinear_status_string(ql_status status);

/* Library ABI version (major * 10000 + minor * 100 + patch). */
QL_API int32_t qlinear_version(void);

#ifdef __cplusplus
}
#endif

#endif /* QLINEAR_H */
