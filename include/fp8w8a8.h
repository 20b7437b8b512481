/*
 * fp8w8a8.h — C ABI of the FP8 (e4m3fn) W8A8 linear layer with dynamic
 * per-tensor activation quantization, for NVIDIA sm_103a (GB300).
 *
 * The layer (source pages: "Prototype FP8Linear W8A8 runtime quantization",
 * "[WIP] FP8 support", "[Kernel] Implement fallback for FP8 channelwise using
 * torch._scaled_mm", "Fp8 Quantization Support"):
 *
 *   s_w      = amax(W) / 448              (per tensor, or per output row n)
 *   qW       = e4m3(W / s_w)              once, when weights are loaded
 *   s_a      = amax(A) / 448              every call, on the device
 *   qA       = e4m3(A / s_a)
 *   Y[m, n]  = bf16( s_a * s_w[n] * sum_k qA[m, k] qW[n, k]  (+ bias[n]) )
 *
 * e4m3(x): IEEE fp32 quotient, then round-to-nearest-even to float8_e4m3fn,
 * saturating to +-448; the sign of zero is kept. A zero amax gives scale 1.
 * The product accumulates in fp32 on tensor cores.
 *
 * Conventions for every call:
 *  - Matrices are row-major. A bf16 [M, K] with row stride lda >= K elements;
 *    W bf16 [N, K] (out_features x in_features, as in nn.Linear) with stride
 *    ldw >= K; Y bf16 [M, N] with stride ldy >= N. bf16 strides may be any
 *    value: no padding of the logical dimensions is required ("[WIP] FP8
 *    support": dimensions that are not multiples of 16 must work).
 *  - The library's own FP8 matrices (qA, qW) are u8 [rows, ld] with ld a
 *    multiple of 16 and ld >= K (fp8_min_ld(K) is the smallest). The
 *    quantizers write bytes [K, ld) of every row as zero; consumers rely on
 *    that. The base address of an FP8 matrix must be 16-byte aligned.
 *  - Scales (s_a, s_w) are fp32 in DEVICE memory, so dynamic quantization
 *    never needs a host round trip.
 *  - Every pointer is a device pointer owned by the caller. The library
 *    allocates nothing, never synchronizes (except fp8_last_device_status),
 *    and enqueues all work on `stream` (NULL = the legacy default stream).
 *  - Argument errors are returned synchronously before anything is enqueued.
 *    FP8_ERR_CUDA reports a failed launch. Kernel-side errors (a bounded wait
 *    that expired) are reported later by fp8_last_device_status().
 *  - M == 0 or N == 0 is a no-op returning FP8_OK. K == 0 gives Y = bias (or 0).
 *  - A workspace may be used by one call at a time; calls are otherwise
 *    reentrant and thread-safe.
 *  - Launch ordering: kernels use programmatic dependent launch. The weight
 *    operands (qW, s_w, bias) of a linear call may be read before the kernel
 *    enqueued just before it has finished, so they must not be written by the
 *    immediately preceding kernel unless that kernel is fp8_quantize_weight,
 *    fp8_block_quantize_weight or one that does not trigger programmatic
 *    launch early (any ordinary CUDA or PyTorch kernel). Activations,
 *    workspace and Y are always ordered.
 */
#ifndef FP8W8A8_H
#define FP8W8A8_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t / CUstream. */
typedef struct CUstream_st* fp8_stream_t;

typedef enum fp8_status {
  FP8_OK = 0,
  FP8_ERR_INVALID_ARG = 1,        /* null pointer, negative size, ld too small, bad flag */
  FP8_ERR_MISALIGNED = 2,         /* FP8 ld not a multiple of 16, or a base address not aligned */
  FP8_ERR_WORKSPACE = 3,          /* workspace too small or not 256-byte aligned */
  FP8_ERR_CUDA = 4,               /* a CUDA runtime/driver call or kernel launch failed */
  FP8_ERR_TIMEOUT = 5,            /* a device-side bounded wait expired (see fp8_last_device_status) */
  FP8_ERR_UNSUPPORTED_DEVICE = 6  /* current device is not sm_103 */
} fp8_status;

/* FP8 storage formats. float8_e4m3fn is the pages' format ("Fp8 Quantization
 * Support": fp8 is assumed to be torch.float8_e4m3fn); float8_e5m2 is the one that
 * page names as the later extension. Every call without an _ex suffix uses e4m3. */
typedef enum fp8_format {
  FP8_E4M3 = 0, /* 1 sign, 4 exponent (bias 7), 3 mantissa bits; max 448; no infinity */
  FP8_E5M2 = 1  /* 1 sign, 5 exponent (bias 15), 2 mantissa bits; max 57344 */
} fp8_format;

#define FP8_E4M3_MAX 448.0f
#define FP8_E5M2_MAX 57344.0f
#define FP8_LD_ALIGN 16
/* Workspace needed by fp8_quantize_weight / fp8_quantize_act (partial amax values). */
#define FP8_QUANT_WORKSPACE_BYTES 4352

/* Smallest valid leading dimension (bytes) of an FP8 matrix with K columns: K rounded up to 16 (16 for K == 0). */
int64_t fp8_min_ld(int64_t K);

/* Bytes of workspace fp8_linear / fp8_linear_channelwise use for this shape.
 * 0 for decode shapes of up to 16 tokens (fp8_uses_gemv): the GEMV quantizes A
 * itself. Every other shape (the GEMV at 17..32 tokens, the GEMM) needs at
 * least FP8_QUANT_WORKSPACE_BYTES (partial amax values, s_a) plus the
 * quantized activations qA [M, fp8_min_ld(K)]. GEMM shapes with too few
 * output tiles to fill the GPU (small M) split K across CTAs when the
 * workspace also holds, from the next 256-byte boundary, fp32 partials
 * [splits, M, N rounded up to 4]; the value returned includes that space for
 * the split a GB300 (152 SMs) takes. A workspace between the two sizes works
 * too, with a smaller split or none. 0 when M or K is 0. Host-only, never
 * touches the device. */
size_t fp8_workspace_bytes(int64_t M, int64_t K, int64_t N);

/* 1 when fp8_linear takes the decode GEMV path for this shape, 0 for the GEMM path:
 * M <= the crossover (32 by default, see fp8_set_gemv_max_m) and K <= 32768. Host-only. */
int fp8_uses_gemv(int64_t M, int64_t K, int64_t N);

/* Sets the decode crossover: calls with M <= m (and K <= 32768) run the GEMV,
 * larger M the GEMM. m is clamped to [0, 32] (32 is the GEMV's largest M; 0
 * sends every shape to the GEMM); m < 0 only queries. Returns the previous
 * value. The start-up value is 32, or FP8W8A8_GEMV_MAX_M from the environment.
 * Process-wide; it changes which kernels later calls enqueue (and so
 * fp8_workspace_bytes), never their results beyond the stated tolerance.
 * ("[WIP] FP8 support": decode runs at sequence length < 16 and wants its own
 * GEMV; where exactly to switch is a tuning choice.) Host-only. */
int fp8_set_gemv_max_m(int m);

/*
 * Quantize bf16 weights W [N, K] (stride ldw) to qW u8 [N, ldq] and scales s_w.
 * per_channel == 0: one scale, s_w[0] = amax(W)/448 ("Fp8 Quantization
 * Support", recipe strategy "tensor"). per_channel == 1: s_w[n] = amax(W[n,:])/448
 * for each output channel ("[Kernel] Implement fallback for FP8 channelwise
 * using torch._scaled_mm"). Bytes [K, ldq) of each row are written as zero.
 * ws: device workspace of >= FP8_QUANT_WORKSPACE_BYTES bytes, 256-byte aligned
 * (unused when per_channel == 1; may then be NULL).
 */
fp8_status fp8_quantize_weight(const void* w_bf16, int64_t N, int64_t K, int64_t ldw,
                               int per_channel, uint8_t* qw, int64_t ldq, float* s_w,
                               void* ws, size_t ws_bytes, fp8_stream_t stream);

/*
 * Dynamic per-tensor activation quantization ("Prototype FP8Linear W8A8
 * runtime quantization": activations are quantized at run time):
 * s_a[0] = amax(A)/448, qA = e4m3(A / s_a) as u8 [M, ldq], tail bytes zero.
 * ws: >= FP8_QUANT_WORKSPACE_BYTES bytes, 256-byte aligned.
 */
fp8_status fp8_quantize_act(const void* a_bf16, int64_t M, int64_t K, int64_t lda,
                            uint8_t* qa, int64_t ldq, float* s_a,
                            void* ws, size_t ws_bytes, fp8_stream_t stream);

/*
 * Scaled FP8 GEMM on already-quantized operands — the step the pages run with
 * torch._scaled_mm ("Prototype FP8Linear W8A8 runtime quantization";
 * "[Kernel] Implement fallback for FP8 channelwise using torch._scaled_mm"):
 *   Y[m, n] = bf16( s_a[0] * s_w[n or 0] * sum_k qA[m,k] qW[n,k] (+ bias[n]) ).
 * qa u8 [M, ldqa], qw u8 [N, ldqw] (both ld multiples of 16, tails zero);
 * s_a device fp32 [1]; s_w device fp32 [1] (per_channel == 0) or [N]
 * (per_channel == 1); bias bf16 [N] or NULL; y bf16 [M, ldy].
 * Uses no workspace.
 */
fp8_status fp8_scaled_mm(const uint8_t* qa, int64_t M, int64_t K, int64_t ldqa, const float* s_a,
                         const uint8_t* qw, int64_t N, int64_t ldqw, const float* s_w,
                         int per_channel, const void* bias_bf16, void* y_bf16, int64_t ldy,
                         fp8_stream_t stream);

/*
 * The W8A8 linear with dynamic per-tensor activation quantization and a
 * per-tensor weight scale s_w[0]: amax(A) -> s_a -> e4m3(A/s_a) -> FP8 GEMM
 * (fp32 accumulate) -> s_a*s_w (+bias) epilogue -> bf16 Y.
 * Decode shapes (fp8_uses_gemv) run one persistent split-K GEMV kernel that
 * quantizes A itself and streams qW once ("[WIP] FP8 support": LLM decode runs
 * at sequence length < 16 and wants a custom gemv); larger M runs amax + cast
 * + the tcgen05 GEMM. No padding or repacking of A, W or Y happens on any path.
 * ws: >= fp8_workspace_bytes(M, K, N) bytes, 256-byte aligned (may be NULL
 * when that is 0).
 */
fp8_status fp8_linear(const void* a_bf16, int64_t M, int64_t K, int64_t lda,
                      const uint8_t* qw, int64_t N, int64_t ldqw, const float* s_w,
                      const void* bias_bf16, void* y_bf16, int64_t ldy,
                      void* ws, size_t ws_bytes, fp8_stream_t stream);

/*
 * Same as fp8_linear with one weight scale per output channel, s_w[N]; the
 * channel scale is applied to column n after the product, using
 * (s_a A)(s_w,n W_n)^T = s_a s_w,n (A W_n^T) ("[Kernel] Implement fallback for
 * FP8 channelwise using torch._scaled_mm"), fused into the epilogue.
 */
fp8_status fp8_linear_channelwise(const void* a_bf16, int64_t M, int64_t K, int64_t lda,
                                  const uint8_t* qw, int64_t N, int64_t ldqw, const float* s_w,
                                  const void* bias_bf16, void* y_bf16, int64_t ldy,
                                  void* ws, size_t ws_bytes, fp8_stream_t stream);

/*
 * fp8_linear (per_channel == 0) or fp8_linear_channelwise (per_channel == 1)
 * without a workspace argument, for callers that cannot allocate device memory:
 * for example code that runs inside a host application which owns the whole
 * device-memory budget and hands a kernel only its input and output buffers,
 * or a latency-critical path that must not call cudaMalloc, which can block
 * until other work on the device has finished. The source pages have no
 * counterpart of this call; it exists only for such callers.
 *
 * The scratch lives in one fixed array inside the library of
 * FP8_NOALLOC_SCRATCH_BYTES bytes, which every GPU that loads the library holds
 * until the process exits. A call needs the least workspace fp8_linear
 * accepts: nothing for decode shapes, and for GEMM shapes M * fp8_min_ld(K)
 * may be at most FP8_NOALLOC_SCRATCH_BYTES - 4352. Larger shapes are refused
 * with FP8_ERR_WORKSPACE before anything is enqueued. The rest of the array
 * serves a K split where one fits (the same launches fp8_linear makes with a
 * workspace of FP8_NOALLOC_SCRATCH_BYTES). The call allocates nothing.
 *
 * The first call on a device looks up the array's device address
 * (cudaGetSymbolAddress) with that device current; make that first call
 * before any stream capture. After a device reset (cudaDeviceReset) the
 * address is looked up again on the next call, which then also belongs
 * outside any capture. All calls share the one array and it keeps the
 * previous call's contents: nothing in it has to start at zero (each call
 * writes every scratch byte it reads before reading it), but two calls whose
 * kernels overlap on the GPU — on different streams or from different host
 * threads — race on it and give wrong results. Order such calls on one stream.
 * Arguments and every other rule are those of fp8_linear.
 */
#define FP8_NOALLOC_SCRATCH_BYTES (8u * 1024u * 1024u)
fp8_status fp8_linear_noalloc(const void* a_bf16, int64_t M, int64_t K, int64_t lda,
                              const uint8_t* qw, int64_t N, int64_t ldqw, const float* s_w,
                              int per_channel, const void* bias_bf16, void* y_bf16, int64_t ldy,
                              fp8_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Wider calls: the format of each FP8 operand, and a static activation scale.
 * In all of them, for format F: max(F) = 448 (FP8_E4M3) or 57344 (FP8_E5M2),
 * dynamic scale = amax / max(F), q = F(x / scale) with the rounding and
 * saturation rules above (saturation to +-max(F), never infinity).
 * Invalid format values return FP8_ERR_INVALID_ARG.
 * ---------------------------------------------------------------------------
 */

/* fp8_quantize_weight with the weight format `fmt`. */
fp8_status fp8_quantize_weight_ex(const void* w_bf16, int64_t N, int64_t K, int64_t ldw,
                                  int per_channel, fp8_format fmt, uint8_t* qw, int64_t ldq,
                                  float* s_w, void* ws, size_t ws_bytes, fp8_stream_t stream);

/*
 * fp8_quantize_act with the activation format `fmt` and an optional static
 * scale. s_static == NULL: dynamic, s_a[0] = amax(A) / max(fmt); ws as for
 * fp8_quantize_act. s_static != NULL (device fp32 [1], 4-byte aligned): the
 * calibrated scale is used as given ("Fp8 Quantization Support": the recipe
 * quantizes input activations per tensor with scales from the calibration
 * run), no amax pass runs, s_a[0] receives a copy of it and ws may be NULL.
 * Elements beyond s * max(fmt) saturate. The scale must be positive and finite.
 */
fp8_status fp8_quantize_act_ex(const void* a_bf16, int64_t M, int64_t K, int64_t lda,
                               fp8_format fmt, const float* s_static, uint8_t* qa, int64_t ldq,
                               float* s_a, void* ws, size_t ws_bytes, fp8_stream_t stream);

/* fp8_scaled_mm with the formats of qA (fmt_a) and qW (fmt_w); any pairing. */
fp8_status fp8_scaled_mm_ex(const uint8_t* qa, fp8_format fmt_a, int64_t M, int64_t K, int64_t ldqa,
                            const float* s_a, const uint8_t* qw, fp8_format fmt_w, int64_t N,
                            int64_t ldqw, const float* s_w, int per_channel, const void* bias_bf16,
                            void* y_bf16, int64_t ldy, fp8_stream_t stream);

/*
 * The W8A8 linear with a static (calibrated) per-tensor activation scale s_a
 * (device fp32 [1]) instead of the dynamic one: qA = e4m3(A / s_a), then the
 * same product and epilogue as fp8_linear (per_channel == 0) or
 * fp8_linear_channelwise (per_channel == 1). No amax is computed. Workspace as
 * for fp8_linear (fp8_workspace_bytes).
 */
fp8_status fp8_linear_static(const void* a_bf16, int64_t M, int64_t K, int64_t lda,
                             const float* s_a, const uint8_t* qw, int64_t N, int64_t ldqw,
                             const float* s_w, int per_channel, const void* bias_bf16,
                             void* y_bf16, int64_t ldy, void* ws, size_t ws_bytes,
                             fp8_stream_t stream);

/*
 * The general linear: activation format fmt_a, weight format fmt_w (qW as
 * written by fp8_quantize_weight_ex with that format), dynamic activation
 * scale when s_static is NULL, else the static one; per_channel selects the
 * weight-scale mode. Workspace as for fp8_linear.
 */
fp8_status fp8_linear_ex(const void* a_bf16, int64_t M, int64_t K, int64_t lda, fp8_format fmt_a,
                         const float* s_static, const uint8_t* qw, fp8_format fmt_w, int64_t N,
                         int64_t ldqw, const float* s_w, int per_channel, const void* bias_bf16,
                         void* y_bf16, int64_t ldy, void* ws, size_t ws_bytes, fp8_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Weight-only FP8: the FP8 weights are kept for memory and up-converted to the
 * original dtype for the product ("Prototype FP8Linear W8A8 runtime
 * quantization": the path below compute capability 9.0, where weights are
 * dequantized into higher precision with no compute savings). A stays bf16:
 *   Y[m, n] = bf16( s_w[n or 0] * sum_k A[m, k] * decode(qW[n, k]) (+ bias[n]) ).
 * Every e4m3 / e5m2 value is a bf16 value, so the up-conversion is exact; the
 * weight scale multiplies the fp32 accumulator in the epilogue, as in the
 * channelwise identity (s_w,n W_n) A = s_w,n (W_n A).
 * Decode shapes (M <= the crossover, K <= 32768) run the split-K GEMV, which up-converts
 * each weight tile in registers and needs no workspace; larger shapes
 * up-convert W into the workspace once per call and run a bf16 tcgen05 GEMM.
 * ---------------------------------------------------------------------------
 */

/* Workspace fp8_linear_weight_only needs: 0 for decode shapes; otherwise the
 * up-converted weights (N * round_up(K, 8) bf16, rounded up to 256 bytes) plus
 * M * round_up(K, 8) bf16 for an aligned copy of A, used only when A's row
 * stride or base address is not a multiple of 16 bytes. Host-only. */
size_t fp8_weight_only_workspace_bytes(int64_t M, int64_t K, int64_t N);

/* qw, s_w from fp8_quantize_weight(_ex) with format fmt_w; per_channel as
 * there; other arguments and rules as for fp8_linear. */
fp8_status fp8_linear_weight_only(const void* a_bf16, int64_t M, int64_t K, int64_t lda,
                                  const uint8_t* qw, fp8_format fmt_w, int64_t N, int64_t ldqw,
                                  const float* s_w, int per_channel, const void* bias_bf16,
                                  void* y_bf16, int64_t ldy, void* ws, size_t ws_bytes,
                                  fp8_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Block-scaled FP8 linear: one scale per token and 128 values of K for the
 * activations, one per 128 x 128 block of the weights. With K blocks
 * b = [128 b, min(K, 128 b + 128)), KB = ceil(K / 128), NB = ceil(N / 128):
 *
 *   s_a[b][m] = max_{k in b} |A[m, k]| / 448        qA[m, k] = e4m3(A[m, k] / s_a[b][m])
 *   s_w[j][b] = max over rows 128 j .. and b |W| / 448   qW[n, k] = e4m3(W[n, k] / s_w[j][b])
 *   Y[m, n]   = bf16( sum_b s_a[b][m] s_w[n / 128][b] sum_{k in b} qA[m, k] qW[n, k] (+ bias[n]) )
 *
 * with the quotient, rounding and zero rules above (a block of zeros has scale
 * 1). Both formats are e4m3: a scale for every 128 values leaves no use for the
 * wider range of e5m2. Sums are fp32. A block that holds a NaN has a NaN
 * scale, so its token's (weights: its 128 rows') results are NaN; an infinity
 * gives an infinite scale and NaN as well. Other rows are not affected.
 * FP8 matrices are laid out as above (ld a multiple of 16; the quantizers write bytes
 * [K, ld) of each row as zero).
 * ---------------------------------------------------------------------------
 */

/* Quantizes B matrices W [N, K] (row stride ldw, matrix stride mat_stride, in
 * elements; ignored when B is 1) to qw u8 [B][N, ldq] and s_w fp32
 * [B][NB][KB], both without gaps between matrices. */
fp8_status fp8_block_quantize_weight(const void* w_bf16, int64_t B, int64_t N, int64_t K, int64_t ldw,
                                     int64_t mat_stride, uint8_t* qw, int64_t ldq, float* s_w,
                                     fp8_stream_t stream);

/* Quantizes activations A [M, K] to qa u8 [M, ldq] and s_a fp32 [KB][lds],
 * lds >= M (the scales of one K block are adjacent). */
fp8_status fp8_block_quantize_act(const void* a_bf16, int64_t M, int64_t K, int64_t lda, uint8_t* qa,
                                  int64_t ldq, float* s_a, int64_t lds, fp8_stream_t stream);

/* The product on operands quantized by the two calls above. Uses no workspace. */
fp8_status fp8_block_scaled_mm(const uint8_t* qa, int64_t M, int64_t K, int64_t ldqa, const float* s_a,
                               int64_t lds, const uint8_t* qw, int64_t N, int64_t ldqw, const float* s_w,
                               const void* bias_bf16, void* y_bf16, int64_t ldy, fp8_stream_t stream);

/* Workspace fp8_block_linear needs for this shape. Host-only. */
size_t fp8_block_workspace_bytes(int64_t M, int64_t K, int64_t N);

/* The linear: quantizes A, then the product. ws: >= fp8_block_workspace_bytes,
 * 256-byte aligned. */
fp8_status fp8_block_linear(const void* a_bf16, int64_t M, int64_t K, int64_t lda, const uint8_t* qw,
                            int64_t N, int64_t ldqw, const float* s_w, const void* bias_bf16, void* y_bf16,
                            int64_t ldy, void* ws, size_t ws_bytes, fp8_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Mixture of experts: the choice of experts, and the chosen experts' networks
 * on block-scaled FP8 weights.
 * ---------------------------------------------------------------------------
 */

/*
 * Chooses k of E experts for each of T tokens from logits x [T, E] (row stride
 * ld; fp32, or bf16 when logits_bf16 is 1), in fp32:
 *   sigmoid == 0: p = exp(x - max x) / sum;  sigmoid == 1: p = 1 / (1 + exp(-x))
 *   choice c = p + bias (bias fp32 [E], a term for load balance that steers the
 *   choice only; NULL: c = p, for softmax compared as x, the same order).
 * groups > 1: the experts form `groups` equal consecutive groups; a group's
 * score is the sum of its two largest c (its largest for softmax without bias)
 * and only the keep_groups best groups take part.
 * ids[t, 0..k) (int32): the experts with the largest c in descending order, ties
 * to the lowest index; weights[t, j] (fp32) = p of ids[t, j], divided by
 * (their sum + 1e-20) when renormalize is 1, times factor.
 * A NaN logit counts as -inf. A softmax row of only -inf has p = 0 (weights 0;
 * the bias, if any, alone orders its experts).
 * Limits: E <= 512, k <= 32, groups <= 32, E a multiple of groups,
 * k <= keep_groups * E / groups (else FP8_ERR_INVALID_ARG).
 */
fp8_status fp8_moe_route(const void* logits, int logits_bf16, int64_t T, int64_t E, int64_t ld, int sigmoid,
                         const float* bias, int groups, int keep_groups, int k, int renormalize, float factor,
                         int32_t* ids, float* weights, fp8_stream_t stream);

/* The same with group_max: 1 scores a group by its largest c in every case, 0 as above. Gates that are
 * published with groups take the largest where they have no bias, for sigmoid too: such a sigmoid gate
 * without a bias is called with 1. */
fp8_status fp8_moe_route_ex(const void* logits, int logits_bf16, int64_t T, int64_t E, int64_t ld, int sigmoid,
                            const float* bias, int groups, int keep_groups, int group_max, int k, int renormalize,
                            float factor, int32_t* ids, float* weights, fp8_stream_t stream);

/* Workspace fp8_moe_experts needs (0 for sizes it refuses). Host-only. */
size_t fp8_moe_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I);

/*
 * The experts' gated networks over tokens x bf16 [T, H], summed by routing
 * weight. For each pair (t, j) with e = ids[t, j] in [0, E):
 *   g = x_t W13[e, 0]^T,  u = x_t W13[e, 1]^T        (block-scaled products, fp32)
 *   h = silu(g) * u, quantized like activations (1 x 128 along I) from fp32
 *   y[t] = bf16( sum_j weights[t, j] * (h W2[e]^T) )  (fp32, in the order of j)
 * Pairs with any other id (experts that live elsewhere) contribute nothing; a
 * token with none gets zeros. ids, weights [T, k] without gaps; an expert may
 * occur more than once in a row. qw13 u8 [E][2][I, ldq13], s13 fp32
 * [E][2][ceil(I/128)][ceil(H/128)]; qw2 u8 [E][H, ldq2], s2 fp32
 * [E][ceil(H/128)][ceil(I/128)], as fp8_block_quantize_weight writes them for
 * 2 E and E matrices. Results do not depend on timing. y may not overlap x.
 * ws: >= fp8_moe_workspace_bytes, 256-byte aligned: from two tokens on about
 * T * k * (5 H + I) bytes, most of it the pairs' fp32 rows of H (8192 tokens, 8
 * experts each, H 4096, I 2048: 1.5 GB). Limits: E <= 512, k <= 32.
 */
fp8_status fp8_moe_experts(const void* x_bf16, int64_t T, int64_t H, int64_t ldx, const int32_t* ids,
                           const float* weights, int64_t k, const uint8_t* qw13, int64_t ldq13, const float* s13,
                           const uint8_t* qw2, int64_t ldq2, const float* s2, int64_t E, int64_t I, void* y_bf16,
                           int64_t ldy, void* ws, size_t ws_bytes, fp8_stream_t stream);

/*
 * Tokens to rows sorted by expert, and back: for experts' networks other than the one above (a per-tensor
 * fp8_linear of each, or ones that are trained). Rows are bf16, or fp32 when f32 is 1.
 *
 * fp8_moe_dispatch: pair (t, j) with ids[t, j] in [0, E) gets row pos[t, j] of xs, rows sorted by expert and, within one,
 * by t and j; any other id gets pos -1 and no row. offsets[e] is expert e's first row, offsets[E] the number
 * of rows; xs[pos[t, j]] = x[t]. xs has T * k rows; those from offsets[E] on are left as they were. What is written
 * may not overlap what is read. ids and pos int32
 * [T, k], offsets int32 [E + 1], in device memory. ws: >= fp8_moe_dispatch_workspace_bytes, 256-byte aligned.
 */
size_t fp8_moe_dispatch_workspace_bytes(int64_t T, int64_t k, int64_t E);
fp8_status fp8_moe_dispatch(const void* x, int f32, int64_t T, int64_t H, int64_t ldx, const int32_t* ids, int64_t k,
                            int64_t E, void* xs, int64_t ldxs, int32_t* pos, int32_t* offsets, void* ws,
                            size_t ws_bytes, fp8_stream_t stream);

/* y[t] = sum_j weights[t, j] ys[pos[t, j]] over the pairs with pos in [0, R), in the order of j, in fp32 with one
 * rounding; a token with none gets zeros. weights fp32 [T, k], or NULL for ones. y may not overlap ys. */
fp8_status fp8_moe_combine(const void* ys, int f32, int64_t R, int64_t H, int64_t ldys, const int32_t* pos,
                           const float* weights, int64_t T, int64_t k, void* y, int64_t ldy, fp8_stream_t stream);

/* The gradient of fp8_moe_combine: dys[pos[t, j]] = weights[t, j] dy[t] (rows of no pair are left as they were) and
 * dw[t, j] = <dy[t], ys[pos[t, j]]>, fp32 [T, k], 0 for a pair without a row. No two pairs may have the same row (those
 * of fp8_moe_dispatch do not). dys may be ys, with the same stride, and may overlap nothing else. */
fp8_status fp8_moe_combine_grad(const void* dy, int f32, int64_t T, int64_t H, int64_t lddy, const void* ys, int64_t R,
                                int64_t ldys, const int32_t* pos, const float* weights, int64_t k, void* dys,
                                int64_t lddys, float* dw, fp8_stream_t stream);

/* The gradient of fp8_moe_dispatch: dx[t] = sum_j dxs[pos[t, j]], as fp8_moe_combine without weights. */
fp8_status fp8_moe_dispatch_grad(const void* dxs, int f32, int64_t R, int64_t H, int64_t lddxs, const int32_t* pos,
                                 int64_t T, int64_t k, void* dx, int64_t lddx, fp8_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Low-rank adapters of many requests beside a projection they share. For each
 * token m with e = ids[m] in [0, L):
 *   out[m] = bf16( y[m] + scales[e] * B[e] (A[e] x[m]) )
 * and out[m] = y[m] for any other id. y bf16 [M, N] is the output of a linear
 * of x bf16 [M, K] (any of the linears here), A bf16 [L][r, K], B bf16
 * [L][N, r], without gaps; ids int32 [M], scales fp32 [L] (NULL: ones). Sums and
 * A x are fp32, in every form (tensor cores take A x as the sum of three bf16 numbers, all of its bits down to 2^-133);
 * the only rounding to bf16 is that of out. Results do not depend
 * on timing. A NaN or an infinity, in B too, gives what the formula gives in
 * fp32, and stays with the tokens of its row or adapter. out may be y (with the same stride), else may not overlap it, nor
 * anything else that is read. ws: >= fp8_lora_workspace_bytes, 256-byte aligned (fewer tokens may need more, since K is split
 * further for them: one kept for several M has the largest of theirs). Limits: r 1 to 256, L <= 511, K
 * and N <= 2^30 (FP8_ERR_INVALID_ARG).
 * ---------------------------------------------------------------------------
 */
size_t fp8_lora_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t L, int64_t r);
fp8_status fp8_lora_add(const void* y_bf16, int64_t M, int64_t N, int64_t ldy, const void* x_bf16, int64_t K,
                        int64_t ldx, const void* a_bf16, const void* b_bf16, int64_t L, int64_t r, const int32_t* ids,
                        const float* scales, void* out_bf16, int64_t ldo, void* ws, size_t ws_bytes,
                        fp8_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Norms before and after a block, with its gate and residual.
 * ---------------------------------------------------------------------------
 */

/*
 * The end of one block and the norm before the next, row by row, in fp32:
 *   t = y                                                  (post_w NULL)
 *   t = y / sqrt(mean y^2 + eps) * post_w                  (else)
 *   r = residual + scale * gate * t                        (NULL: 0 and 1)
 *   n = r / sqrt(mean r^2 + eps) * w                       (of r before its rounding)
 * y, residual bf16 [M, H]; post_w, w bf16 [H], with plus_one 1 both stand for
 * 1 + their values; gate bf16 [M, H] with row stride ldg, or [H] with ldg 0.
 * Writes r and n as bf16 [M, H]; either may be NULL (w NULL with n). r may be y
 * or residual itself (with the same stride), and so may n where r is not; r and n are never the same
 * (FP8_ERR_INVALID_ARG). The mean is over H columns;
 * rows whose squares pass fp32's range, at either end, are normalised as the formula has it. A
 * NaN or an infinity in a row makes NaN of what it multiplies in that row and
 * of no other row. eps > 0, scale finite, H <= 32768
 * (FP8_ERR_INVALID_ARG).
 */
fp8_status fp8_residual_norm(const void* y_bf16, int64_t M, int64_t H, int64_t ldy, const void* post_w_bf16,
                             const void* gate_bf16, int64_t ldg, float scale, const void* residual_bf16,
                             int64_t ldr, const void* w_bf16, float eps, int plus_one, void* r_bf16, int64_t ldro,
                             void* n_bf16, int64_t ldn, fp8_stream_t stream);

/* The same with n quantized as fp8_block_quantize_act quantizes, from fp32: qn u8 [M, ldq] (bytes [H, ldq) of
 * each row zero) and s_n fp32 [ceil(H/128)][lds], lds >= M: operands of fp8_block_scaled_mm. r may be NULL. */
fp8_status fp8_residual_norm_quantize(const void* y_bf16, int64_t M, int64_t H, int64_t ldy, const void* post_w_bf16,
                                      const void* gate_bf16, int64_t ldg, float scale, const void* residual_bf16,
                                      int64_t ldr, const void* w_bf16, float eps, int plus_one, void* r_bf16,
                                      int64_t ldro, uint8_t* qn, int64_t ldq, float* s_n, int64_t lds,
                                      fp8_stream_t stream);

/*
 * Diagnostics (no counterpart on the source pages): the launch the GEMM path of
 * fp8_linear (and fp8_scaled_mm, which never splits K) would use for FP8
 * operands qa [M, ldqa] and qw [N, ldqw] (ld in bytes), K columns, and a
 * linear workspace of ws_bytes, on the current device. *two_sm = 1 when CTA
 * pairs run the two-SM MMA (tcgen05 cta_group::2), which needs at least two
 * 128-row blocks and both operands in the current device's own memory
 * (cudaMalloc'd on it); any other memory (pinned or managed host memory,
 * another GPU's memory) takes one CTA per tile, *two_sm = 0. *grid = CTAs
 * launched; *group_n = column tiles per raster group; *splits = CTAs that
 * share each output tile's K (1: no split; more when there are too few tiles
 * to fill the GPU and ws_bytes holds the fp32 partials); *tail_split = column
 * units each tile of the last, partial wave is divided into (1: none; 2 or 4
 * when that many units per left-over tile still fit one wave, each computing
 * 256 / tail_split columns over all of K). Output pointers may be NULL.
 * Enqueues nothing; FP8_ERR_INVALID_ARG for non-positive sizes,
 * FP8_ERR_CUDA or FP8_ERR_UNSUPPORTED_DEVICE when the device cannot be queried.
 */
fp8_status fp8_gemm_config(const uint8_t* qa, int64_t M, int64_t ldqa, const uint8_t* qw, int64_t N,
                           int64_t ldqw, int64_t K, size_t ws_bytes, int* two_sm, int* grid, int* group_n,
                           int* splits, int* tail_split);

/* The same plan as fp8_gemm_config, computed on the host without a device for a GPU with
 * num_sms SMs and pair_slots co-resident CTA pairs (0: no pair mode), with both operands in
 * that GPU's own memory and gap-free (leading dimension fp8_min_ld(K)). Outputs as above
 * (NULL allowed). FP8_ERR_INVALID_ARG for non-positive sizes or num_sms, negative pair_slots.
 * Host-only, never touches the device. */
fp8_status fp8_gemm_plan_model(int64_t M, int64_t N, int64_t K, int num_sms, int pair_slots, size_t ws_bytes,
                               int* two_sm, int* grid, int* group_n, int* splits, int* tail_split);

/* The decode GEMV's launch configuration, computed on the host without a device ("[WIP] FP8
 * support": the decode GEMV). mode: 0 activations already quantized (fp8_scaled_mm, and
 * fp8_linear from 17 tokens on), 1 quantized inside the kernel (fp8_linear up to 16 tokens;
 * static_scale != 0 for fp8_linear_static), 2 bf16 activations (weight-only). smem_limit:
 * dynamic shared memory a CTA may use; clusters_of_size[s - 1]: co-resident clusters of s CTAs
 * at that shared memory, s = 1..8 (host memory, 8 ints). Outputs (NULL allowed): *cluster = CTAs
 * per cluster sharing K, *clusters = clusters launched, *stages = weight-ring depth, *kslice =
 * bytes of K per CTA, *scratch_a = how A reaches shared memory in mode 1 (0 per-thread loads,
 * 1 all of A bulk-copied, 2 the CTA's slice), *cluster_amax = 1 when the dynamic maximum is
 * exchanged over the cluster, *tcgen05 = 1 when the main loop runs on tcgen05. A's rows are
 * taken as 16-byte aligned. FP8_ERR_INVALID_ARG for M outside 1..32, K outside 1..32768, other
 * bad sizes or mode; FP8_ERR_CUDA when no configuration fits (the launch would fail the same
 * way). Host-only, never touches the device. */
fp8_status fp8_gemv_plan_model(int64_t M, int64_t N, int64_t K, int mode, int static_scale, int smem_limit,
                               const int* clusters_of_size, int* cluster, int* clusters, int* stages, int* kslice,
                               int* scratch_a, int* cluster_amax, int* tcgen05);

/*
 * Synchronizes `stream`, then reports and clears device-side errors recorded
 * by the library's kernels on the current device since the last query
 * (FP8_ERR_TIMEOUT when a bounded wait expired), or FP8_ERR_CUDA when the
 * stream itself reports an error. FP8_OK otherwise.
 */
fp8_status fp8_last_device_status(fp8_stream_t stream);

/*
 * Failure-path self-test: enqueues a small kernel whose bounded device wait is
 * made to run out (its producer withholds one item), using the same wait
 * primitive and error word as the library's GEMV. The wait gives up after
 * limit_ns (1e3 .. 1e10 nanoseconds, else FP8_ERR_INVALID_ARG), the kernel
 * returns normally and the context stays usable; the next
 * fp8_last_device_status reports FP8_ERR_TIMEOUT once. Nothing faults or hangs.
 * The pages have no counterpart; it exists so the error path can be tested.
 */
fp8_status fp8_selftest_timeout(int64_t limit_ns, fp8_stream_t stream);

/*
 * The same for the block-scaled product: enqueues it with one load withheld
 * from its waits (the last K block of the first tile of its first CTA), so that
 * they run out after 20 ms, the CTA leaves its work and the next
 * fp8_last_device_status reports FP8_ERR_TIMEOUT once. That tile, and what the
 * CTA had still to do, keeps what Y held; all else is the product. form 0:
 * tiles of 256 columns, Y bf16 [M, N] (N and ldy multiples of 8, Y 16-byte
 * aligned); 1: tiles of 64, each shared by two CTAs (K > 128); 2: the gate and
 * up matrices qw [2][N, ldqw], s_w [2][NB][KB] with SwiGLU, Y the codes
 * [M, ldy] and s_y [NB][lds_y] of h (s_y, lds_y unused otherwise). M, N, K >= 1.
 */
fp8_status fp8_block_selftest_timeout(int form, const uint8_t* qa, int64_t M, int64_t K, int64_t ldqa,
                                      const float* s_a, int64_t lds, const uint8_t* qw, int64_t N, int64_t ldqw,
                                      const float* s_w, void* y, int64_t ldy, float* s_y, int64_t lds_y,
                                      fp8_stream_t stream);

/*
 * The same for the adapters of many tokens (sizes for which fp8_lora_workspace_bytes is not 0): the call with one load
 * withheld from the waits of its first CTA. form 0: the first product's last load of A for its first tile (rows of x and
 * A on 16-byte boundaries): the tile's rows get NaN, all others what the call gives. form 1: the second product's second load of B
 * (rank a multiple of 8 up to 64, rows of y, out and B on 16-byte boundaries); 2: the same by the warps that load B of odd
 * ranks (up to 192). All that the CTA had to do from there on keeps what out held; all else is what the call gives.
 */
fp8_status fp8_lora_selftest_timeout(int form, const void* y_bf16, int64_t M, int64_t N, int64_t ldy, const void* x_bf16,
                                     int64_t K, int64_t ldx, const void* a_bf16, const void* b_bf16, int64_t L, int64_t r,
                                     const int32_t* ids, const float* scales, void* out_bf16, int64_t ldo, void* ws,
                                     size_t ws_bytes, fp8_stream_t stream);

/* Static, human-readable name of a status code. Never NULL. */
const char* fp8_status_string(fp8_status status);

#ifdef __cplusplus
}
#endif

#endif /* FP8W8A8_H */
