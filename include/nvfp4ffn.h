/*
 * nvfp4ffn.h -- C ABI of libnvfp4ffn.so: NVFP4 weight-only SwiGLU FFN decode
 * on one NVIDIA GB300 (sm_103a).
 *
 *   out[M, H] = down( act( gate(x) ) * up(x) ),   M = 1..16 per kernel pass
 *   (up to 64 rows per call, in passes of 16),
 *   x, out BF16;  gate [I, H], up [I, H], down [H, I] NVFP4;  act = SiLU | GeLU-tanh.
 *
 * Beside it: a LoRA delta overlay on the same FFN, the FFN and GEMV on
 * block-scaled FP8 weights (the w8a16 calls), the attention side of a
 * decode layer (norm, rotary positions, 8-bit paged cache, attention), and
 * products for many rows on activations quantised to 4 bits, dense and by
 * expert (the w4a4 and experts calls; near the end of this header).
 *
 * What the calls restate (Atlas engine pages):
 *  - "spark_model/layers/dense_ffn.rs", module doc comment: the dense SwiGLU
 *    FFN, the gated product of the gate and up projections of x fed to the
 *    down projection, with the weights dequantised inside the dot product.
 *  - same page, doc comment of DenseFfnLayer::ensure_int8_weight: an NVFP4
 *    projection is packed E2M1 codes [N, K/2], one E4M3 scale per 16 K
 *    elements [N, K/16], and one FP32 `weight_scale_2` per tensor.
 *  - same page, DenseFfnLayer::forward: the decode FFN as a dual gate+up GEMV
 *    followed by the activation and a down GEMV; forward_km / forward_k2 /
 *    forward_k3: the same for M verify rows, each weight read once for all M.
 *  - same page, DenseFfnLayer::ensure_nvfp4_mmq_weight: a load-time repack of
 *    the checkpoint NVFP4 into a kernel layout that is a raw bit shuffle of the
 *    same codes and scale bytes.
 *  - "spark_model/weight_loader/qwen35_dense.rs", load_layers: BF16/FP32
 *    weights become NVFP4 at load time through a global-absmax kernel and a
 *    quantize kernel (quantize_to_nvfp4).
 *
 * Conventions for every call:
 *  - Pointers marked (device) are device pointers owned by the caller; the
 *    library never frees them and keeps no reference after the call returns.
 *  - Calls are asynchronous on `stream` unless marked "synchronises".
 *  - The return value is a status; nothing aborts or throws across the ABI.
 *    Argument errors are detected on the host before any launch; a failed
 *    launch is reported as NVFP4_ERR_CUDA with the CUDA error left readable
 *    through cudaGetLastError().
 *  - BF16 tensors are row-major with a row stride equal to their width.
 *  - Device pointers must be 16-byte aligned.
 *  - Every GEMV/FFN pass (up to 16 rows) reads its weights once and sums
 *    split-K partials in a fixed order, so results are bit-reproducible.
 *  - The GEMV/FFN and LoRA kernels use programmatic dependent launch: they
 *    may start while the preceding kernel on `stream` is still finishing and
 *    begin reading their (repacked) weights or adapter matrices at once; they
 *    read x and write every output only after that kernel has completed.  So
 *    the weight and adapter buffers must not be written by the kernel issued
 *    immediately before the call on the same stream.  This library's
 *    quantise and repack calls are safe predecessors (their blocks fence
 *    their stores before exiting).
 *  - The GEMV/FFN kernels launch one block per SM.  With 4 or more token rows
 *    a launch may finish its split row blocks cooperatively: its blocks then
 *    wait for one another, which assumes that every block of the launch can
 *    be resident at once.  Two such calls overlapping on the GPU (issued on
 *    different streams or from different threads or processes sharing the
 *    SMs) can each hold SMs that the other's blocks need; their waits then
 *    give up after about a second and the call reports NVFP4_ERR_TIMEOUT
 *    (nvfp4_workspace_status).  Issue the calls for one device on one stream,
 *    or order the streams with events.
 */
#ifndef NVFP4FFN_H
#define NVFP4FFN_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    NVFP4_OK = 0,
    NVFP4_ERR_NULL = 1,      /* a required pointer is NULL */
    NVFP4_ERR_SHAPE = 2,     /* a size is <= 0, or K/H/I is not a multiple of 16 */
    NVFP4_ERR_ALIGN = 3,     /* a device pointer is not 16-byte aligned */
    NVFP4_ERR_RANGE = 4,     /* M outside the call's range, or an unknown enum value */
    NVFP4_ERR_WORKSPACE = 5, /* workspace smaller than the size query returns */
    NVFP4_ERR_CUDA = 6,      /* a CUDA runtime call or launch failed */
    NVFP4_ERR_TIMEOUT = 7,   /* a kernel gave up on a bounded wait (device status word) */
    NVFP4_ERR_ALIAS = 8      /* input and output buffers overlap */
} nvfp4_status;

/* Gating nonlinearity (enum FfnActivation on the dense-FFN page).
 * SiLU(t) = t / (1 + e^-t); GeLU-tanh(t) = 0.5 t (1 + tanh(sqrt(2/pi)(t + 0.044715 t^3))). */
typedef enum { NVFP4_ACT_SILU = 0, NVFP4_ACT_GELU_TANH = 1 } nvfp4_act;

/* Element type of the weight handed to nvfp4_quantize. */
typedef enum { NVFP4_SRC_F32 = 0, NVFP4_SRC_BF16 = 1 } nvfp4_src_dtype;

/* ------------------------------------------------------------------ quantise */

/* Bytes of scratch nvfp4_quantize needs (a few words; independent of N, K). */
size_t nvfp4_quantize_scratch_bytes(int N, int K);

/*
 * Quantise a weight W [N, K] (row-major, fp32 or bf16, device) to NVFP4 in the
 * canonical checkpoint layout ("spark_model/weight_loader/qwen35_dense.rs",
 * load_layers: global absmax, then quantize):
 *   amax   = max |W|;  scale2 = amax / 2688 (= 6 * 448), or 1 when amax == 0
 *   per 16-element block b of a row:  s_b = E4M3(bamax_b / 6 / scale2)
 *   per element:  code = E2M1(w / (E4M3value(s_b) * scale2))   (code 0 with
 *   the element's sign when s_b == 0)
 * in IEEE fp32 with that operation order; both conversions round to nearest,
 * ties to even, saturate at the largest finite value and keep the sign.
 *   codes  (device, out) u8 [N, K/2]: element 2j in the low nibble of byte j.
 *   scales (device, out) u8 [N, K/16]: E4M3 ("fn": bias 7, max 448).
 *   scale2_out (host, out): the per-tensor FP32 scale.  A device copy is left
 *   at byte offset 4 of `scratch`.
 *   scratch (device) >= nvfp4_quantize_scratch_bytes(N, K).
 * Requirements: N >= 1, K >= 16, K % 16 == 0, W finite.
 * Synchronises `stream` (it reads scale2 back to the host): a load-time call.
 */
nvfp4_status nvfp4_quantize(const void* w, nvfp4_src_dtype dtype, int N, int K,
                            uint8_t* codes, uint8_t* scales, float* scale2_out,
                            void* scratch, size_t scratch_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------ repack */

/*
 * Kernel layout ("fragment layout"): a byte permutation of the canonical codes
 * and scales (the principle of DenseFfnLayer::ensure_nvfp4_mmq_weight: same
 * codes, same scale bytes, no numerics), zero-padded to N' = roundup(N, 256)
 * rows and K' = roundup(K, 256) columns.  For N % 256 == 0 and K % 256 == 0 it
 * holds exactly the canonical byte count N*K*9/16.  The layout is opaque to
 * callers; nvfp4_unpack inverts it.
 */
size_t nvfp4_repacked_bytes(int N, int K);

/* codes [N, K/2], scales [N, K/16] (device, canonical) -> packed (device,
 * nvfp4_repacked_bytes(N, K) bytes).  N >= 1, K % 16 == 0. */
nvfp4_status nvfp4_repack(const uint8_t* codes, const uint8_t* scales, int N, int K,
                          void* packed, cudaStream_t stream);

/* Gate and up projections ([I, H] each) interleaved so that one kernel reads
 * gate row n and up row n together: 2 * nvfp4_repacked_bytes(I, H) bytes. */
size_t nvfp4_repacked_gate_up_bytes(int I, int H);
nvfp4_status nvfp4_repack_gate_up(const uint8_t* gate_codes, const uint8_t* gate_scales,
                                  const uint8_t* up_codes, const uint8_t* up_scales,
                                  int I, int H, void* packed, cudaStream_t stream);

/* Inverse of nvfp4_repack (a test and inspection aid): packed -> canonical
 * codes [N, K/2] and scales [N, K/16] (device). */
nvfp4_status nvfp4_unpack(const void* packed, int N, int K, uint8_t* codes,
                          uint8_t* scales, cudaStream_t stream);

/* ------------------------------------------------------------------ GEMV */

/*
 * Workspace bytes for nvfp4_gemv on the current device (cross-CTA partial
 * sums and their counters); 0 for invalid sizes or N > 524288.
 * Workspace contract (all GEMV/FFN calls): zero-fill the workspace once after
 * it is allocated (cudaMemset or nvfp4_workspace_init).  Every call that
 * completes normally leaves it ready for the next one, whatever the next
 * call's entry point and shape, provided the workspace is large enough for
 * that call.  Calls sharing one workspace must be ordered (one stream).
 */
size_t nvfp4_gemv_workspace_bytes(int M, int N, int K);

/*
 * One NVFP4 projection (the w4a16 decode GEMV of "spark_model/layers/
 * dense_ffn.rs", DenseFfnLayer::forward / forward_km):
 *   y[m, n] = bf16( scale2 * sum_k x[m, k] * E2M1(c[n, k]) * E4M3(s[n, k/16]) )
 *   x (device) bf16 [M, K];  packed_w (device) from nvfp4_repack(N, K);
 *   y (device, out) bf16 [M, N];  ws (device) >= nvfp4_gemv_workspace_bytes.
 * Requirements: 1 <= M <= 64, N >= 1, K >= 16, K % 16 == 0, x and y disjoint.
 * Accumulation is fp32 on exactly dequantised weights; every x row is scaled
 * by a power of two into the fp16 operand range, so any finite bf16 x works.
 * The kernels take up to 16 token rows at a time: M > 16 (a verify batch or a
 * small prefill, the page's forward_prefill range M <= 64) runs as groups of
 * 16 rows and a remainder, each group streaming the weights once.
 */
nvfp4_status nvfp4_gemv(const void* x, int M, int K, const void* packed_w, float scale2,
                        int N, void* y, void* ws, size_t ws_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------ FFN */

/* Workspace bytes for ffn_swiglu_nvfp4 on the current device: the bf16
 * activation h [M, I] plus the partial sums of both kernels (0 for invalid
 * sizes or I + H above about 524288).  Contract as for nvfp4_gemv. */
size_t ffn_swiglu_nvfp4_workspace_bytes(int M, int H, int I);

/* Byte offset inside an ffn_swiglu_nvfp4 workspace of the bf16 activation
 * h [M, I] (row-major) that the call leaves there (an inspection aid). */
size_t ffn_swiglu_nvfp4_hidden_offset(void);

/*
 * The decode FFN (DenseFfnLayer::forward and forward_km on the dense-FFN
 * page), in two launches:
 *   1. g = bf16(gate_scale2 * gate.x),  u = bf16(up_scale2 * up.x),
 *      h = bf16(act(g) * u)                      [M, I] bf16, in ws
 *   2. out = bf16(down_scale2 * down.h)          [M, H] bf16
 *   x (device) bf16 [M, H];  gate_up_packed (device) from
 *   nvfp4_repack_gate_up(I, H);  down_packed (device) from nvfp4_repack(H, I);
 *   out (device, out) bf16 [M, H];  ws (device) >= ffn_swiglu_nvfp4_workspace_bytes.
 * Requirements: 1 <= M <= 64, H and I >= 16 and multiples of 16, x and out
 * disjoint, act a nvfp4_act value.  M > 16 runs in groups of 16 rows, as for
 * nvfp4_gemv.
 */
nvfp4_status ffn_swiglu_nvfp4(const void* x, int M, int H, int I,
                              const void* gate_up_packed, float gate_scale2, float up_scale2,
                              const void* down_packed, float down_scale2, nvfp4_act act,
                              void* out, void* ws, size_t ws_bytes, cudaStream_t stream);

/* Workspace bytes for ffn_gate_up_nvfp4 on the current device (zero-fill once). */
size_t ffn_gate_up_nvfp4_workspace_bytes(int M, int H, int I);

/*
 * The gate/up half of the FFN alone (step 1 of ffn_swiglu_nvfp4; the fused
 * dual GEMV + activation of DenseFfnLayer::forward on the dense-FFN page):
 *   h[m, i] = bf16( act(bf16(gate_scale2 * gate.x)) * bf16(up_scale2 * up.x) )
 *   x (device) bf16 [M, H];  gate_up_packed (device) from nvfp4_repack_gate_up;
 *   h (device, out) bf16 [M, I];  ws (device) >= ffn_gate_up_nvfp4_workspace_bytes.
 * A caller that adds its own terms to h (an adapter) finishes the layer with
 * nvfp4_gemv on the down projection.  Requirements as for ffn_swiglu_nvfp4.
 */
nvfp4_status ffn_gate_up_nvfp4(const void* x, int M, int H, int I, const void* gate_up_packed,
                               float gate_scale2, float up_scale2, nvfp4_act act, void* h,
                               void* ws, size_t ws_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------ LoRA overlay */

/*
 * The adapter overlay of the dense-FFN page (DenseFfnLayer::apply_lora_gate_up
 * and apply_lora_down): gate and up take dW x after their projections and
 * before the activation, the output takes dW h after the down projection,
 * contracted over the activation h.  dW = B A with A [r, in] and B [out, r]
 * bf16 row-major (device), 1 <= r <= 64; any alpha/r is folded into B.  Each
 * intermediate is bf16: xa = bf16(A v), d = bf16(B xa), base = bf16(base + d).
 */

/* Workspace bytes for ffn_swiglu_nvfp4_lora (the FFN's plus the adapter
 * intermediates); contract as for nvfp4_gemv. */
size_t ffn_swiglu_nvfp4_lora_workspace_bytes(int M, int H, int I, int rank);

/*
 * ffn_swiglu_nvfp4 with the overlay:
 *   g = bf16(bf16(gate_scale2 * gate.x) + bf16(Bg bf16(Ag x)))   (likewise u)
 *   h = bf16(act(g) * u),  out = bf16(bf16(down_scale2 * down.h) + bf16(Bd bf16(Ad h)))
 * gate_a [r, H] / gate_b [I, r], up_a [r, H] / up_b [I, r], down_a [r, I] /
 * down_b [H, r] (device, bf16); a pair given as two NULL pointers is absent
 * (its delta is zero).  A pair with one NULL pointer is NVFP4_ERR_NULL; rank
 * outside [1, 64] is NVFP4_ERR_RANGE.  Other arguments and requirements as
 * ffn_swiglu_nvfp4, except 1 <= M <= 16.  Up to four small launches join the
 * FFN's two.
 */
nvfp4_status ffn_swiglu_nvfp4_lora(const void* x, int M, int H, int I,
                                   const void* gate_up_packed, float gate_scale2,
                                   float up_scale2, const void* down_packed,
                                   float down_scale2, nvfp4_act act, int rank,
                                   const void* gate_a, const void* gate_b, const void* up_a,
                                   const void* up_b, const void* down_a, const void* down_b,
                                   void* out, void* ws, size_t ws_bytes, cudaStream_t stream);

/* Scratch bytes for nvfp4_lora_apply (fp32 partial sums of a v over K slices;
 * independent of K). */
size_t nvfp4_lora_apply_scratch_bytes(int M, int rank);

/*
 * The page's apply_lora_delta on its own: base[m][n] = bf16(base[m][n] +
 * bf16(sum_j b[n][j] xa[m][j])) with xa = bf16(a v):  v (device) bf16 [M, K],
 * a [rank, K], b [N, rank] (device, bf16), base (device, in/out) bf16 [M, N],
 * scratch (device) >= nvfp4_lora_apply_scratch_bytes.  1 <= M <= 16, K even,
 * v and base disjoint.
 */
nvfp4_status nvfp4_lora_apply(const void* v, int M, int K, const void* a, const void* b,
                              int rank, int N, void* base, void* scratch, size_t scratch_bytes,
                              cudaStream_t stream);

/*
 * ffn_swiglu_nvfp4 (1 <= M <= 16) for callers that cannot allocate device
 * memory where they run the FFN (a process that reserves the device's memory for its own pool at
 * start-up and forbids later cudaMalloc, or code that must not risk the
 * implicit device synchronisation of an allocation).  The pages have no
 * counterpart of this call; it exists for such callers.
 *   Same arguments and results as ffn_swiglu_nvfp4, without ws/ws_bytes: the
 *   workspace is one library-owned device array of 24 MiB, held by every GPU
 *   that loads the library until the process exits.  Shapes whose
 *   ffn_swiglu_nvfp4_workspace_bytes exceeds 24 MiB are rejected with
 *   NVFP4_ERR_WORKSPACE (M = 16 at H = 5376, I = 21504 needs about 21 MiB).
 *   Every argument is checked before anything is touched: a rejected call
 *   changes nothing on the device.
 *   The first call on each device (with that device current) resolves the
 *   array's device address (cudaGetSymbolAddress) and zero-fills the array on
 *   `stream`, synchronising it; make that first call before any stream
 *   capture.  Later calls only enqueue the two FFN kernels on `stream`: like
 *   ffn_swiglu_nvfp4's workspace, the array is left ready for the next call by
 *   every call that completes normally.  The call allocates nothing.
 *   Every call shares the one array, so calls that overlap on the GPU
 *   (different streams without ordering between them) race and corrupt each
 *   other's results.
 *   A call whose kernel abandoned a bounded wait is reported only by
 *   nvfp4_noalloc_status, which also repairs the array; until it is called,
 *   later calls may return wrong results.
 */
nvfp4_status ffn_swiglu_nvfp4_noalloc(const void* x, int M, int H, int I,
                                      const void* gate_up_packed, float gate_scale2,
                                      float up_scale2, const void* down_packed, float down_scale2,
                                      nvfp4_act act, void* out, cudaStream_t stream);

/*
 * Status of ffn_swiglu_nvfp4_noalloc calls on the current device, the
 * counterpart of nvfp4_workspace_status for the library's fixed array (no
 * counterpart on the pages).  Synchronises `stream`, reads and clears the
 * array's status word: NVFP4_OK, or NVFP4_ERR_TIMEOUT when a kernel abandoned
 * a bounded wait since the last check, in which case the whole array is
 * zero-filled again (on `stream`, synchronised) so the next call starts clean.
 * Performs the first-call set-up if no call has yet run on this device.
 */
nvfp4_status nvfp4_noalloc_status(cudaStream_t stream);

/* ------------------------------------------------------ block-scaled FP8 (w8a16) */

/*
 * The dense-FFN page's native FP8 arm (DenseFfnWeightsFp8 and set_fp8_weights;
 * the FP8 dispatch of DenseFfnLayer::forward: w8a16_gemv_dual for gate and up,
 * then w8a16_gemv_silu_input for the down projection on the activation),
 * weights used as loaded, with no NVFP4 requantisation.  A projection [N, K]:
 *   codes (device) E4M3 bytes [N, K] row-major, the "fn" variant (0x7F/0xFF
 *         are NaN, outside the contract);
 *   grid  (device) fp32 [ceil(N/128), ceil(K/128)] row-major, 4-byte aligned;
 *   W[n][k] = e4m3(codes[n][k]) * grid[n/128][k/128]  (the block grid the
 *   weight loader's proj_is_fp8_any_scale accepts; a per-tensor scalar scale
 *   is the uniform grid).
 * The roundings are those of the NVFP4 path: g, u, h and out are bf16.  Every
 * call below follows the conventions of its NVFP4 counterpart (status codes,
 * validation before any launch, asynchronous on `stream`, the workspace
 * contract, M up to 64 in groups of 16, K/H/I multiples of 16).
 */

/* Bytes of a repacked FP8 projection [N, K] / gate+up pair [I, H] (0 for
 * invalid sizes): the codes, padded to 256 rows and 256 K, plus one fp32
 * scale per 16 rows and 64 K. */
size_t w8a16_repacked_bytes(int N, int K);
size_t w8a16_repacked_gate_up_bytes(int I, int H);

/* Canonical FP8 -> kernel layout (codes permuted, grid entries copied per
 * 16-row tile and 64-K chunk; no arithmetic).  packed (device, out) >=
 * w8a16_repacked_bytes(N, K), 16-byte aligned. */
nvfp4_status w8a16_repack(const uint8_t* codes, const float* grid, int N, int K, void* packed,
                          cudaStream_t stream);

/* Gate and up [I, H] into one blob (each tile's gate and up codes back to
 * back), >= w8a16_repacked_gate_up_bytes(I, H). */
nvfp4_status w8a16_repack_gate_up(const uint8_t* gate_codes, const float* gate_grid,
                                  const uint8_t* up_codes, const float* up_grid, int I, int H,
                                  void* packed, cudaStream_t stream);

/* Inverse of w8a16_repack (a test aid): codes [N, K] and grid. */
nvfp4_status w8a16_unpack(const void* packed, int N, int K, uint8_t* codes, float* grid,
                          cudaStream_t stream);

/* Workspace bytes for w8a16_gemv; contract as for nvfp4_gemv. */
size_t w8a16_gemv_workspace_bytes(int M, int N, int K);

/*
 * y[m][n] = bf16(sum_k x[m][k] * W[n][k]) for the FP8 projection (the page's
 * w8a16_gemv):  x (device) bf16 [M, K];  packed_w from w8a16_repack(N, K);
 * y (device, out) bf16 [M, N];  ws >= w8a16_gemv_workspace_bytes.
 */
nvfp4_status w8a16_gemv(const void* x, int M, int K, const void* packed_w, int N, void* y,
                        void* ws, size_t ws_bytes, cudaStream_t stream);

/* Workspace bytes for ffn_swiglu_w8a16; h [M, I] lies at
 * ffn_swiglu_nvfp4_hidden_offset() in it, as for ffn_swiglu_nvfp4. */
size_t ffn_swiglu_w8a16_workspace_bytes(int M, int H, int I);

/*
 * The decode FFN on FP8 weights, in two launches:
 *   1. g = bf16(gate.x), u = bf16(up.x), h = bf16(act(g) * u)   [M, I] in ws
 *   2. out = bf16(down.h)                                        [M, H]
 *   gate_up_packed from w8a16_repack_gate_up(I, H); down_packed from
 *   w8a16_repack(H, I); other arguments as ffn_swiglu_nvfp4.
 */
nvfp4_status ffn_swiglu_w8a16(const void* x, int M, int H, int I, const void* gate_up_packed,
                              const void* down_packed, nvfp4_act act, void* out, void* ws,
                              size_t ws_bytes, cudaStream_t stream);

/* ------------------------------------------------------ attention side of a layer */

/*
 * What a decode layer runs beside the projections and the FFN: the norms in
 * front of them, rotary positions, and attention over a paged key/value cache
 * of 8-bit floats.  Conventions as for every call (status codes, validation
 * before any launch, asynchronous on `stream`, 16-byte aligned bf16 and code
 * buffers).  These calls take any number of token rows.  Results are
 * bit-reproducible.  They use programmatic dependent launch where noted, but
 * read no input before the preceding kernel on `stream` has completed.
 */

/*
 * Root-mean-square norm of x + residual, [M, H] bf16:
 *   r = x + residual (fp32; residual may be NULL for none)
 *   sum_out = bf16(r)                        (NULL to leave it out)
 *   y = r * (mean(r^2) + eps)^(-1/2) * (weight + weight_bias),   out = bf16(y)
 * weight (device) bf16 [H].  M >= 1, H a multiple of 16, 16 <= H <= 32768,
 * eps >= 0.  sum_out may be x or residual, and out may be x or residual (not
 * the buffer that sum_out is); other overlaps are NVFP4_ERR_ALIAS.
 */
nvfp4_status add_rmsnorm_bf16(const void* x, const void* residual, const void* weight, int M,
                              int H, float eps, float weight_bias, void* sum_out, void* out,
                              cudaStream_t stream);

/*
 * The same norm into 8 bits: for each row and group of 128 columns (the last
 * one may be shorter) scale = max(amax|y| / 448, 2^-126), or 1 when amax is 0,
 * and code = E4M3(y / scale), to nearest even, saturated, NaN kept (of the
 * quotient rounded to fp32).
 *   codes (device, out) u8 [M, H];  scales (device, out) fp32 [M, ceil(H/128)].
 * Neither overlaps another buffer.
 */
nvfp4_status add_rmsnorm_e4m3(const void* x, const void* residual, const void* weight, int M,
                              int H, float eps, float weight_bias, void* sum_out, uint8_t* codes,
                              float* scales, cudaStream_t stream);

/* How rotary frequencies change for contexts longer than the trained one. */
typedef enum {
    ROPE_PLAIN = 0,  /* f_i = base^(-2i/rot_dim) */
    ROPE_LINEAR = 1, /* f_i / factor */
    ROPE_BASE = 2,   /* base * factor^(rot_dim/(rot_dim-2)) in place of base */
    ROPE_RAMP = 3    /* f_i * (g + (1-g)/factor), g = clamp((turns - slow)/(fast - slow), 0, 1),
                        turns = f_i * context / 2 pi */
} rope_scaling;

/*
 * Table of rotations (a load-time call, fp64 arithmetic):
 *   table (device, out) fp32 [positions, rot_dim/2, 2] = magnitude * (cos, sin)(p * f_i).
 * rot_dim a multiple of 16 up to 256, base > 1; factor > 0 unless ROPE_PLAIN;
 * context > 0 and 0 <= slow < fast for ROPE_RAMP (ignored otherwise).
 */
nvfp4_status rope_table(int positions, int rot_dim, double base, rope_scaling scaling,
                        double factor, double context, double slow, double fast, double magnitude,
                        float* table, cudaStream_t stream);

/*
 * The cache: pages of `page` tokens, each page holding every head of one
 * block of tokens, E4M3 codes with one fp32 scale per page and head:
 *   k[page][head][row][d] = k_scales[page][head] * e4m3(k_codes[page][head][row][d])
 * page a power of two in 16..256, head_dim 64, 128 or 256.  Scales are
 * positive and finite.
 */
typedef struct {
    void* k_codes;   /* (device) u8 [pages, kv_heads, page, head_dim] */
    void* v_codes;   /* (device) the same */
    float* k_scales; /* (device) [pages, kv_heads] */
    float* v_scales; /* (device) the same */
    int pages, kv_heads, page, head_dim;
} kv8_cache;

/*
 * A batch of sequences and their new tokens.  Tokens q_start[b] ..
 * q_start[b+1] - 1 of the call's rows belong to sequence b and take the last
 * positions of its kv_len[b]: with n of them, the i-th has position
 * kv_len[b] - n + i.  Position p lies in page page_table[b][p / page], row
 * p % page.  n may be 0 (the sequence takes no part).  Rows in front of q_start[0]
 * and from q_start[batch] on belong to no sequence: nothing is written or
 * reported for them, so a captured call may have rows to spare.
 * The lists live on the device and are not read by the host.  The kernels
 * check them: a page outside the cache, a length beyond the table, decreasing
 * or too large q_start, n > kv_len or a position beyond the rotation table
 * reads and writes nothing outside the buffers (what it concerns is left out:
 * not written, or masked) and sets the status word.  Where a decreasing q_start
 * gives rows to several sequences, any of them may have written a row, and
 * kv8_attention may leave out the whole batch.
 */
typedef struct {
    const int* q_start;    /* (device) [batch + 1], from 0, not decreasing */
    const int* kv_len;     /* (device) [batch], the new tokens included */
    const int* page_table; /* (device) [batch, table_width] */
    int* status;           /* (device) one word, zeroed once by the caller, or NULL */
    int batch;             /* 1..1024 */
    int table_width;       /* pages a sequence can have; table_width * page < 2^31 - 256 */
} kv8_batch;

/* Synchronises `stream`, reads and clears the batch's status word: NVFP4_OK, or
 * NVFP4_ERR_RANGE when a call met an index outside its buffers since. */
nvfp4_status kv8_batch_status(const kv8_batch* batch, cudaStream_t stream);

/*
 * Writes the batch's new tokens into the cache, with rotary positions:
 *   k, v (device) bf16 [tokens, kv_heads, head_dim], k_stride and v_stride
 *        values between tokens (multiples of 8: views of a fused projection);
 *   rope (device) fp32 [rope_positions, rot_dim/2, 2], or NULL for no rotation:
 *        the first rot_dim values of each head of q and k turn in pairs
 *        (i, i + rot_dim/2), or (2i, 2i+1) when interleaved:
 *        (a cos - b sin, b cos + a sin), in fp32;
 *   q (device) bf16 [tokens, heads, head_dim] with q_stride -> q_out (device,
 *        out) bf16 [tokens, heads, head_dim] contiguous, rotated and rounded;
 *        both NULL to leave q out.  q_out may be q when q is contiguous.
 * For each head of k (rotated, not rounded in between) and v, and each page
 * that gets new tokens:
 *   need  = the smallest 2^e with max|new values| <= 448 * 2^e, e in -60..119
 *   scale = max(old scale, need) when rows in front of the new ones hold
 *           tokens of the page, else need
 *   codes = E4M3(value / scale) (nearest even, saturated, NaN kept; NaN does
 *           not enter the maximum); the older rows' codes are re-scaled by
 *           old scale / scale when it changed.  An old scale that is kept but is
 *           no power of two (it did not come from this call) takes
 *           value * fp32(1 / scale).
 * A page that gets new tokens belongs to one sequence of the batch.
 */
nvfp4_status kv8_append(const kv8_cache* cache, const kv8_batch* batch, int tokens, const void* k,
                        int64_t k_stride, const void* v, int64_t v_stride, const void* q,
                        int64_t q_stride, int heads, void* q_out, const float* rope,
                        int rope_positions, int rot_dim, int interleaved, cudaStream_t stream);

/*
 * Reads the batch's tokens back (the positions that kv8_append with this batch
 * writes; a whole sequence when it has kv_len[b] tokens in the batch):
 *   k_out, v_out (device, out) bf16 [tokens, kv_heads, head_dim] =
 *   bf16(scale * code).
 */
nvfp4_status kv8_read(const kv8_cache* cache, const kv8_batch* batch, int tokens, void* k_out,
                      void* v_out, cudaStream_t stream);

/* Workspace bytes for kv8_attention on the current device, from the sizes alone
 * (the descriptions' pointers may be NULL), 0 for sizes that the call refuses;
 * contract as for nvfp4_gemv (zero-fill once, calls sharing one
 * ordered). */
size_t kv8_attention_workspace_bytes(const kv8_cache* cache, const kv8_batch* batch, int tokens,
                                     int heads);

/*
 * Attention of the batch's tokens over the cache (which holds them already).
 * The query at position p sees key j <= p and, with window > 0, only
 * j > p - window or j < sinks (sinks first tokens stay visible):
 *   s_j = softmax_scale * q . k_j,   out = sum_j softmax(s)_j v_j,
 *   lse = log(sum_j e^(s_j))
 *   q (device) bf16 [tokens, heads, head_dim], q_stride values between tokens
 *        (a multiple of 8); head h reads the cache's head h / (heads/kv_heads);
 *   out (device, out) bf16 [tokens, heads, head_dim] contiguous;
 *   lse (device, out) fp32 [tokens, heads], or NULL;
 *   ws (device) >= kv8_attention_workspace_bytes.
 * A query that sees nothing gets 0 and -infinity.  Masked keys and values do
 * not enter the result, whatever they hold.  Scores, maxima and sums are fp32;
 * softmax_j v_scale_j is rounded to 11 bits before it multiplies v's codes; below
 * 2^-20 of the largest one of its row it has fewer, and below 2^-30 it is lost from
 * out (not from lse).
 * heads a multiple of kv_heads, tokens * heads / kv_heads at most 2^30;
 * window, sinks >= 0 (sinks without a window have no effect).  v_scales below
 * 2^-80 or above 2^126 count as these; those of one sequence's visible keys may
 * differ by up to 2^100 (beyond that a page with the smaller one may be lost from
 * lse too).  A batch of 2^31 or more tiles is left out and reported: a tile is 16
 * keys by 8 to 32 rows (128 by 256 for many rows of up to 128 values) of one kv
 * head, as in 131072 new tokens with 16 query heads on each of 8 kv heads of 256.
 * A kernel that waited for itself longer than its limit leaves wrong outputs and
 * NVFP4_ERR_TIMEOUT for nvfp4_workspace_status on ws.
 */
nvfp4_status kv8_attention(const void* q, int64_t q_stride, int tokens, int heads,
                           const kv8_cache* cache, const kv8_batch* batch, float softmax_scale,
                           int window, int sinks, void* out, float* lse, void* ws, size_t ws_bytes,
                           cudaStream_t stream);

/* ------------------------------------------------------ 4-bit activations (w4a4) */

/*
 * Products for many token rows, on the FP4 tensor cores: activations are
 * quantised to NVFP4 like the weights (the W4A4 prefill path of "spark_model/
 * layers/dense_ffn.rs", forward_prefill_inner: quantize_bf16_to_nvfp4, then
 * w4a4_gemm), dense or grouped by expert.  Other numerics than the calls above,
 * which keep activations in bf16: a user chooses.  These calls take any number of
 * rows up to 2^22 (RANGE beyond), K, H and I multiples of 16 up to 65536, N up to
 * 2^20.  They are asynchronous and use programmatic dependent launch; their results
 * are bit-reproducible.  They read nothing, their weights neither, before the preceding
 * kernel on `stream` has completed, so that kernel may write any of their inputs; and the
 * kernel behind them is not launched before it has.  Blocks of different pairs do not wait
 * for one another, so calls on different streams may overlap if their workspaces (and rows
 * buffers) differ.
 *
 * A row of x [M, K] becomes a scale r per row, one E4M3 scale per 16 values and
 * E2M1 codes (all to nearest, ties to even, saturating):
 *   r    = the smallest 2^e with max|x| <= 2688 * 2^e, e in -100..117; 1 for a row
 *          of zeros, NaN for a row that holds an infinity or a NaN
 *   s_b  = E4M3(max|x_b| / 6 / r)        per block b of 16
 *   code = E2M1(x / (s_b * r))           0 where s_b is 0
 * A row that is not finite gives an output row of NaN and leaves the others as they
 * are.  Sums may be cut along K in another way for another number of rows, so a row's
 * product may differ in the last place between calls of different sizes.
 */

/*
 * Weights in the products' layout: canonical NVFP4 codes [experts, N, K/2] and
 * scales [experts, N, K/16] (nvfp4_quantize's), moved byte by byte, zero-padded to
 * N' = roundup(N, 256) and K' = roundup(K, 256).  experts 1..1024, 1 for a dense
 * weight.  The gate/up pair [experts, I, H] interleaves gate and up (I a multiple
 * of 16; padded to 128 features).  Sizes are 0 where the call refuses.
 */
size_t w4a4_repacked_bytes(int experts, int N, int K);
size_t w4a4_repacked_gate_up_bytes(int experts, int I, int H);
nvfp4_status w4a4_repack(const uint8_t* codes, const uint8_t* scales, int experts, int N, int K,
                         void* packed, cudaStream_t stream);
nvfp4_status w4a4_repack_gate_up(const uint8_t* gate_codes, const uint8_t* gate_scales,
                                 const uint8_t* up_codes, const uint8_t* up_scales, int experts,
                                 int I, int H, void* packed, cudaStream_t stream);
/* Inverse of w4a4_repack (a test and inspection aid). */
nvfp4_status w4a4_unpack(const void* packed, int experts, int N, int K, uint8_t* codes,
                         uint8_t* scales, cudaStream_t stream);

/*
 * Rows that belong to experts: rows start[e] .. start[e+1] - 1 of the call's M to
 * expert e.  start does not decrease; rows in front of start[0] and from
 * start[experts] on belong to none: nothing is read or written for them.  The
 * lists live on the device and are not read by the host.  The products check them:
 * an expert whose rows do not lie in 0..M has none, and where start decreases no
 * expert has any; w4a4_quantize leaves rows out that have no place.
 */
typedef struct {
    const int* start; /* (device) [experts + 1] */
    int experts;      /* 1..1024 */
} w4a4_groups;

/* Bytes of M quantised rows (0 for sizes that the calls refuse); experts as in the
 * groups, 1 without. */
size_t w4a4_rows_bytes(int M, int K, int experts);

/*
 * x (device) bf16 [M, K] -> rows (device, out, w4a4_rows_bytes, opaque).  groups NULL
 * for a dense product.
 */
nvfp4_status w4a4_quantize(const void* x, int M, int K, const w4a4_groups* groups, void* rows,
                           cudaStream_t stream);

/*
 * The rows of a routed batch, tokens * choices of them: x (device) bf16 [tokens, K],
 * each token quantised once and written to the rows of its choices; ids and place
 * (device) int32 [tokens, choices] and groups->start as experts_order has and writes
 * them.  A pair with an id or a place out of range is left out.
 */
nvfp4_status w4a4_quantize_routed(const void* x, int tokens, int K, const int* ids,
                                  const int* place, int choices, const w4a4_groups* groups,
                                  void* rows, cudaStream_t stream);

/* The values that rows stand for: out (device, out) bf16 [M, K] = code * s_b * r, which
 * bf16 holds exactly unless r is near the end of its range (a test and inspection aid). */
nvfp4_status w4a4_dequantize(const void* rows, int M, int K, const w4a4_groups* groups, void* out,
                             cudaStream_t stream);

/* Workspace bytes for the products below on the current device (N features, of a
 * weight or a gate/up pair; experts 1 without groups); contract as for nvfp4_gemv. */
size_t w4a4_gemm_workspace_bytes(int M, int N, int K, int experts);

/*
 * y[m][n] = bf16(r_m * (scale2 * sum_k xc[m][k] xs[m][k/16] wc[n][k] ws[n][k/16])),
 * sums in fp32:  rows from w4a4_quantize(M, K);  packed_w from w4a4_repack(1, N, K);
 * y (device, out) bf16 [M, N].  N may be odd.
 */
nvfp4_status w4a4_gemm(const void* rows, int M, int K, const void* packed_w, float scale2, int N,
                       void* y, void* ws, size_t ws_bytes, cudaStream_t stream);

/* h[m][i] = bf16(act(g) * u) with g, u such products in bf16, of the gate and the up
 * weight: gate_up_packed from w4a4_repack_gate_up(1, I, H); h (device, out) bf16 [M, I]. */
nvfp4_status w4a4_gate_up(const void* rows, int M, int H, const void* gate_up_packed,
                          float gate_scale2, float up_scale2, int I, nvfp4_act act, void* h,
                          void* ws, size_t ws_bytes, cudaStream_t stream);

/* The same with each row's weight that of its expert: packed from w4a4_repack(experts,
 * ...), scale2 (device) fp32 [experts], rows quantised with the same groups. */
nvfp4_status w4a4_experts_gemm(const void* rows, int M, int K, const w4a4_groups* groups,
                               const void* packed_w, const float* scale2, int N, void* y, void* ws,
                               size_t ws_bytes, cudaStream_t stream);
nvfp4_status w4a4_experts_gate_up(const void* rows, int M, int H, const w4a4_groups* groups,
                                  const void* gate_up_packed, const float* gate_scale2,
                                  const float* up_scale2, int I, nvfp4_act act, void* h, void* ws,
                                  size_t ws_bytes, cudaStream_t stream);

/*
 * The FFN on quantised activations: x quantised, h = act(gate(x)) * up(x) in bf16,
 * h quantised, out = down(h).  x (device) bf16 [M, H], out (device, out) bf16 [M, H],
 * not overlapping; ws >= ffn_swiglu_w4a4_workspace_bytes (contract as for nvfp4_gemv).
 */
size_t ffn_swiglu_w4a4_workspace_bytes(int M, int H, int I);
nvfp4_status ffn_swiglu_w4a4(const void* x, int M, int H, int I, const void* gate_up_packed,
                             float gate_scale2, float up_scale2, const void* down_packed,
                             float down_scale2, nvfp4_act act, void* out, void* ws, size_t ws_bytes,
                             cudaStream_t stream);

/*
 * A routed batch in the order of its experts: ids (device) int32 [tokens, choices] are
 * the experts of each token; one outside 0..experts-1 belongs to none (a token of a
 * padded batch).  Pairs (token, choice) are sorted by expert, those of an expert in
 * the order of the list:
 *   start  (device, out) [experts + 1]: each expert's first row, and their end
 *   source (device, out) [tokens * choices]: each row's token, -1 from the end on
 *   place  (device, out) [tokens, choices]: each pair's row, -1 for none
 * choices 1..64, tokens * choices up to 2^22.
 */
nvfp4_status experts_order(const int* ids, int tokens, int choices, int experts, int* start,
                           int* source, int* place, cudaStream_t stream);

/*
 * out[t] = bf16(sum_j weights[t][j] * y[place[t][j]]) in fp32, in the order of j:
 * y (device) bf16 [rows, H], weights (device) fp32 [tokens, choices], out (device,
 * out) bf16 [tokens, H].  A place outside 0..rows-1 adds nothing, whatever its weight.
 */
nvfp4_status experts_sum(const void* y, int rows, const int* place, const float* weights, int tokens,
                         int choices, int H, void* out, cudaStream_t stream);

/*
 * The experts' FFN of a routed batch: experts_order, the rows' FFN (as ffn_swiglu_w4a4,
 * with each expert's weights; its output rows in bf16), experts_sum.  x, out (device)
 * bf16 [tokens, H]; scales (device) fp32 [experts].  A token without an expert gets 0.
 */
size_t experts_swiglu_w4a4_workspace_bytes(int tokens, int choices, int experts, int H, int I);
nvfp4_status experts_swiglu_w4a4(const void* x, int tokens, int H, int I, const int* ids,
                                 const float* weights, int choices, int experts,
                                 const void* gate_up_packed, const float* gate_scale2,
                                 const float* up_scale2, const void* down_packed,
                                 const float* down_scale2, nvfp4_act act, void* out, void* ws,
                                 size_t ws_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------ utilities */

/* Zero-fill a workspace (asynchronous memset on `stream`). */
nvfp4_status nvfp4_workspace_init(void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * Synchronises `stream`, then reads and clears the device status word at the
 * start of a GEMV/FFN workspace: NVFP4_OK, or NVFP4_ERR_TIMEOUT when a kernel
 * abandoned a bounded wait since the last check.  A kernel that gave up may
 * leave the workspace's split-K counters off zero: after NVFP4_ERR_TIMEOUT,
 * zero-fill the workspace again (nvfp4_workspace_init) before reusing it.
 */
nvfp4_status nvfp4_workspace_status(void* ws, cudaStream_t stream);

/* Static, human-readable name of a status code. */
const char* nvfp4_status_string(nvfp4_status status);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4FFN_H */
