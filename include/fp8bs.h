/*
 * fp8bs.h -- C ABI of libfp8bs: block-scaled FP8 (E4M3), MXFP8 and per-row /
 * per-tensor FP8 weight quantization, the W8A16 GEMV / skinny GEMM /
 * prefill GEMM that consumes it, the W8A8 route (dynamic per-tensor
 * activation quantization + e4m3 x e4m3 GEMM), the grouped MoE GEMV with
 * its routing and the weighted sum of the experts' outputs, FP8
 * E4M3 and 4-bit paged KV caches with split-KV decode attention, the norm and
 * rotation of q and k on their way there, the step's paging plan, token log
 * probabilities and sampling, for NVIDIA GB300 (sm_103a).
 *
 * Common conventions
 * ------------------
 *  - Every pointer argument is a DEVICE pointer owned by the caller; the
 *    library never allocates, frees or keeps a pointer after the call
 *    returns ("The BF16 source is the caller's to free -- this does not take
 *    ownership", Atlas spark_model/weight_map/quantize_fp8_bs.rs).
 *  - Matrices are row-major with the last index contiguous:
 *      weight w   bf16  [n, k]   (n = output features, k = input features)
 *      codes      e4m3  [n, k]   one byte per weight
 *      scales     fp32  [ceil(n/128), ceil(k/128)]   one per 128x128 tile
 *      e8m0       uint8 [n, ceil(k/32)]              one per 32 k of a row
 *      row scales fp32  [n] (per row) or [1] (per tensor)
 *      x          bf16  [m, k]
 *      y          bf16  [m, n]
 *  - `stream` is a cudaStream_t (NULL = legacy default stream).  Every call
 *    only enqueues work on `stream` and returns: no host synchronisation, no
 *    allocation, and the kernel choice depends on shapes only, never on
 *    values, so a sequence of calls can be captured into a CUDA graph.
 *  - Arguments are validated before anything is enqueued; on a negative
 *    status nothing was launched.  Launch failures report FP8BS_ERR_CUDA.
 *  - Inputs must be finite (no NaN or Inf); results for non-finite inputs
 *    are unspecified.
 *  - Results are deterministic: for a given shape the reduction order is
 *    fixed.
 */
#ifndef FP8BS_H
#define FP8BS_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FP8BS_OK = 0,
    FP8BS_ERR_NULL = -1,    /* a required pointer is NULL                     */
    FP8BS_ERR_SHAPE = -2,   /* n, k or m out of range                         */
    FP8BS_ERR_BLOCK = -3,   /* block size other than 128                      */
    FP8BS_ERR_ALIGN = -4,   /* pointer not aligned to its element size        */
    FP8BS_ERR_CUDA = -5,    /* a CUDA runtime/driver call or launch failed    */
    FP8BS_ERR_DEVICE = -6,  /* a kernel gave up a bounded wait (see below)    */
    FP8BS_ERR_PATH = -7     /* the requested kernel path cannot take the call */
} fp8bs_status;

/* Kernel paths for the *_ex entry points. */
typedef enum {
    FP8BS_PATH_AUTO = 0,     /* choose by shape (what fp8bs_gemv does)         */
    FP8BS_PATH_DECODE = 1,   /* TMA-staged skinny kernel, m <= 32 per launch
                                (larger m runs in chunks of 32 rows)          */
    FP8BS_PATH_PREFILL = 2,  /* tcgen05 tensor-core kernel (block / row / tensor
                                scales, MXFP8)                               */
    FP8BS_PATH_GENERIC = 3   /* plain-load kernel for any shape / alignment    */
} fp8bs_path;

/*
 * fp8bs_quantize -- load-time requantization of a bf16 [n, k] weight to FP8
 * E4M3 codes with one fp32 scale per 128x128 tile.
 *
 * Defined by: Atlas spark_model/weight_map/quantize_fp8_bs.rs
 * (quantize_to_fp8_blockscaled: [n, k] bf16 in, one byte per weight, one f32
 * per [128,128] tile laid out [n_blocks, k_blocks], n > 0 && k > 0 required,
 * launch grid [k_blocks, n_blocks]); FreeToken PR #636 "opt-in fp8-block QAT
 * for the lm_head" (How it works: quantize to fp8 with a 128-block scale
 * after load); FreeToken issue #624 (amax/448).
 *
 * For each tile (bn, bk), over the tile's real elements only (edge tiles may
 * be partial): amax = max|w|, s = amax / 448 as an IEEE fp32 division, s = 1
 * when amax = 0; codes[r, c] = e4m3(w[r, c] / s) with the quotient an IEEE
 * fp32 division, rounded to nearest-even and saturated to +-448.
 *
 *   w_bf16      device, n*k bf16, 2-byte aligned
 *   n, k        > 0 (else FP8BS_ERR_SHAPE)
 *   block       must be 128, the tile edge the consumers hard-code
 *               (else FP8BS_ERR_BLOCK)
 *   codes_u8    device, n*k bytes, written
 *   scales_f32  device, ceil(n/128)*ceil(k/128) floats, 4-byte aligned
 *   stream      cudaStream_t
 * Any alignment is accepted; 16-byte-aligned w with k % 8 == 0 takes the
 * vectorised kernel, everything else a scalar kernel with identical results.
 */
int fp8bs_quantize(const void *w_bf16, int64_t n, int64_t k, int block,
                   uint8_t *codes_u8, float *scales_f32, void *stream);

/*
 * fp8bs_gemv -- decode-time W8A16 block-FP8 linear:
 *   y[i, j] = bf16_rn( sum_kb s[j/128, kb] * sum_{c in kb} x[i, c] * dec(q[j, c]) )
 * with fp32 accumulation.  dec(q) is exact in bf16; the scale multiplies the
 * fp32 partial sum of each 128-wide K block (it is never folded into a
 * rounded bf16 weight).
 *
 * Defined by: InfiniLM PR #586 (Summary: 128x128 block-FP8 W8A16 weights run
 * without materialising bf16 weights; decode routing by M); FreeToken PR #389
 * (the decode GEMV micro-benchmark over M = 1/8/16, and testing the op
 * against a linear on the dequantized weight); FreeToken PR #636 (the fp8
 * lm_head served by the block-FP8 GEMV).
 *
 *   x_bf16   device, m*k bf16, 2-byte aligned
 *   m        >= 0; m == 0 is a no-op returning FP8BS_OK
 *   codes    device, n*k bytes from fp8bs_quantize
 *   scales   device, fp32 [ceil(n/128), ceil(k/128)], 4-byte aligned
 *   n, k     > 0
 *   y_bf16   device, m*n bf16, written (must not overlap the inputs)
 * Shape-only dispatch (FP8BS_PATH_AUTO): m <= 32 -> decode kernel; larger m
 * -> tcgen05 prefill kernel; k % 16 != 0 or unaligned (non-16-byte) x/codes
 * -> generic kernel.
 */
int fp8bs_gemv(const void *x_bf16, int64_t m, const uint8_t *codes,
               const float *scales, int64_t n, int64_t k, void *y_bf16,
               void *stream);

/* fp8bs_gemv with an explicit kernel path (fp8bs_path).  A path that cannot
 * take the call (e.g. DECODE with k % 16 != 0) returns FP8BS_ERR_PATH. */
int fp8bs_gemv_ex(const void *x_bf16, int64_t m, const uint8_t *codes,
                  const float *scales, int64_t n, int64_t k, void *y_bf16,
                  int path, void *stream);

/*
 * fp8bs_gemv_ws -- fp8bs_gemv with caller-provided device scratch, for the
 * decode path (m <= 32, k % 16 == 0, 16-byte aligned x and codes): a first
 * kernel writes an f16 copy of x with one power-of-two factor per (row,
 * 128-column K block) -- the largest |x| of the block moved into
 * [2^14, 2^15), every x within 2^-31 of it converting exactly -- into the
 * workspace, and the GEMV reads it in place of x: e4m3 codes then enter the
 * tensor cores as f16 (one conversion per code pair) at every m, where
 * fp8bs_gemv decodes to bf16 above m = 8.  The result obeys the same
 * definition and tolerance as fp8bs_gemv; the factor's inverse multiplies
 * each K block's fp32 partial together with the block scale.
 *
 * Defined by: InfiniLM PR #586 (Notes for Reviewers: 9 <= M <= 32 decode
 * batches on the tensor-core path) for the arithmetic, which is fp8bs_gemv's.
 *
 *   workspace        device, 16-byte aligned, >= fp8bs_gemv_ws_bytes(m, k)
 *                    bytes; its contents on entry do not matter, and it may
 *                    be reused once the call's work on `stream` is done
 *   other arguments  as fp8bs_gemv
 * Calls that do not take the decode path (m > 32: tensor-core prefill;
 * unaligned or k % 16 != 0: generic kernel) ignore the workspace.
 * FP8BS_ERR_NULL / FP8BS_ERR_ALIGN / FP8BS_ERR_SHAPE for a missing,
 * misaligned or too small workspace, before anything is launched.
 *
 * fp8bs_gemv_ws_bytes: bytes of workspace fp8bs_gemv_ws needs for m rows
 * of x with k columns (0 for m = 0), or FP8BS_ERR_SHAPE.  Host only.
 */
int64_t fp8bs_gemv_ws_bytes(int64_t m, int64_t k);
int fp8bs_gemv_ws(const void *x_bf16, int64_t m, const uint8_t *codes,
                  const float *scales, int64_t n, int64_t k, void *y_bf16,
                  void *workspace, int64_t workspace_bytes, void *stream);

/*
 * fp8bs_gemv_noalloc -- fp8bs_gemv_ws without a caller workspace, for
 * callers that cannot allocate device memory: a plugin whose host framework
 * owns all device memory through its own pool, a real-time loop that cannot
 * afford cudaMalloc / cudaFree (cudaFree synchronises the device), or a C
 * caller with nowhere to keep a buffer.  The scratch fp8bs_gemv_ws would
 * take from the caller (the f16 copy of x and its per-block factors) comes
 * from a fixed array of FP8BS_NOALLOC_SCRATCH_BYTES in the library's own
 * device memory; the call allocates and frees nothing.
 *
 * Defined by: no passage of the source pages has a counterpart; the
 * arithmetic and tolerance are fp8bs_gemv's (fp8bs_gemv_ws's).
 *
 *   arguments  as fp8bs_gemv (x, codes, scales, y are the caller's)
 *   returns    FP8BS_ERR_SHAPE, before anything is launched, when the
 *              decode path would need more scratch than the array holds:
 *              fp8bs_gemv_ws_bytes(m, k) > FP8BS_NOALLOC_SCRATCH_BYTES
 *              (2 MiB: m = 32 with k up to 32,256).  Calls that do not take
 *              the decode path (m > 32, unaligned, k % 16 != 0) need no
 *              scratch and run as fp8bs_gemv.
 * Every device that loads the library holds the array until the process
 * exits.  The first call on each device looks up the array's device address
 * once (cudaGetSymbolAddress, with that device current): make that first
 * call before any stream capture.  Every call shares the one array and
 * leaves its contents behind; each call writes all it reads, so nothing has
 * to be cleared, but calls that overlap on the GPU (different streams, no
 * ordering between them) race on it.  Calls on one stream are ordered.
 */
#define FP8BS_NOALLOC_SCRATCH_BYTES (2 * 1024 * 1024)
int fp8bs_gemv_noalloc(const void *x_bf16, int64_t m, const uint8_t *codes,
                       const float *scales, int64_t n, int64_t k, void *y_bf16,
                       void *stream);

/*
 * mxfp8_quantize -- load-time MXFP8 requantization: per row, per group of 32
 * consecutive k (the last group may be shorter), e = the smallest integer with
 * 448 * 2^e >= amax (i.e. 2^ceil(log2(amax/448))), E = clamp(e + 127, 0, 254)
 * (E = 127 when amax = 0), codes = e4m3(w * 2^(127 - E)) rounded to
 * nearest-even and saturated.
 *
 * Defined by: FreeToken issue #624 "Load-time MXFP8 requantization"
 * (Proposed solution: e4m3 codes with one e8m0 scale per 32 elements, ceil-log2
 * of amax/448, served by a W8A16 path).  This kernel streams bf16 straight to
 * codes; it needs no fp32 staging buffer.
 *
 *   w_bf16       device, n*k bf16, 2-byte aligned
 *   n, k         > 0
 *   codes_u8     device, n*k bytes, written
 *   scales_e8m0  device, n*ceil(k/32) bytes, written
 */
int mxfp8_quantize(const void *w_bf16, int64_t n, int64_t k,
                   uint8_t *codes_u8, uint8_t *scales_e8m0, void *stream);

/*
 * mxfp8_gemv -- W8A16 linear over MXFP8 weights:
 *   y[i, j] = bf16_rn( sum_g 2^(E[j,g]-127) * sum_{c in g} x[i, c] * dec(q[j, c]) )
 * Same argument rules and paths as fp8bs_gemv, with scales_e8m0
 * [n, ceil(k/32)].  Defined by: FreeToken issue #624 (the "mxfp8_linear
 * W8A16 path", which serves every batch size).
 * m > 32 runs on the tensor cores (PREFILL): each group's 2^(E-127) is
 * folded into the exact bf16 decode of its weights, which is exact for
 * every group with 3 <= E (amax >= 2^-116); groups with a smaller E have
 * their scaled weights rounded to bf16's subnormal grid (|error| <= 2^-134
 * per weight).
 */
int mxfp8_gemv(const void *x_bf16, int64_t m, const uint8_t *codes,
               const uint8_t *scales_e8m0, int64_t n, int64_t k, void *y_bf16,
               void *stream);

/* mxfp8_gemv with an explicit path (AUTO, DECODE, PREFILL or GENERIC). */
int mxfp8_gemv_ex(const void *x_bf16, int64_t m, const uint8_t *codes,
                  const uint8_t *scales_e8m0, int64_t n, int64_t k,
                  void *y_bf16, int path, void *stream);

/*
 * fp8bs_gemv_batch / mxfp8_gemv_batch -- a sequence of W8A16 GEMVs with the
 * same m, e.g. the dense projections of every layer of a decode step:
 * the result is that of calling fp8bs_gemv (mxfp8_gemv) on ops[0],
 * ops[1], ..., ops[count-1] in that order on `stream`.
 *
 * Defined by: FreeToken PR #389 (Why: the decode micro-benchmark streams a
 * whole rotation of per-layer projection weights, 48 layers larger than L2,
 * at M = 1/8/16, and times the rotation, not one weight); InfiniLM PR #586
 * (Summary: block-FP8 W8A16 decode without bf16 weights) for the
 * arithmetic, which is fp8bs_gemv's (mxfp8_gemv's) exactly.
 *
 * Runs of consecutive ops that are independent (no op reads or writes the
 * bytes another op of the run writes) and fit the decode kernel (m <= 32,
 * k % 16 == 0, 16-byte aligned x and codes) go to one persistent launch of
 * up to 96 ops, which streams all their weights as one continuous sequence
 * of 128-row tiles instead of paying each GEMV's start-up and tail.  An op
 * that reads or writes an earlier op's output starts a new launch, so it
 * sees that output complete (stream order); ops that the decode kernel
 * cannot take run as their own fp8bs_gemv call in their place in the order.
 * A run too small to fill the GPU (fewer 128-row tiles than half its CTA
 * slots) runs as one launch per op.
 *
 *   ops      host array of count descriptors (read during the call only):
 *              x_bf16  device, m*k bf16      codes  device, n*k e4m3
 *              scales  device: fp32 [ceil(n/128), ceil(k/128)] (block) or
 *                      e8m0 uint8 [n, ceil(k/32)] (MXFP8)
 *              y_bf16  device, m*n bf16, written
 *              n, k    > 0
 *   count    >= 0 (0: no-op); m >= 0 (0: no-op), the same for every op
 * Every op is validated as fp8bs_gemv / mxfp8_gemv validates its arguments
 * before anything is enqueued; the first failure is returned and nothing
 * is launched.  The launches' parameters hold the ops (no device memory is
 * allocated or written besides y), so the call can be captured in a CUDA
 * graph.  _ex: path AUTO as above; DECODE runs every eligible run through the
 * batched kernel whatever its size (FP8BS_ERR_PATH if an op cannot take the
 * decode kernel); PREFILL / GENERIC run every op as fp8bs_gemv_ex
 * (mxfp8_gemv_ex) with that path.
 */
typedef struct fp8bs_gemv_op {
    const void *x_bf16;
    const uint8_t *codes;
    const void *scales;
    void *y_bf16;
    int64_t n, k;
} fp8bs_gemv_op;

int fp8bs_gemv_batch(const fp8bs_gemv_op *ops, int64_t count, int64_t m,
                     void *stream);
int fp8bs_gemv_batch_ex(const fp8bs_gemv_op *ops, int64_t count, int64_t m,
                        int path, void *stream);
int mxfp8_gemv_batch(const fp8bs_gemv_op *ops, int64_t count, int64_t m,
                     void *stream);
int mxfp8_gemv_batch_ex(const fp8bs_gemv_op *ops, int64_t count, int64_t m,
                        int path, void *stream);

/*
 * fp8row_quantize / fp8tensor_quantize -- load-time FP8 with one fp32 scale
 * per output row (scales_f32[n]) or one for the whole weight (scale_f32[1]).
 *
 * Defined by: FreeToken PR #389 "load-time per-tensor FP8 dense projections"
 * (What this adds: each weight quantized to e4m3 with one fp32 scale; Why:
 * the per-row W8A16 route in its decode table).  The scale rule is the tile
 * rule applied to a row / the tensor: amax over its elements, s = amax / 448
 * as an IEEE fp32 division, s = 1 when amax = 0, codes = e4m3(w / s) with an
 * IEEE fp32 quotient, nearest-even, saturated to +-448.
 *
 *   w_bf16      device, n*k bf16, 2-byte aligned
 *   n, k        > 0 (else FP8BS_ERR_SHAPE)
 *   codes_u8    device, n*k bytes, written
 *   scales_f32  device, n floats (per row) / 1 float (per tensor), 4-byte
 *               aligned, written.  The per-tensor form uses its one float as
 *               the amax accumulator before it writes s there, so no other
 *               work may read it until the call has completed on `stream`.
 * Asynchronous on `stream`; allocates nothing.
 */
int fp8row_quantize(const void *w_bf16, int64_t n, int64_t k,
                    uint8_t *codes_u8, float *scales_f32, void *stream);
int fp8tensor_quantize(const void *w_bf16, int64_t n, int64_t k,
                       uint8_t *codes_u8, float *scale_f32, void *stream);

/*
 * fp8row_gemv / fp8tensor_gemv -- W8A16 linear over per-row / per-tensor FP8:
 *   y[i, j] = bf16_rn( s_j * sum_c x[i, c] * dec(q[j, c]) )
 * with the sum in fp32 and s_j = scales[j] (per row) or scale[0] (per
 * tensor), applied once to the fp32 sum.  Same argument rules, paths and
 * errors as fp8bs_gemv, with the scale arrays of the quantizers above.
 * Defined by: FreeToken PR #389 (Why: the per-row W8A16 route of the decode
 * micro-benchmark over M = 1/8/16).
 */
int fp8row_gemv(const void *x_bf16, int64_t m, const uint8_t *codes,
                const float *scales, int64_t n, int64_t k, void *y_bf16,
                void *stream);
int fp8row_gemv_ex(const void *x_bf16, int64_t m, const uint8_t *codes,
                   const float *scales, int64_t n, int64_t k, void *y_bf16,
                   int path, void *stream);
int fp8tensor_gemv(const void *x_bf16, int64_t m, const uint8_t *codes,
                   const float *scale, int64_t n, int64_t k, void *y_bf16,
                   void *stream);
int fp8tensor_gemv_ex(const void *x_bf16, int64_t m, const uint8_t *codes,
                      const float *scale, int64_t n, int64_t k, void *y_bf16,
                      int path, void *stream);

/*
 * fp8bs_moe_gemv -- grouped block-FP8 W8A16 GEMV over routed experts:
 *   y[t, j, :] = x[t, :] . dequant(W[e])^T  with e = expert_ids[t, j],
 * each expert a block-FP8 weight [n, k] (fp8bs_quantize), the num_experts
 * weights stored back to back: codes [num_experts, n, k], scales
 * [num_experts, ceil(n/128), ceil(k/128)].  Every expert any token selected
 * is streamed once per call (whatever the number of its tokens); experts no
 * token selected are not read.  Same arithmetic and tolerance as fp8bs_gemv.
 *
 * Defined by: Atlas spark_model/weight_map/quantize_fp8_bs.rs (module
 * notes: the block-scaled quantizer exists for routed MoE experts; the
 * grouped MoE GEMM reads [N/128, K/128] fp32 block scales; decode reads the
 * top-12 of 256 experts per token).
 *
 *   x_bf16       device, m*k bf16, 16-byte aligned, k % 16 == 0
 *   expert_ids   device, m*topk int32; ids of one token must be distinct
 *                (a token listing an expert twice gets only its lowest such
 *                slot written and sets the device error word); an id
 *                outside [0, num_experts) selects nothing and sets the
 *                device error word (fp8bs_check_device_error)
 *   topk         1..num_experts;  num_experts 1..1024, num_experts*n < 2^31
 *   y_bf16       device, m*topk*n bf16, written for every valid id
 * The ids are read on the device (no host synchronisation); m > 32 runs in
 * chunks of 32 tokens.  FP8BS_ERR_PATH if k % 16 != 0 or x / codes are not
 * 16-byte aligned.
 */
int fp8bs_moe_gemv(const void *x_bf16, int64_t m, const int32_t *expert_ids,
                   int64_t topk, const uint8_t *codes, const float *scales,
                   int64_t num_experts, int64_t n, int64_t k, void *y_bf16,
                   void *stream);

/*
 * fp8bs_moe_gemv_ws -- fp8bs_moe_gemv with caller-provided device scratch,
 * for batches of m > 32 tokens: four small kernels group the (token, slot)
 * pairs by expert in the workspace (counts, prefix sums, the pairs expert by
 * expert, and a copy of each pair's x row in that order), then each selected
 * expert's weight is multiplied with exactly the x rows routed to it and
 * each output row written to its (token, slot).  With at most 32 pairs per
 * expert on average (m * topk <= 32 * num_experts) the decode kernel streams
 * each expert once per tile of up to 32 of its pairs, on an f16 copy of the
 * x rows with one power-of-two factor per (row, 128-column K block), as
 * fp8bs_gemv_ws prepares x (every x within 2^-31 of its block's largest
 * |x| converts exactly; the codes enter the tensor cores as f16); otherwise one grouped
 * GEMM on the 5th-generation tensor cores (the weight decoded to bf16 in
 * shared memory) runs tiles of up to 128 pairs of one expert (a deeper
 * pipeline) while the experts average at most 128 pairs, else of up to
 * 256.  Every
 * selected expert's weight is read once per tile of its pairs;
 * fp8bs_moe_gemv instead runs the decode kernel per 32 tokens, reading
 * every selected expert once per 32 tokens.
 * Same definition, arguments and tolerance as fp8bs_moe_gemv; m <= 32
 * takes fp8bs_moe_gemv's decode path and ignores the workspace.  In the
 * grouped path a token that lists an expert twice has both slots computed.
 *
 * Defined by: Atlas spark_model/weight_map/quantize_fp8_bs.rs (module
 * notes: the grouped MoE GEMM over block-FP8 routed experts with
 * [N/128, K/128] fp32 scales).
 *
 *   workspace        device, 256-byte aligned, >= fp8bs_moe_gemv_ws_bytes(m,
 *                    topk, num_experts, k) bytes (0 for m <= 32; about
 *                    2 * m * topk * k for the x copy, plus the factors);
 *                    contents on entry do not matter
 *   other arguments  as fp8bs_moe_gemv (m * topk < 2^31)
 * FP8BS_ERR_NULL / FP8BS_ERR_ALIGN / FP8BS_ERR_SHAPE for a missing,
 * misaligned or too small workspace, before anything is launched.
 */
int64_t fp8bs_moe_gemv_ws_bytes(int64_t m, int64_t topk, int64_t num_experts,
                                int64_t k);
int fp8bs_moe_gemv_ws(const void *x_bf16, int64_t m, const int32_t *expert_ids,
                      int64_t topk, const uint8_t *codes, const float *scales,
                      int64_t num_experts, int64_t n, int64_t k, void *y_bf16,
                      void *workspace, int64_t workspace_bytes, void *stream);

/*
 * fp8bs_moe_route -- which experts each token goes to and with which weights,
 * from the router's logits x: the ids that fp8bs_moe_gemv takes, on the device.
 *   s_e = softmax(x)_e (FP8BS_SCORE_SOFTMAX) or 1 / (1 + e^-x_e) (FP8BS_SCORE_SIGMOID)
 *   c_e = s_e + bias_e
 * The experts stand in `groups` groups of equal size, one after the other; a
 * group's score is the sum of the group_top (1 or 2) largest c in it, the
 * topk_groups groups with the highest scores are open, and of their experts
 * the topk with the largest c are chosen, largest first:
 *   expert_ids[t, j],  weights[t, j] = scale * s_e,  divided by the sum of the
 *   chosen s where renormalize is not 0 (0 where that sum is 0).
 * Equals go to the lowest index.  c and groups' scores are compared in multiples
 * of 2^-44 (each c within two of them, whatever its bias; biases taken as at most
 * 65536 in magnitude); without a bias experts are compared by x itself, which is
 * the same order.  Weights within 2^-18 of themselves; e^-|x| below 2^-126 counts as 0.
 *
 * Defined by: no passage of the source pages has a counterpart (Atlas
 * spark_model/weight_map/quantize_fp8_bs.rs: decode reads the top-12 of 256
 * experts per token, with the choice as given).
 *
 *   logits       device, [num_tokens, num_experts] bf16, or fp32 if logits_f32 is
 *                non-zero, rows row_stride elements apart (>= num_experts, or 0:
 *                one row for every token); aligned to its element size.  -inf
 *                shuts an expert out of the softmax (all of them: s = 0).  An
 *                expert whose c is NaN, by its logit or its bias, comes after
 *                every other, a group with one among its group_top best after
 *                every group without; the ids are distinct and in range
 *                whatever the logits and the biases
 *   num_experts  1..1024;  topk 1..32, <= topk_groups * num_experts / groups
 *   bias         device, [num_experts] fp32, or NULL
 *   groups       1..32, a divisor of num_experts;  topk_groups 1..groups;
 *                group_top 1 or 2, <= num_experts / groups
 *   expert_ids   device, [num_tokens, topk] int32, written
 *   weights      device, [num_tokens, topk] fp32, written
 */
#define FP8BS_SCORE_SOFTMAX 0
#define FP8BS_SCORE_SIGMOID 1
int fp8bs_moe_route(const void *logits, int logits_f32, int64_t row_stride,
                    int64_t num_tokens, int64_t num_experts, int64_t topk,
                    int scoring, const float *bias, int64_t groups,
                    int64_t topk_groups, int64_t group_top, int renormalize,
                    float scale, int32_t *expert_ids, float *weights,
                    void *stream);

/*
 * fp8bs_moe_combine -- the experts' outputs y [num_tokens, topk, n]
 * (fp8bs_moe_gemv's) brought together:
 *   out[t, :] = bf16_rn( residual[t, :] + sum_j weights[t, j] * y[t, j, :] )
 * summed in fp32 in the order of j, from the residual on.
 *
 * Defined by: no passage of the source pages has a counterpart; y is that of
 * Atlas' grouped MoE GEMM (spark_model/weight_map/quantize_fp8_bs.rs).
 *
 *   y_bf16       device, [num_tokens, topk, n] bf16
 *   weights      device, [num_tokens, topk] fp32
 *   expert_ids   device, [num_tokens, topk] int32, or NULL; a slot whose id is
 *                outside [0, num_experts) adds nothing, and its y, which
 *                fp8bs_moe_gemv does not write, is not read
 *   residual_bf16  device, [num_tokens, n] bf16, or NULL (0)
 *   topk         1..1024
 *   out_bf16     device, [num_tokens, n] bf16, written; may be residual_bf16
 * Any alignment of 2 bytes; 16-byte aligned tensors with n % 8 == 0 are read
 * 16 bytes at a time, with the same results.
 */
int fp8bs_moe_combine(const void *y_bf16, const float *weights,
                      const int32_t *expert_ids, int64_t num_experts,
                      const void *residual_bf16, int64_t num_tokens,
                      int64_t topk, int64_t n, void *out_bf16, void *stream);

/*
 * FP8 E4M3 KV cache for paged decode attention.
 *
 * Defined by: InfiniLM PR #586 (Summary: an F8 cache with per-layer fp32
 * k_scale / v_scale for paged attention; Benchmark: split-KV decode
 * attention over the FP8 cache, "halves cache capacity and decode attention
 * read bandwidth").
 *
 * Cache layout: [num_blocks, page_size, num_kv_heads, head_dim] e4m3, token
 * i of sequence b in block block_table[b * max_blocks_per_seq +
 * i / page_size] at offset i % page_size.  head_dim must be 128, page_size a
 * multiple of 16, num_q_heads a multiple of num_kv_heads with at most 8
 * query heads per kv head.
 *
 * fp8kv_append: cache[slot_mapping[t]] = e4m3(x[t] / scale) for the new
 * tokens x [num_tokens, num_kv_heads, head_dim] bf16 (IEEE fp32 quotient,
 * nearest-even, saturating); slot = block * page_size + offset;
 * num_slots = num_blocks * page_size.  A slot outside [0, num_slots) is
 * skipped and sets the device error word.  x 16-byte aligned.
 */
int fp8kv_append(const void *x_bf16, int64_t num_tokens, int64_t num_kv_heads,
                 int64_t head_dim, const int32_t *slot_mapping,
                 const float *scale, uint8_t *cache, int64_t num_slots,
                 void *stream);

/*
 * fp8kv_decode_attention: one query token per sequence,
 *   o[b, h, :] = sum_l p_l * dec(V[l, g]) * v_scale,
 *   p = softmax_l( sm_scale * q[b, h, :] . dec(K[l, g]) * k_scale ),
 * g = h / (num_q_heads / num_kv_heads), over the seq_lens[b] tokens of
 * sequence b (0 tokens: o = 0).  K and V decode exactly; scores, the
 * softmax and the sums are fp32 (the weights enter the V sum as f16); one
 * bf16 rounding at the end.  The KV range of a sequence is split over a
 * thread-block cluster and merged on chip (no workspace).
 *
 *   q_bf16       device, [batch, num_q_heads, 128] bf16, 16-byte aligned
 *   k_cache, v_cache   device, e4m3 caches as above, 16-byte aligned
 *   k_scale, v_scale   device, 1 float each
 *   block_table  device, [batch, max_blocks_per_seq] int32
 *   seq_lens     device, [batch] int32, each <= max_blocks_per_seq * page_size
 *                (a larger or negative length is clamped and sets the device
 *                error word, as does a block id outside [0, num_blocks))
 *   max_seq_len  host upper bound of seq_lens (sizes the split), <=
 *                max_blocks_per_seq * page_size
 *   out_bf16     device, [batch, num_q_heads, 128] bf16, written
 */
int fp8kv_decode_attention(const void *q_bf16, const uint8_t *k_cache,
                           const uint8_t *v_cache, const float *k_scale,
                           const float *v_scale, const int32_t *block_table,
                           int64_t max_blocks_per_seq, const int32_t *seq_lens,
                           int64_t batch, int64_t num_q_heads,
                           int64_t num_kv_heads, int64_t head_dim,
                           int64_t page_size, int64_t num_blocks,
                           int64_t max_seq_len, float sm_scale, void *out_bf16,
                           void *stream);

/*
 * fp8act_quantize -- dynamic per-tensor activation quantization for the
 * W8A8 route: the per-tensor rule applied to x [m, k] (amax over all m*k
 * elements, s = amax / 448 in fp32, s = 1 if all zero, codes = e4m3(x / s)
 * with an IEEE fp32 quotient).  Up to 65536 elements run as one single-CTA
 * launch (amax and cast fused; the per-call cost dominates at decode sizes),
 * larger tensors as the grid-wide fp8tensor_quantize, bit for bit the same.
 *
 * Defined by: FreeToken PR #389 (What this adds: a dynamic per-tensor
 * activation scale, an amax pass then the cast; the follow-up commit: a
 * block-parallel partial amax plus a reduce and cast for large inputs).
 *
 *   x_bf16     device, m*k bf16
 *   codes_u8   device, m*k bytes, written
 *   scale_f32  device, 1 float, written (used as the amax accumulator by
 *              the grid-wide form, see fp8tensor_quantize)
 */
int fp8act_quantize(const void *x_bf16, int64_t m, int64_t k,
                    uint8_t *codes_u8, float *scale_f32, void *stream);

/*
 * w8a8_gemm -- W8A8 linear:
 *   y[i, j] = bf16_rn( sx * sw * sum_c dec(qx[i, c]) * dec(qw[j, c]) )
 * with e4m3 x e4m3 products (exact) summed in fp32 on the tensor cores.
 *
 * Defined by: FreeToken PR #389 (What this adds / Why: the per-tensor W8A8
 * GEMM of the projections, raw scaled-mm row of its decode table).
 *
 *   x_codes   device, m*k e4m3 (fp8act_quantize), 16-byte aligned for the
 *             TMA paths
 *   x_scale   device, 1 float
 *   w_codes   device, n*k e4m3 (fp8tensor_quantize), w_scale device, 1 float
 *   y_bf16    device, m*n bf16, written
 * Paths: m <= 32 -> DECODE (mma.sync e4m3, m > 32 in chunks of 32 rows);
 * larger m -> PREFILL (tcgen05 kind::f8f6f4); k % 16 != 0 or unaligned
 * codes -> GENERIC.  Errors as fp8bs_gemv.
 */
int w8a8_gemm(const uint8_t *x_codes, int64_t m, const float *x_scale,
              const uint8_t *w_codes, const float *w_scale, int64_t n,
              int64_t k, void *y_bf16, void *stream);
int w8a8_gemm_ex(const uint8_t *x_codes, int64_t m, const float *x_scale,
                 const uint8_t *w_codes, const float *w_scale, int64_t n,
                 int64_t k, void *y_bf16, int path, void *stream);

/*
 * fp8bs_kv_plan -- the paging plan of one serving step, built on the device
 * from request lengths (no host synchronisation): which new cache blocks
 * each request gets, and where each of the step's new tokens goes.  Serves
 * the FP8 cache (fp8kv_append) and the 4-bit cache (fp4kv_append) alike.
 *
 * Defined by: no passage of the source pages has a counterpart (InfiniLM PR
 * #586 takes the slot map and the block table as given).  With
 * c = ctx_lens[b] cached and n = new_lens[b] new tokens of request b,
 * P = page_size:
 *   cu_new[b + 1] = cu_new[b] + n, cu_new[0] = 0   (the step's token axis)
 *   have = ceil(c / P), need = ceil((c + n) / P) - have
 *   the `need` new blocks are free_blocks[h], free_blocks[h + 1], ... with
 *     h = *free_head + (the needs of the requests before b); they are stored
 *     at block_table[b][have ...]
 *   token cu_new[b] + i: requests = b, positions = c + i,
 *     slots = block of (c + i) * P + (c + i) % P
 *   seq_lens[b] = c + n;  *free_head_out = *free_head + (blocks handed out)
 * Entries of the token arrays past cu_new[batch] are -1.
 *
 * A request is refused -- seq_lens[b] = c, its tokens keep their places on
 * the token axis with positions and slots -1, it takes no block -- when the
 * free list has run out for it (blocks are handed out in request order, so
 * every later request that needs a block is refused too; sets
 * bit 5 of the device error word), or when its lengths cannot be: c or n
 * negative, c + n > max_blocks_per_seq * page_size, cu_new[b + 1] >
 * num_tokens (sets bit 4; seq_lens[b] is c clamped to the table's range).
 * Nothing of a refused request's tokens is stored, but cu_new counts them:
 * attention that is given cu_new and seq_lens takes their rows for the last n
 * of the c cached tokens, so what it writes there means nothing.  Give up the
 * results of tokens whose slot is -1, and offer the tokens again once there
 * are blocks.  A
 * block id outside [0, num_blocks) gives slots -1 (a free-list id also a
 * table entry -1) and sets bit 4, as does a *free_head outside
 * [0, num_free], for which every request that needs a block is refused.
 *
 *   ctx_lens, new_lens   device, [batch] int32 (n = 0: nothing new)
 *   batch                0..16384 (0: only cu_new, the token arrays and the head)
 *   block_table          device, [batch, max_blocks_per_seq] int32; entries
 *                        below `have` are read, the new ones written
 *   free_blocks          device, [num_free] int32 (may be NULL if num_free is 0)
 *   free_head            device, 1 int32: blocks of the list already taken.
 *                        A finished request's k blocks come back by writing
 *                        their ids to free_blocks[head - k .. head - 1] and
 *                        head - k to the head, between steps on the stream
 *   page_size            1..65536, num_blocks * page_size < 2^31
 *   num_tokens           size of the token arrays (>= the step's tokens)
 *   seq_lens             device, [batch] int32, written; may be ctx_lens
 *   cu_new               device, [batch + 1] int32, written
 *   slots, positions, requests   device, [num_tokens] int32, written
 *   free_head_out        device, 1 int32, written; may be free_head
 * No other two arrays may overlap.
 */
int fp8bs_kv_plan(const int32_t *ctx_lens, const int32_t *new_lens,
                  int64_t batch, int32_t *block_table,
                  int64_t max_blocks_per_seq, const int32_t *free_blocks,
                  int64_t num_free, const int32_t *free_head,
                  int64_t page_size, int64_t num_blocks, int64_t num_tokens,
                  int32_t *seq_lens, int32_t *cu_new, int32_t *slots,
                  int32_t *positions, int32_t *requests,
                  int32_t *free_head_out, void *stream);

/*
 * 4-bit KV cache for paged attention: e2m1 codes with one e4m3 scale per 16
 * elements and one fp32 scale per layer, 0.28 of the bytes of bf16.
 *
 * Defined by: no passage of the source pages has a counterpart; the paging,
 * the per-layer fp32 k_scale / v_scale and the attention are those of
 * InfiniLM PR #586's FP8 cache, the group format the element and block-scale
 * formats of the 4-bit float type (e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6).
 *
 * Cache layout, K and V each: uint8 [num_blocks, num_kv_heads,
 * page_size / 16, 9 * head_dim]; a tile of 16 tokens of one kv head is its
 * codes [16, head_dim / 2] (element 2j in the low nibble of byte j), then its
 * scales [16, head_dim / 16].  The value of an element is code * scale * s.
 * Token i of sequence b is in block block_table[b][i / page_size] at offset
 * i % page_size.  head_dim is 64 or 128, page_size a multiple of 16 up to
 * 4096, num_kv_heads < 4096, num_blocks * page_size < 2^31.
 *
 * fp4kv_append: for each token t and group of 16 elements x of k[t] (v[t]),
 *   scale = e4m3(fl32(amax / fl32(6 s))), den = fl32(s * scale),
 *   code = e2m1(fl32(x / den)), code = 0 where den = 0
 * (nearest-even, saturating), stored at slot slots[t] = block * page_size +
 * offset.  A group with NaN in it is stored as a NaN scale: all of it reads
 * as NaN.  Slot -1 stores nothing (padding, refused requests); any other
 * slot outside [0, num_blocks * page_size) stores nothing and sets the
 * device error word (bit 4).  Two tokens of one call may not share a slot.
 *
 *   k_bf16, v_bf16     device, [num_tokens, num_kv_heads, head_dim] bf16,
 *                      16-byte aligned, tokens k_stride (v_stride) elements
 *                      apart, a multiple of 8 (e.g. rows of a fused
 *                      projection)
 *   slots              device, [num_tokens] int32
 *   k_scale, v_scale   device, 1 positive float each (amax / 2688 of the
 *                      layer's keys or values uses the whole range)
 *   k_cache, v_cache   device, 16-byte aligned, written at the slots
 */
int fp4kv_append(const void *k_bf16, int64_t k_stride, const void *v_bf16,
                 int64_t v_stride, int64_t num_tokens, int64_t num_kv_heads,
                 int64_t head_dim, const int32_t *slots, const float *k_scale,
                 const float *v_scale, uint8_t *k_cache, uint8_t *v_cache,
                 int64_t page_size, int64_t num_blocks, void *stream);

/*
 * fp4kv_gather: the tokens at slots[t] of a 4-bit cache in bf16, e.g. a
 * cached prefix for a dense prompt attention:
 *   k_bf16[t] = bf16(fl32(code * scale * s))   (code * scale is exact)
 * [num_tokens, num_kv_heads, head_dim], contiguous, 16-byte aligned.  Slot
 * -1 gives zeros; any other slot out of range too, with bit 4 of the device
 * error word.  Defined by: the cache above.
 */
int fp4kv_gather(const uint8_t *k_cache, const uint8_t *v_cache,
                 const int32_t *slots, int64_t num_tokens,
                 int64_t num_kv_heads, int64_t head_dim, int64_t page_size,
                 int64_t num_blocks, const float *k_scale,
                 const float *v_scale, void *k_bf16, void *v_bf16,
                 void *stream);

/*
 * fp8kv_rope_append / fp4kv_rope_append: the rows of a fused q, k, v
 * projection made ready for the attention in one pass: each query and key head
 * normed and rotated by its token's position, q written out in bf16, k and v
 * written into the paged cache (the FP8 cache of fp8kv_append, the 4-bit cache
 * of fp4kv_append).  Of a head vector a with norm weights w, each fl one fp32
 * rounding:
 *   r = fl(1 / sqrt(mean a^2 + eps)),  n_i = fl(fl(a_i * r) * w_i)
 * (n = a where the weights are NULL; where they are not |a| is below 2^50 and
 * mean a^2 + eps at least 2^-100: beyond, r may be off by more than its rounding,
 * and NaN from |a| = 2^60 on or below a sum of 2^-126); of a pair (n1, n2) with the
 * cos c and the sin s of the token's position:
 *   o1 = fl(fl(n1 * c) - fl(n2 * s)),  o2 = fl(fl(n2 * c) + fl(n1 * s))
 * over the first rot_dim elements, the others o = n.  q_out = bf16(o), where a
 * query's squares are summed in plain fp32, so that next to a border between two
 * bf16 numbers it may be either; k is stored as o is by the cache's own rule
 * (e4m3(fl(o / k_scale)), or the group rule of fp4kv_append with x = o), v as the
 * append stores it.
 *
 * Defined by: no passage of the source pages has a counterpart for the norm
 * and the rotation; the FP8 cache and its scales are InfiniLM PR #586's.
 *
 *   q_bf16, k_bf16, v_bf16   device, [num_tokens, heads, head_dim] bf16, 16-byte
 *                aligned, tokens *_stride elements apart, a multiple of 8
 *   head_dim     128; fp4kv_rope_append 64 too
 *   positions    device, [num_tokens] int32; a token at -1 (padding, a refused
 *                request) stores nothing and leaves its row of q_out as it was,
 *                one outside [-1, max_pos) too, with bit 4 of the device error word
 *   slots        device, [num_tokens] int32, as fp4kv_append: slot -1 stores
 *                nothing, any other one out of range too, with bit 4 (q_out is
 *                written).  Two tokens of one call may not share a slot
 *   cos_sin      device, [max_pos, rot_dim] fp32, 16-byte aligned: the cos of a
 *                position's rot_dim / 2 pairs, then the sin
 *   rot_dim      16..head_dim, a multiple of 16
 *   interleaved  0: pair j is elements j and j + rot_dim / 2; else 2j and 2j + 1
 *   q_weight, k_weight   device, [head_dim] bf16, 16-byte aligned, or NULL
 *   eps          >= 0, finite (with eps = 0 a head of zeros gives NaN)
 *   q_out        device, [num_tokens, num_q_heads, head_dim] bf16, 16-byte aligned;
 *                may be q_bf16 itself where q_stride is num_q_heads * head_dim
 *   k_scale, v_scale   device, 1 positive float each
 *   k_cache, v_cache   device, 16-byte aligned, written at the slots
 */
int fp8kv_rope_append(const void *q_bf16, int64_t q_stride, const void *k_bf16,
                      int64_t k_stride, const void *v_bf16, int64_t v_stride,
                      int64_t num_tokens, int64_t num_q_heads,
                      int64_t num_kv_heads, int64_t head_dim,
                      const int32_t *positions, const int32_t *slots,
                      const float *cos_sin, int64_t max_pos, int64_t rot_dim,
                      int interleaved, const void *q_weight,
                      const void *k_weight, float eps, void *q_out,
                      const float *k_scale, const float *v_scale,
                      uint8_t *k_cache, uint8_t *v_cache, int64_t num_slots,
                      void *stream);
int fp4kv_rope_append(const void *q_bf16, int64_t q_stride, const void *k_bf16,
                      int64_t k_stride, const void *v_bf16, int64_t v_stride,
                      int64_t num_tokens, int64_t num_q_heads,
                      int64_t num_kv_heads, int64_t head_dim,
                      const int32_t *positions, const int32_t *slots,
                      const float *cos_sin, int64_t max_pos, int64_t rot_dim,
                      int interleaved, const void *q_weight,
                      const void *k_weight, float eps, void *q_out,
                      const float *k_scale, const float *v_scale,
                      uint8_t *k_cache, uint8_t *v_cache, int64_t page_size,
                      int64_t num_blocks, void *stream);

/*
 * fp4kv_decode_attention: attention of the newest tokens of each sequence
 * over its 4-bit cache (one per sequence when decoding; several when drafted
 * tokens are verified or a short prompt chunk is appended).  The keys of the
 * query tokens themselves are already in the cache.  For query token i of
 * the n_q of sequence b, at position p = seq_lens[b] - n_q + i:
 *   o[i, h, :] = sum_l w_l * dec(V[l, g]),
 *   w = softmax_l(sm_scale * q[i, h, :] . dec(K[l, g])),
 *   lse[i, h] = log sum_l exp(sm_scale * q[i, h, :] . dec(K[l, g]))
 * over keys l <= p (with window > 0: p - window < l <= p),
 * g = h / (num_q_heads / num_kv_heads).  A row that sees no key gives o = 0,
 * lse = -inf.  A row takes nothing from a key that it does not see, whatever
 * is stored there; NaN that it does see goes the formula's way: in q or a key
 * to the whole row and its lse, in a value to the elements of its group.
 * K and V decode exactly to f16 (code * scale); q enters as f16, each row
 * brought to the type's range by a power of two, which is exact for elements
 * down to 2^-31 of the row's largest; scores, the softmax and all
 * sums are fp32 (the weights enter the V sum as f16, held against the running
 * maximum so that 2^-39 of it is the smallest); one bf16 rounding at the end.
 *
 * Defined by: InfiniLM PR #586 (Benchmark: split-KV decode attention over
 * the paged cache) for the decode form; several query tokens, the window and
 * lse have no counterpart there.
 *
 *   q_bf16       device, [num_q_tokens, num_q_heads, head_dim] bf16, 16-byte
 *                aligned, tokens q_stride elements apart, a multiple of 8
 *   cu_q         device, [batch + 1] int32: sequence b's query tokens are
 *                cu_q[b] .. cu_q[b + 1] - 1 (fp8bs_kv_plan's cu_new; the rows
 *                of a request that it refused mean nothing), at most max_q of
 *                them; NULL: one per sequence, num_q_tokens = batch.
 *                A range outside [0, num_q_tokens] or longer than max_q is
 *                skipped (its rows are not written) and sets bit 4 of the
 *                device error word.  Rows of no sequence are not written
 *   k_scale, v_scale   device, 1 float each
 *   block_table  device, [batch, max_blocks_per_seq] int32; the tokens of an
 *                id outside [0, num_blocks) are left out and bit 4 is set
 *   seq_lens     device, [batch] int32, 0..max_seq_len (clamped, bit 4)
 *   max_seq_len  host upper bound of seq_lens, <= max_blocks_per_seq * page_size
 *   max_q        host upper bound of the query tokens of a sequence, >= 1
 *   out_bf16     device, [num_q_tokens, num_q_heads, head_dim] bf16,
 *                16-byte aligned, written
 *   lse          device, [num_q_tokens, num_q_heads] fp32, written, or NULL
 *   workspace    device, 16-byte aligned, >= fp4kv_attention_ws_bytes(head_dim)
 *                bytes: the partial results of sequences split over CTAs, and
 *                counters of their arrival in its first
 *                FP4KV_WORKSPACE_COUNTER_BYTES, which have to be zero before
 *                its first use; every call leaves them zero.  Calls that
 *                overlap on the GPU need one each
 * The split of the work follows the lengths on the device: results are
 * deterministic for given shapes and lengths.
 */
#define FP4KV_WORKSPACE_COUNTER_BYTES 1280
int64_t fp4kv_attention_ws_bytes(int64_t head_dim);
int fp4kv_decode_attention(const void *q_bf16, int64_t q_stride,
                           const int32_t *cu_q, int64_t num_q_tokens,
                           int64_t max_q, const uint8_t *k_cache,
                           const uint8_t *v_cache, const float *k_scale,
                           const float *v_scale, const int32_t *block_table,
                           int64_t max_blocks_per_seq, const int32_t *seq_lens,
                           int64_t batch, int64_t num_q_heads,
                           int64_t num_kv_heads, int64_t head_dim,
                           int64_t page_size, int64_t num_blocks,
                           int64_t max_seq_len, int64_t window,
                           float sm_scale, void *out_bf16, float *lse,
                           void *workspace, int64_t workspace_bytes,
                           void *stream);

/*
 * fp8bs_token_logprobs -- log probabilities of given tokens over rows of
 * logits (e.g. fp8bs_gemv's lm_head output), with each row's entropy and top
 * alternatives, reading the logits once:
 *   lse = log sum_j exp(x_j),  logprobs[r] = x_target - lse,
 *   entropy[r] = -sum_j p_j log p_j (nats),  p_j = exp(x_j - lse),
 *   top_ids[r, :], top_logprobs[r, :] = the first `top` tokens of the row in
 *   the order of value, highest first, then index, lowest first, and x - lse.
 * All sums in fp32.  Logits may be -inf (masked tokens: p = 0, log
 * probability -inf); a row of nothing but -inf gives logprob -inf, entropy 0
 * and the tokens 0 .. top - 1 with -inf.  A row with NaN or +inf gives
 * unspecified values (ids stay within [0, vocab) or are -1).
 *
 * Defined by: no passage of the source pages has a counterpart (FreeToken PR
 * #636 serves the lm_head whose logits these are).
 *
 *   logits        device, [rows, vocab], rows row_stride elements apart
 *                 (>= vocab, or 0: one row for every target); bf16, or
 *                 fp32 if logits_f32 is non-zero; aligned to its element size
 *   targets       device, [rows] int32; a negative target gives logprob 0,
 *                 one >= vocab too, with bit 4 of the device error word
 *   top           0..32, <= vocab (0: top_ids and top_logprobs may be NULL)
 *   logprobs, entropy        device, [rows] fp32, written
 *   top_ids, top_logprobs    device, [rows, top] int32 / fp32, written
 */
int fp8bs_token_logprobs(const void *logits, int logits_f32,
                         int64_t row_stride, int64_t rows, int64_t vocab,
                         const int32_t *targets, int64_t top, float *logprobs,
                         float *entropy, int32_t *top_ids,
                         float *top_logprobs, void *stream);

/*
 * fp8bs_sample_tokens -- the next token of each row of logits x (e.g.
 * fp8bs_gemv's lm_head output), drawn with given random numbers:
 *   w_j = exp((x_j - max x) / T);  tokens stand in the order of value, highest
 *   first, then index, lowest first; kept are the first of them that all allow:
 *     top_k (> 0):  the first top_k,
 *     top_p (< 1):  the fewest whose mass reaches top_p times that of the
 *                   first top_k (of all without top_k); one at least,
 *     min_p (> 0):  those with w_j >= min_p (> 1 counts as 1);
 *   block b of 1024 tokens (1024 b .. 1024 b + 1023): the first one for which the kept mass
 *     of the blocks to it exceeds u[r, 0] times the kept mass of all,
 *   tokens[r] = the first kept token of the block for which the kept mass of
 *     the block to it exceeds u[r, 1] times that of the block,
 *   logprobs[r] = log(w_token / kept mass), the log probability of the draw.
 * Two numbers a row, because one fp32 number in steps of 2^-24 cannot give
 * 152064 tokens their probabilities, and the borders of as many tokens on
 * one line would be moved by every rounding of a sum.  T = 0 is greedy (the
 * first token, log probability 0).  Masses are whole multiples of 2^-41 of the
 * largest weight: what is below half of that may count as nothing.  What rounds is
 * a weight (2^-22 of itself, or half a step of the histogram that finds a cut) and
 * a block's sum in fp32: a first number or a top_p nearer than 2^-17 of itself
 * (a top_p over more than 2^18 tokens 2^-16) to a border may fall to either side;
 * as a rule what is further than 2^-21 does not.
 *
 * Defined by: no passage of the source pages has a counterpart (FreeToken PR
 * #636 serves the lm_head whose logits these are).
 *
 *   logits        device, [rows, vocab], rows row_stride elements apart
 *                 (>= vocab, or 0: one row for every draw); bf16, or fp32
 *                 if logits_f32 is non-zero; aligned to its element size
 *   vocab         1..1048576
 *   u             device, [rows, 2] fp32 in [0, 1] (others are taken as the nearer end, NaN as 0)
 *   temperature   device, [rows] fp32: 0, or 1e-30..1e30; NULL: 1
 *   top_k         device, [rows] int32, <= 0 or >= vocab: off; NULL: off
 *   top_p, min_p  device, [rows] fp32; NULL: off
 *   tokens        device, [rows] int32, written
 *   logprobs      device, [rows] fp32, written, or NULL
 * A row of nothing but -inf gives token -1 and log probability 0.  So does one
 * with NaN or +inf, or with a temperature out of range or a NaN setting, which
 * also sets bit 4 of the device error word.
 */
int fp8bs_sample_tokens(const void *logits, int logits_f32, int64_t row_stride,
                        int64_t rows, int64_t vocab, const float *u,
                        const float *temperature, const int32_t *top_k,
                        const float *top_p, const float *min_p,
                        int32_t *tokens, float *logprobs, void *stream);

/* Path FP8BS_PATH_AUTO would take for these shapes and pointers
 * (host-only, launches nothing).  `mx` selects the MXFP8 GEMV; the block,
 * per-row and per-tensor GEMVs share the same paths (mx = 0). */
int fp8bs_select_path(int64_t m, int64_t n, int64_t k, const void *x_bf16,
                      const void *codes, int mx);

/* Human-readable text for a status code (static storage).
 * Defined by: no passage of the source pages (library infrastructure). */
const char *fp8bs_strerror(int status);

/*
 * Debug query: every wait inside the pipelined kernels is bounded; a kernel
 * that gives up sets a device-side error word instead of hanging.  This
 * synchronises `stream`, copies the word to *word_out (may be NULL), clears
 * it, and returns FP8BS_ERR_DEVICE if it was non-zero, else FP8BS_OK (or
 * FP8BS_ERR_CUDA if the synchronisation itself failed).
 *
 * Defined by: no passage of the source pages (library infrastructure: the
 * bounded waits' failure report).  Beyond a status, the call hands back the
 * word itself (word_out) so that a caller can tell a wait expiry
 * (bits 0-3) from a bad index argument (bit 4) and from a free list that
 * ran out (bit 5).
 */
int fp8bs_check_device_error(void *stream, uint32_t *word_out);

/*
 * Debug: exercise the give-up path of the bounded waits without a fault.
 * Launches one thread on `stream` that waits, with the same bounded wait the
 * pipelined kernels use, on a barrier nothing completes; after the bound
 * (about 2 s) it sets the FULL_WAIT bit (1) of the device error word and
 * returns, leaving the context usable.  Reads and writes no caller memory.
 * Returns FP8BS_OK once launched (FP8BS_ERR_CUDA if the launch failed);
 * fp8bs_check_device_error then reports FP8BS_ERR_DEVICE.
 *
 * Defined by: no passage of the source pages; this is the library's own
 * test hook for its failure detection.
 */
int fp8bs_debug_wait_expiry(void *stream);

/*
 * Debug: the e4m3 encode step that every quantizer here applies to its
 * fp32 quotients (round to nearest even, saturating to +-448, the sign kept
 * on zero results), run on consecutive binary32 bit patterns:
 * codes_u8[i] = e4m3(the float whose bits are first_bits + i), 0 <= i < count.
 *
 *   first_bits  first binary32 bit pattern
 *   count       > 0, a multiple of 4, first_bits + count <= 2^32
 *   codes_u8    device, count bytes, 4-byte aligned (written)
 *
 * Codes for NaN or Inf patterns are unspecified.  Asynchronous on `stream`.
 * Returns FP8BS_ERR_NULL, FP8BS_ERR_SHAPE or FP8BS_ERR_ALIGN before any
 * launch, FP8BS_ERR_CUDA if the launch failed.
 *
 * Defined by: the rounding of the block quantizer's codes (Atlas
 * spark_model/weight_map/quantize_fp8_bs.rs, one e4m3 byte per weight;
 * FreeToken PR #636, How it works: fp8 with a 128-block scale).  A test
 * hook so that the encode step can be compared with an independent encoder
 * over every finite binary32 value.
 */
int fp8bs_debug_encode_f32(uint32_t first_bits, int64_t count, uint8_t *codes_u8, void *stream);

/* ABI version (major * 100 + minor). */
int fp8bs_version(void);

#ifdef __cplusplus
}
#endif
#endif /* FP8BS_H */
