// api.cu -- the C ABI (include/fp8bs.h): argument validation and shape-only
// dispatch to the kernels.  Nothing here allocates, synchronises (except the
// explicit debug query) or branches on tensor values.
#include "fp8bs.h"
#include "internal.h"

namespace {

using namespace fp8bs;

constexpr int64_t kDecodeMaxM = 32;   // rows of x per decode launch
constexpr int64_t kMaxDim = 1ll << 31;  // n, k and m must fit int32 for the kernels
// Grouped MoE: the largest average of pairs per expert that runs the GEMM on
// 128-pair tiles (beyond it, 256-pair tiles).  Measured on [2048, 4096]
// experts, top-12, same box: 48 pairs per expert 396 vs 450 us, 96: 229 vs
// 264 and 819 vs 954, 192: 787 vs 632, 384: 708 vs 608 (128 vs 256 pairs).
constexpr int64_t kMoeNarrowAvg = 128;

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? FP8BS_OK : FP8BS_ERR_CUDA; }

// The TMA-staged kernels need 16-byte aligned x and codes with k % 16 == 0
// (TMA row pitch and base address rules).
inline bool tma_ok(int64_t k, const void *x, const void *codes) {
    return (k % 16) == 0 && aligned(x, 16) && aligned(codes, 16);
}

int select_path(int64_t m, int64_t k, const void *x, const void *codes, bool mx) {
    (void)mx;  // MXFP8 takes the same paths (its prefill folds the group scales into the decode)
    if (!tma_ok(k, x, codes)) return FP8BS_PATH_GENERIC;
    if (m <= kDecodeMaxM) return FP8BS_PATH_DECODE;
    return FP8BS_PATH_PREFILL;
}

int check_gemv_args(const void *x, int64_t m, const uint8_t *codes, const void *scales, int64_t n,
                    int64_t k, void *y, int path) {
    if (m < 0 || n <= 0 || k <= 0 || m >= kMaxDim || n >= kMaxDim || k >= kMaxDim) return FP8BS_ERR_SHAPE;
    if (path < FP8BS_PATH_AUTO || path > FP8BS_PATH_GENERIC) return FP8BS_ERR_PATH;
    if (m == 0) return FP8BS_OK;
    if (!x || !codes || !scales || !y) return FP8BS_ERR_NULL;
    if (!aligned(x, 2) || !aligned(y, 2)) return FP8BS_ERR_ALIGN;
    return FP8BS_OK;
}

int run_decode_chunks(const DecodeArgs &a, cudaStream_t st) {
    for (int64_t m0 = 0; m0 < a.m; m0 += kDecodeMaxM) {
        DecodeArgs c = a;
        c.m = a.m - m0 < kDecodeMaxM ? a.m - m0 : kDecodeMaxM;
        c.x = static_cast<const char *>(a.x) + m0 * a.k * 2;
        c.y = static_cast<char *>(a.y) + m0 * a.n * 2;
        const cudaError_t e = launch_decode(c, st);
        if (e != cudaSuccess) return FP8BS_ERR_CUDA;
    }
    return FP8BS_OK;
}

int gemv_dispatch(const DecodeArgs &a, int path, cudaStream_t st) {
    const bool tma = tma_ok(a.k, a.x, a.codes);
    if (path == FP8BS_PATH_AUTO) path = select_path(a.m, a.k, a.x, a.codes, a.kind == kScaleMx);
    switch (path) {
        case FP8BS_PATH_GENERIC:
            return cuda_status(launch_generic_gemv(a, st));
        case FP8BS_PATH_DECODE:
            if (!tma) return FP8BS_ERR_PATH;
            return run_decode_chunks(a, st);
        case FP8BS_PATH_PREFILL: {
            if (!tma) return FP8BS_ERR_PATH;
            const cudaError_t e = launch_prefill(a, st);
            if (e == cudaErrorNotSupported) return run_decode_chunks(a, st);
            return cuda_status(e);
        }
        default:
            return FP8BS_ERR_PATH;
    }
}

// ------------------------------------------------------------ batches
struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};
inline Range range_of(const void *p, int64_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{lo, lo + static_cast<uintptr_t>(bytes)};
}
inline bool overlap(const Range &a, const Range &b) { return a.lo < b.hi && b.lo < a.hi; }

// What one op of a batch reads and writes.
struct OpSpan {
    Range x, codes, scales, y;
};
OpSpan span_of(const fp8bs_gemv_op &o, int64_t m, bool mx) {
    const int64_t sb = mx ? o.n * ((o.k + 31) / 32) : 4 * ((o.n + 127) / 128) * ((o.k + 127) / 128);
    return OpSpan{range_of(o.x_bf16, 2 * m * o.k), range_of(o.codes, o.n * o.k), range_of(o.scales, sb),
                  range_of(o.y_bf16, 2 * m * o.n)};
}
// b must wait for a if b writes what a reads or writes, or reads what a writes
bool depends(const OpSpan &b, const OpSpan &a) {
    return overlap(b.y, a.x) || overlap(b.y, a.codes) || overlap(b.y, a.scales) || overlap(b.y, a.y) ||
           overlap(b.x, a.y) || overlap(b.codes, a.y) || overlap(b.scales, a.y);
}

int gemv_batch_impl(const fp8bs_gemv_op *ops, int64_t count, int64_t m, bool mx, int path, cudaStream_t st) {
    if (count < 0 || count >= kMaxDim) return FP8BS_ERR_SHAPE;
    if (path < FP8BS_PATH_AUTO || path > FP8BS_PATH_GENERIC) return FP8BS_ERR_PATH;
    if (count == 0) return FP8BS_OK;
    if (!ops) return FP8BS_ERR_NULL;
    // validate everything before anything is enqueued
    for (int64_t i = 0; i < count; ++i) {
        const fp8bs_gemv_op &o = ops[i];
        const int s = check_gemv_args(o.x_bf16, m, o.codes, o.scales, o.n, o.k, o.y_bf16, path);
        if (s != FP8BS_OK) return s;
        if (m == 0) continue;
        if (!mx && !aligned(o.scales, 4)) return FP8BS_ERR_ALIGN;
        const bool tma = tma_ok(o.k, o.x_bf16, o.codes);
        if ((path == FP8BS_PATH_DECODE || path == FP8BS_PATH_PREFILL) && !tma) return FP8BS_ERR_PATH;
    }
    if (m == 0) return FP8BS_OK;
    const ScaleKind kind = mx ? kScaleMx : kScaleBlock;
    const bool batchable_path = path == FP8BS_PATH_AUTO || path == FP8BS_PATH_DECODE;
    BatchItem run[kBatchMaxOps];
    OpSpan spans[kBatchMaxOps];
    int nrun = 0;
    auto flush = [&]() -> int {
        if (nrun == 0) return FP8BS_OK;
        const cudaError_t e = launch_decode_batch(run, nrun, m, kind, path == FP8BS_PATH_DECODE, st);
        nrun = 0;
        return cuda_status(e);
    };
    for (int64_t i = 0; i < count; ++i) {
        const fp8bs_gemv_op &o = ops[i];
        const bool eligible = batchable_path && m <= kDecodeMaxM && tma_ok(o.k, o.x_bf16, o.codes);
        if (!eligible) {
            int s = flush();
            if (s != FP8BS_OK) return s;
            const DecodeArgs a{o.x_bf16, o.codes, mx ? nullptr : static_cast<const float *>(o.scales),
                               mx ? static_cast<const uint8_t *>(o.scales) : nullptr, o.y_bf16, m, o.n, o.k, kind, 0};
            s = gemv_dispatch(a, path, st);
            if (s != FP8BS_OK) return s;
            continue;
        }
        const OpSpan sp = span_of(o, m, mx);
        bool dep = nrun == kBatchMaxOps;
        for (int j = 0; j < nrun && !dep; ++j) dep = depends(sp, spans[j]);
        if (dep) {
            const int s = flush();
            if (s != FP8BS_OK) return s;
        }
        run[nrun] = BatchItem{o.x_bf16, o.codes, o.scales, o.y_bf16, o.n, o.k};
        spans[nrun] = sp;
        ++nrun;
    }
    return flush();
}

int run_w8a8_decode_chunks(const W8A8Args &a, cudaStream_t st) {
    for (int64_t m0 = 0; m0 < a.m; m0 += kDecodeMaxM) {
        W8A8Args c = a;
        c.m = a.m - m0 < kDecodeMaxM ? a.m - m0 : kDecodeMaxM;
        c.xq = a.xq + m0 * a.k;
        c.y = static_cast<char *>(a.y) + m0 * a.n * 2;
        if (launch_w8a8_decode(c, st) != cudaSuccess) return FP8BS_ERR_CUDA;
    }
    return FP8BS_OK;
}

}  // namespace

extern "C" {

int fp8bs_version(void) { return 106; }

const char *fp8bs_strerror(int status) {
    switch (status) {
        case FP8BS_OK: return "ok";
        case FP8BS_ERR_NULL: return "a required pointer is NULL";
        case FP8BS_ERR_SHAPE: return "shape out of range (need n > 0, k > 0, m >= 0, all < 2^31)";
        case FP8BS_ERR_BLOCK: return "unsupported block size (only 128 is supported)";
        case FP8BS_ERR_ALIGN: return "pointer not aligned to its element size";
        case FP8BS_ERR_CUDA: return "CUDA call or kernel launch failed";
        case FP8BS_ERR_DEVICE: return "a kernel gave up a bounded wait (device error word set)";
        case FP8BS_ERR_PATH: return "the requested kernel path cannot take this call";
        default: return "unknown status";
    }
}

int fp8bs_quantize(const void *w_bf16, int64_t n, int64_t k, int block, uint8_t *codes_u8, float *scales_f32,
                   void *stream) {
    if (n <= 0 || k <= 0 || n >= kMaxDim || k >= kMaxDim) return FP8BS_ERR_SHAPE;
    if (block != 128) return FP8BS_ERR_BLOCK;
    if (!w_bf16 || !codes_u8 || !scales_f32) return FP8BS_ERR_NULL;
    if (!aligned(w_bf16, 2) || !aligned(scales_f32, 4)) return FP8BS_ERR_ALIGN;
    const bool vec = (k % 8) == 0 && aligned(w_bf16, 16) && aligned(codes_u8, 8);
    return cuda_status(
        launch_block_quantize(w_bf16, n, k, codes_u8, scales_f32, vec, static_cast<cudaStream_t>(stream)));
}

int mxfp8_quantize(const void *w_bf16, int64_t n, int64_t k, uint8_t *codes_u8, uint8_t *scales_e8m0,
                   void *stream) {
    if (n <= 0 || k <= 0 || n >= kMaxDim || k >= kMaxDim) return FP8BS_ERR_SHAPE;
    if (!w_bf16 || !codes_u8 || !scales_e8m0) return FP8BS_ERR_NULL;
    if (!aligned(w_bf16, 2)) return FP8BS_ERR_ALIGN;
    const bool vec = (k % 8) == 0 && aligned(w_bf16, 16) && aligned(codes_u8, 8);
    return cuda_status(
        launch_mx_quantize(w_bf16, n, k, codes_u8, scales_e8m0, vec, static_cast<cudaStream_t>(stream)));
}

int fp8bs_gemv_ex(const void *x_bf16, int64_t m, const uint8_t *codes, const float *scales, int64_t n,
                  int64_t k, void *y_bf16, int path, void *stream) {
    int st = check_gemv_args(x_bf16, m, codes, scales, n, k, y_bf16, path);
    if (st != FP8BS_OK || m == 0) return st;
    if (!aligned(scales, 4)) return FP8BS_ERR_ALIGN;
    DecodeArgs a{x_bf16, codes, scales, nullptr, y_bf16, m, n, k, kScaleBlock, 0};
    return gemv_dispatch(a, path, static_cast<cudaStream_t>(stream));
}

int fp8bs_gemv(const void *x_bf16, int64_t m, const uint8_t *codes, const float *scales, int64_t n, int64_t k,
               void *y_bf16, void *stream) {
    return fp8bs_gemv_ex(x_bf16, m, codes, scales, n, k, y_bf16, FP8BS_PATH_AUTO, stream);
}

int64_t fp8bs_gemv_ws_bytes(int64_t m, int64_t k) {
    if (m < 0 || k <= 0 || m >= kMaxDim || k >= kMaxDim) return FP8BS_ERR_SHAPE;
    return m == 0 ? 0 : xprep_bytes(m < kDecodeMaxM ? m : kDecodeMaxM, k);
}

int fp8bs_gemv_ws(const void *x_bf16, int64_t m, const uint8_t *codes, const float *scales, int64_t n, int64_t k,
                  void *y_bf16, void *workspace, int64_t workspace_bytes, void *stream) {
    int st = check_gemv_args(x_bf16, m, codes, scales, n, k, y_bf16, FP8BS_PATH_AUTO);
    if (st != FP8BS_OK || m == 0) return st;
    if (!aligned(scales, 4)) return FP8BS_ERR_ALIGN;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    DecodeArgs a{x_bf16, codes, scales, nullptr, y_bf16, m, n, k, kScaleBlock, 0};
    // only the decode path (m <= 32, TMA-eligible) uses the workspace
    if (select_path(m, k, x_bf16, codes, false) != FP8BS_PATH_DECODE) return gemv_dispatch(a, FP8BS_PATH_AUTO, s);
    if (!workspace) return FP8BS_ERR_NULL;
    if (!aligned(workspace, 16)) return FP8BS_ERR_ALIGN;
    if (workspace_bytes < xprep_bytes(m, k)) return FP8BS_ERR_SHAPE;
    return cuda_status(launch_decode_xprep(a, workspace, s));
}

int mxfp8_gemv_ex(const void *x_bf16, int64_t m, const uint8_t *codes, const uint8_t *scales_e8m0, int64_t n,
                  int64_t k, void *y_bf16, int path, void *stream) {
    int st = check_gemv_args(x_bf16, m, codes, scales_e8m0, n, k, y_bf16, path);
    if (st != FP8BS_OK || m == 0) return st;
    DecodeArgs a{x_bf16, codes, nullptr, scales_e8m0, y_bf16, m, n, k, kScaleMx, 0};
    return gemv_dispatch(a, path, static_cast<cudaStream_t>(stream));
}

int mxfp8_gemv(const void *x_bf16, int64_t m, const uint8_t *codes, const uint8_t *scales_e8m0, int64_t n,
               int64_t k, void *y_bf16, void *stream) {
    return mxfp8_gemv_ex(x_bf16, m, codes, scales_e8m0, n, k, y_bf16, FP8BS_PATH_AUTO, stream);
}

int fp8bs_gemv_batch_ex(const fp8bs_gemv_op *ops, int64_t count, int64_t m, int path, void *stream) {
    return gemv_batch_impl(ops, count, m, false, path, static_cast<cudaStream_t>(stream));
}

int fp8bs_gemv_batch(const fp8bs_gemv_op *ops, int64_t count, int64_t m, void *stream) {
    return gemv_batch_impl(ops, count, m, false, FP8BS_PATH_AUTO, static_cast<cudaStream_t>(stream));
}

int mxfp8_gemv_batch_ex(const fp8bs_gemv_op *ops, int64_t count, int64_t m, int path, void *stream) {
    return gemv_batch_impl(ops, count, m, true, path, static_cast<cudaStream_t>(stream));
}

int mxfp8_gemv_batch(const fp8bs_gemv_op *ops, int64_t count, int64_t m, void *stream) {
    return gemv_batch_impl(ops, count, m, true, FP8BS_PATH_AUTO, static_cast<cudaStream_t>(stream));
}

static int rowwise_quantize(const void *w_bf16, int64_t n, int64_t k, uint8_t *codes_u8, float *scales_f32,
                            bool per_tensor, void *stream) {
    if (n <= 0 || k <= 0 || n >= kMaxDim || k >= kMaxDim) return FP8BS_ERR_SHAPE;
    if (!w_bf16 || !codes_u8 || !scales_f32) return FP8BS_ERR_NULL;
    if (!aligned(w_bf16, 2) || !aligned(scales_f32, 4)) return FP8BS_ERR_ALIGN;
    const bool vec = (k % 8) == 0 && aligned(w_bf16, 16) && aligned(codes_u8, 8);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return cuda_status(per_tensor ? launch_tensor_quantize(w_bf16, n, k, codes_u8, scales_f32, vec, st)
                                  : launch_row_quantize(w_bf16, n, k, codes_u8, scales_f32, vec, st));
}

int fp8row_quantize(const void *w_bf16, int64_t n, int64_t k, uint8_t *codes_u8, float *scales_f32, void *stream) {
    return rowwise_quantize(w_bf16, n, k, codes_u8, scales_f32, false, stream);
}

int fp8tensor_quantize(const void *w_bf16, int64_t n, int64_t k, uint8_t *codes_u8, float *scale_f32,
                       void *stream) {
    return rowwise_quantize(w_bf16, n, k, codes_u8, scale_f32, true, stream);
}

static int rowwise_gemv(const void *x_bf16, int64_t m, const uint8_t *codes, const float *scales, int64_t n,
                        int64_t k, void *y_bf16, int row_stride, int path, void *stream) {
    int st = check_gemv_args(x_bf16, m, codes, scales, n, k, y_bf16, path);
    if (st != FP8BS_OK || m == 0) return st;
    if (!aligned(scales, 4)) return FP8BS_ERR_ALIGN;
    DecodeArgs a{x_bf16, codes, scales, nullptr, y_bf16, m, n, k, kScaleRow, row_stride};
    return gemv_dispatch(a, path, static_cast<cudaStream_t>(stream));
}

int fp8row_gemv_ex(const void *x_bf16, int64_t m, const uint8_t *codes, const float *scales, int64_t n, int64_t k,
                   void *y_bf16, int path, void *stream) {
    return rowwise_gemv(x_bf16, m, codes, scales, n, k, y_bf16, 1, path, stream);
}

int fp8row_gemv(const void *x_bf16, int64_t m, const uint8_t *codes, const float *scales, int64_t n, int64_t k,
                void *y_bf16, void *stream) {
    return rowwise_gemv(x_bf16, m, codes, scales, n, k, y_bf16, 1, FP8BS_PATH_AUTO, stream);
}

int fp8tensor_gemv_ex(const void *x_bf16, int64_t m, const uint8_t *codes, const float *scale, int64_t n,
                      int64_t k, void *y_bf16, int path, void *stream) {
    return rowwise_gemv(x_bf16, m, codes, scale, n, k, y_bf16, 0, path, stream);
}

int fp8tensor_gemv(const void *x_bf16, int64_t m, const uint8_t *codes, const float *scale, int64_t n, int64_t k,
                   void *y_bf16, void *stream) {
    return rowwise_gemv(x_bf16, m, codes, scale, n, k, y_bf16, 0, FP8BS_PATH_AUTO, stream);
}

static int moe_check(const void *x_bf16, int64_t m, const int32_t *expert_ids, int64_t topk, const uint8_t *codes,
                     const float *scales, int64_t num_experts, int64_t n, int64_t k, void *y_bf16) {
    if (m < 0 || n <= 0 || k <= 0 || m >= kMaxDim || n >= kMaxDim || k >= kMaxDim) return FP8BS_ERR_SHAPE;
    if (topk < 1 || num_experts < 1 || num_experts > 1024 || topk > num_experts) return FP8BS_ERR_SHAPE;
    if (num_experts * n >= kMaxDim || m * topk >= kMaxDim) return FP8BS_ERR_SHAPE;
    if (m == 0) return FP8BS_OK;
    if (!x_bf16 || !expert_ids || !codes || !scales || !y_bf16) return FP8BS_ERR_NULL;
    if (!aligned(x_bf16, 2) || !aligned(y_bf16, 2) || !aligned(scales, 4) || !aligned(expert_ids, 4))
        return FP8BS_ERR_ALIGN;
    if (!tma_ok(k, x_bf16, codes)) return FP8BS_ERR_PATH;
    return FP8BS_OK;
}

static int moe_decode_chunks(const void *x_bf16, int64_t m, const int32_t *expert_ids, int64_t topk,
                             const uint8_t *codes, const float *scales, int64_t num_experts, int64_t n, int64_t k,
                             void *y_bf16, cudaStream_t st) {
    for (int64_t m0 = 0; m0 < m; m0 += kDecodeMaxM) {
        const int64_t mc = m - m0 < kDecodeMaxM ? m - m0 : kDecodeMaxM;
        DecodeArgs a{static_cast<const char *>(x_bf16) + m0 * k * 2, codes, scales, nullptr,
                     static_cast<char *>(y_bf16) + m0 * topk * n * 2, mc, n, k, kScaleBlock, 0};
        const MoeArgs g{expert_ids + m0 * topk, topk, num_experts};
        if (launch_moe_decode(a, g, st) != cudaSuccess) return FP8BS_ERR_CUDA;
    }
    return FP8BS_OK;
}

int fp8bs_moe_gemv(const void *x_bf16, int64_t m, const int32_t *expert_ids, int64_t topk, const uint8_t *codes,
                   const float *scales, int64_t num_experts, int64_t n, int64_t k, void *y_bf16, void *stream) {
    const int s = moe_check(x_bf16, m, expert_ids, topk, codes, scales, num_experts, n, k, y_bf16);
    if (s != FP8BS_OK || m == 0) return s;
    return moe_decode_chunks(x_bf16, m, expert_ids, topk, codes, scales, num_experts, n, k, y_bf16,
                             static_cast<cudaStream_t>(stream));
}

int64_t fp8bs_moe_gemv_ws_bytes(int64_t m, int64_t topk, int64_t num_experts, int64_t k) {
    if (m < 0 || topk < 1 || num_experts < 1 || num_experts > 1024 || m >= kMaxDim || m * topk >= kMaxDim ||
        k <= 0 || k >= kMaxDim)
        return FP8BS_ERR_SHAPE;
    return m <= kDecodeMaxM ? 0 : moe_route_bytes(m * topk, num_experts, k);
}

int fp8bs_moe_gemv_ws(const void *x_bf16, int64_t m, const int32_t *expert_ids, int64_t topk, const uint8_t *codes,
                      const float *scales, int64_t num_experts, int64_t n, int64_t k, void *y_bf16, void *workspace,
                      int64_t workspace_bytes, void *stream) {
    const int s = moe_check(x_bf16, m, expert_ids, topk, codes, scales, num_experts, n, k, y_bf16);
    if (s != FP8BS_OK || m == 0) return s;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (m <= kDecodeMaxM)
        return moe_decode_chunks(x_bf16, m, expert_ids, topk, codes, scales, num_experts, n, k, y_bf16, st);
    if (!workspace) return FP8BS_ERR_NULL;
    if (!aligned(workspace, 256)) return FP8BS_ERR_ALIGN;
    if (workspace_bytes < moe_route_bytes(m * topk, num_experts, k)) return FP8BS_ERR_SHAPE;
    MoeRoute r = moe_route_views(workspace, m * topk, num_experts, k);
    // GEMM tiles of 128 pairs (a deeper pipeline) while the experts average
    // at most kMoeNarrowAvg pairs, else of 256
    r.gemm_tile = m * topk <= kMoeNarrowAvg * num_experts ? kMoeGemmTileNarrow : kMoeGemmTileWide;
    // few pairs per expert on average: stream each selected expert once per
    // tile of 32 of its pairs at GEMV speed (x copied as f16 operands); more:
    // the tensor-core GEMM (x copied as bf16)
    const bool decode_tiles = m * topk <= kMoeDecodeTile * num_experts;
    cudaError_t e = launch_moe_route(x_bf16, k, expert_ids, m * topk, static_cast<int>(topk),
                                     static_cast<int>(num_experts), r, decode_tiles, st);
    if (e != cudaSuccess) return FP8BS_ERR_CUDA;
    const DecodeArgs a{x_bf16, codes, scales, nullptr, y_bf16, m, n, k, kScaleBlock, 0};
    const MoeArgs g{expert_ids, topk, num_experts};
    if (decode_tiles) return cuda_status(launch_moe_grouped(a, g, r, st));
    e = launch_prefill_moe(a, g, r, st);
    if (e == cudaErrorNotSupported)
        return moe_decode_chunks(x_bf16, m, expert_ids, topk, codes, scales, num_experts, n, k, y_bf16, st);
    return cuda_status(e);
}

int fp8kv_append(const void *x_bf16, int64_t num_tokens, int64_t num_kv_heads, int64_t head_dim,
                 const int32_t *slot_mapping, const float *scale, uint8_t *cache, int64_t num_slots, void *stream) {
    if (num_tokens < 0 || num_kv_heads <= 0 || num_slots <= 0 || num_tokens >= kMaxDim || num_kv_heads >= 4096)
        return FP8BS_ERR_SHAPE;
    if (head_dim != 128) return FP8BS_ERR_SHAPE;
    if (num_slots * num_kv_heads * head_dim >= (int64_t{1} << 40)) return FP8BS_ERR_SHAPE;
    if (num_tokens == 0) return FP8BS_OK;
    if (!x_bf16 || !slot_mapping || !scale || !cache) return FP8BS_ERR_NULL;
    if (!aligned(x_bf16, 16) || !aligned(cache, 8) || !aligned(slot_mapping, 4) || !aligned(scale, 4))
        return FP8BS_ERR_ALIGN;
    return cuda_status(launch_kv_append(x_bf16, num_tokens, num_kv_heads, slot_mapping, scale, cache, num_slots,
                                        static_cast<cudaStream_t>(stream)));
}

int fp8kv_decode_attention(const void *q_bf16, const uint8_t *k_cache, const uint8_t *v_cache, const float *k_scale,
                           const float *v_scale, const int32_t *block_table, int64_t max_blocks_per_seq,
                           const int32_t *seq_lens, int64_t batch, int64_t num_q_heads, int64_t num_kv_heads,
                           int64_t head_dim, int64_t page_size, int64_t num_blocks, int64_t max_seq_len, float sm_scale,
                           void *out_bf16, void *stream) {
    if (batch < 0 || num_kv_heads <= 0 || num_q_heads <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0)
        return FP8BS_ERR_SHAPE;
    if (head_dim != 128 || num_q_heads % num_kv_heads != 0 || num_q_heads / num_kv_heads > 8) return FP8BS_ERR_SHAPE;
    if (page_size < 16 || page_size % 16 != 0 || page_size > 4096) return FP8BS_ERR_SHAPE;
    if (num_blocks * page_size >= kMaxDim || batch * num_kv_heads >= kMaxDim || max_blocks_per_seq >= kMaxDim)
        return FP8BS_ERR_SHAPE;
    if (max_seq_len < 0 || max_seq_len > max_blocks_per_seq * page_size) return FP8BS_ERR_SHAPE;
    if (!(sm_scale == sm_scale) || sm_scale > 3.0e38f || sm_scale < -3.0e38f) return FP8BS_ERR_SHAPE;
    if (batch == 0) return FP8BS_OK;
    if (!q_bf16 || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !seq_lens || !out_bf16)
        return FP8BS_ERR_NULL;
    if (!aligned(q_bf16, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out_bf16, 2) ||
        !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4))
        return FP8BS_ERR_ALIGN;
    KvAttnArgs a{q_bf16, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out_bf16,
                 batch, num_q_heads, num_kv_heads, page_size, num_blocks, max_blocks_per_seq, max_seq_len, sm_scale};
    return cuda_status(launch_kv_attention(a, static_cast<cudaStream_t>(stream)));
}

int fp8act_quantize(const void *x_bf16, int64_t m, int64_t k, uint8_t *codes_u8, float *scale_f32, void *stream) {
    if (m <= 0 || k <= 0 || m >= kMaxDim || k >= kMaxDim) return FP8BS_ERR_SHAPE;
    if (!x_bf16 || !codes_u8 || !scale_f32) return FP8BS_ERR_NULL;
    if (!aligned(x_bf16, 2) || !aligned(scale_f32, 4)) return FP8BS_ERR_ALIGN;
    const bool vec = (k % 8) == 0 && aligned(x_bf16, 16) && aligned(codes_u8, 8);
    return cuda_status(launch_act_quantize(x_bf16, m, k, codes_u8, scale_f32, vec, static_cast<cudaStream_t>(stream)));
}

int w8a8_gemm_ex(const uint8_t *x_codes, int64_t m, const float *x_scale, const uint8_t *w_codes,
                 const float *w_scale, int64_t n, int64_t k, void *y_bf16, int path, void *stream) {
    if (m < 0 || n <= 0 || k <= 0 || m >= kMaxDim || n >= kMaxDim || k >= kMaxDim) return FP8BS_ERR_SHAPE;
    if (path < FP8BS_PATH_AUTO || path > FP8BS_PATH_GENERIC) return FP8BS_ERR_PATH;
    if (m == 0) return FP8BS_OK;
    if (!x_codes || !x_scale || !w_codes || !w_scale || !y_bf16) return FP8BS_ERR_NULL;
    if (!aligned(x_scale, 4) || !aligned(w_scale, 4) || !aligned(y_bf16, 2)) return FP8BS_ERR_ALIGN;
    const bool tma = tma_ok(k, x_codes, w_codes);
    if (path == FP8BS_PATH_AUTO) path = !tma ? FP8BS_PATH_GENERIC : (m <= kDecodeMaxM ? FP8BS_PATH_DECODE : FP8BS_PATH_PREFILL);
    const W8A8Args a{x_codes, x_scale, w_codes, w_scale, y_bf16, m, n, k};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (path) {
        case FP8BS_PATH_GENERIC: return cuda_status(launch_w8a8_generic(a, st));
        case FP8BS_PATH_DECODE: return tma ? run_w8a8_decode_chunks(a, st) : FP8BS_ERR_PATH;
        case FP8BS_PATH_PREFILL: return tma ? cuda_status(launch_w8a8_prefill(a, st)) : FP8BS_ERR_PATH;
        default: return FP8BS_ERR_PATH;
    }
}

int w8a8_gemm(const uint8_t *x_codes, int64_t m, const float *x_scale, const uint8_t *w_codes, const float *w_scale,
              int64_t n, int64_t k, void *y_bf16, void *stream) {
    return w8a8_gemm_ex(x_codes, m, x_scale, w_codes, w_scale, n, k, y_bf16, FP8BS_PATH_AUTO, stream);
}

int fp8bs_kv_plan(const int32_t *ctx_lens, const int32_t *new_lens, int64_t batch, int32_t *block_table,
                  int64_t max_blocks_per_seq, const int32_t *free_blocks, int64_t num_free, const int32_t *free_head,
                  int64_t page_size, int64_t num_blocks, int64_t num_tokens, int32_t *seq_lens, int32_t *cu_new,
                  int32_t *slots, int32_t *positions, int32_t *requests, int32_t *free_head_out, void *stream) {
    if (batch < 0 || batch > kPlanMaxBatch || max_blocks_per_seq <= 0 || max_blocks_per_seq >= kMaxDim ||
        num_free < 0 || num_free >= kMaxDim || num_tokens < 0 || num_tokens >= kMaxDim)
        return FP8BS_ERR_SHAPE;
    if (page_size < 1 || page_size > 65536 || num_blocks <= 0 || num_blocks >= kMaxDim ||
        num_blocks * page_size >= kMaxDim || max_blocks_per_seq * page_size >= kMaxDim)
        return FP8BS_ERR_SHAPE;
    if (!free_head || !cu_new || !free_head_out || (num_free > 0 && !free_blocks)) return FP8BS_ERR_NULL;
    if (batch > 0 && (!ctx_lens || !new_lens || !block_table || !seq_lens)) return FP8BS_ERR_NULL;
    if (num_tokens > 0 && (!slots || !positions || !requests)) return FP8BS_ERR_NULL;
    const void *const ptrs[] = {ctx_lens, new_lens,  block_table, free_blocks, free_head,    seq_lens,
                                cu_new,   slots,     positions,   requests,    free_head_out};
    for (const void *p : ptrs)
        if (!aligned(p, 4)) return FP8BS_ERR_ALIGN;
    const KvPlanArgs a{ctx_lens, new_lens,  block_table,   free_blocks, free_head,          seq_lens,
                       cu_new,   slots,     positions,     requests,    free_head_out,      batch,
                       max_blocks_per_seq,  num_free,      page_size,   num_blocks,         num_tokens};
    return cuda_status(launch_kv_plan(a, static_cast<cudaStream_t>(stream)));
}

namespace {

int check_kv4_cache(int64_t kv_heads, int64_t head_dim, int64_t page_size, int64_t num_blocks) {
    if (kv_heads <= 0 || kv_heads >= 4096 || (head_dim != 64 && head_dim != 128)) return FP8BS_ERR_SHAPE;
    if (page_size < kKv4Tile || page_size % kKv4Tile != 0 || page_size > 4096) return FP8BS_ERR_SHAPE;
    if (num_blocks <= 0 || num_blocks >= kMaxDim || num_blocks * page_size >= kMaxDim) return FP8BS_ERR_SHAPE;
    if (num_blocks * (page_size / kKv4Tile) * kv_heads >= kMaxDim) return FP8BS_ERR_SHAPE;  // int32 tile numbers
    return FP8BS_OK;
}

bool stride_ok(int64_t stride, int64_t row) { return stride >= 0 && stride < (int64_t{1} << 40) && row > 0; }

}  // namespace

int fp4kv_append(const void *k_bf16, int64_t k_stride, const void *v_bf16, int64_t v_stride, int64_t num_tokens,
                 int64_t num_kv_heads, int64_t head_dim, const int32_t *slots, const float *k_scale,
                 const float *v_scale, uint8_t *k_cache, uint8_t *v_cache, int64_t page_size, int64_t num_blocks,
                 void *stream) {
    if (num_tokens < 0 || num_tokens >= kMaxDim) return FP8BS_ERR_SHAPE;
    const int st = check_kv4_cache(num_kv_heads, head_dim, page_size, num_blocks);
    if (st != FP8BS_OK) return st;
    const int64_t row = num_kv_heads * head_dim;
    if (!stride_ok(k_stride, row) || !stride_ok(v_stride, row)) return FP8BS_ERR_SHAPE;
    if (num_tokens == 0) return FP8BS_OK;
    if (!k_bf16 || !v_bf16 || !slots || !k_scale || !v_scale || !k_cache || !v_cache) return FP8BS_ERR_NULL;
    if (!aligned(k_bf16, 16) || !aligned(v_bf16, 16) || k_stride % 8 != 0 || v_stride % 8 != 0 || !aligned(slots, 4) ||
        !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
        return FP8BS_ERR_ALIGN;
    Kv4CopyArgs a = {};
    a.k = k_bf16, a.v = v_bf16, a.k_stride = k_stride, a.v_stride = v_stride;
    a.slots = slots, a.k_scale = k_scale, a.v_scale = v_scale, a.k_cache = k_cache, a.v_cache = v_cache;
    a.tokens = num_tokens, a.kv_heads = num_kv_heads, a.head_dim = head_dim, a.page_size = page_size;
    a.num_slots = num_blocks * page_size;
    return cuda_status(launch_kv4_append(a, static_cast<cudaStream_t>(stream)));
}

int fp4kv_gather(const uint8_t *k_cache, const uint8_t *v_cache, const int32_t *slots, int64_t num_tokens,
                 int64_t num_kv_heads, int64_t head_dim, int64_t page_size, int64_t num_blocks, const float *k_scale,
                 const float *v_scale, void *k_bf16, void *v_bf16, void *stream) {
    if (num_tokens < 0 || num_tokens >= kMaxDim) return FP8BS_ERR_SHAPE;
    const int st = check_kv4_cache(num_kv_heads, head_dim, page_size, num_blocks);
    if (st != FP8BS_OK) return st;
    if (num_tokens == 0) return FP8BS_OK;
    if (!k_bf16 || !v_bf16 || !slots || !k_scale || !v_scale || !k_cache || !v_cache) return FP8BS_ERR_NULL;
    if (!aligned(k_bf16, 16) || !aligned(v_bf16, 16) || !aligned(slots, 4) || !aligned(k_scale, 4) ||
        !aligned(v_scale, 4) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
        return FP8BS_ERR_ALIGN;
    Kv4CopyArgs a = {};
    a.k_out = k_bf16, a.v_out = v_bf16;
    a.slots = slots, a.k_scale = k_scale, a.v_scale = v_scale;
    a.k_cache = const_cast<uint8_t *>(k_cache), a.v_cache = const_cast<uint8_t *>(v_cache);
    a.tokens = num_tokens, a.kv_heads = num_kv_heads, a.head_dim = head_dim, a.page_size = page_size;
    a.num_slots = num_blocks * page_size;
    return cuda_status(launch_kv4_gather(a, static_cast<cudaStream_t>(stream)));
}

int64_t fp4kv_attention_ws_bytes(int64_t head_dim) {
    if (head_dim != 64 && head_dim != 128) return FP8BS_ERR_SHAPE;
    return kv4_attention_ws_bytes(head_dim);
}

int fp4kv_decode_attention(const void *q_bf16, int64_t q_stride, const int32_t *cu_q, int64_t num_q_tokens,
                           int64_t max_q, const uint8_t *k_cache, const uint8_t *v_cache, const float *k_scale,
                           const float *v_scale, const int32_t *block_table, int64_t max_blocks_per_seq,
                           const int32_t *seq_lens, int64_t batch, int64_t num_q_heads, int64_t num_kv_heads,
                           int64_t head_dim, int64_t page_size, int64_t num_blocks, int64_t max_seq_len,
                           int64_t window, float sm_scale, void *out_bf16, float *lse, void *workspace,
                           int64_t workspace_bytes, void *stream) {
    const int st = check_kv4_cache(num_kv_heads, head_dim, page_size, num_blocks);
    if (st != FP8BS_OK) return st;
    if (batch < 0 || batch >= 65536 || num_q_tokens < 0 || num_q_tokens >= kMaxDim || max_q < 1 || max_q >= 65536)
        return FP8BS_ERR_SHAPE;
    if (num_q_heads <= 0 || num_q_heads >= 65536 || num_q_heads % num_kv_heads != 0) return FP8BS_ERR_SHAPE;
    if (!cu_q && (num_q_tokens != batch || max_q != 1)) return FP8BS_ERR_SHAPE;
    if (max_q * (num_q_heads / num_kv_heads) >= kMaxDim || num_q_tokens * num_q_heads >= (int64_t{1} << 40))
        return FP8BS_ERR_SHAPE;
    if (max_blocks_per_seq <= 0 || max_blocks_per_seq >= kMaxDim || max_blocks_per_seq * page_size >= kMaxDim)
        return FP8BS_ERR_SHAPE;
    if (max_seq_len < 0 || max_seq_len > max_blocks_per_seq * page_size || max_seq_len > kMaxDim - 64 || window < 0 || window >= kMaxDim)
        return FP8BS_ERR_SHAPE;
    if (!stride_ok(q_stride, num_q_heads * head_dim)) return FP8BS_ERR_SHAPE;
    if (!(sm_scale == sm_scale) || sm_scale > 3.0e38f || sm_scale < -3.0e38f) return FP8BS_ERR_SHAPE;
    if (batch == 0 || num_q_tokens == 0) return FP8BS_OK;
    if (!q_bf16 || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !seq_lens || !out_bf16 ||
        !workspace)
        return FP8BS_ERR_NULL;
    if (!aligned(q_bf16, 16) || q_stride % 8 != 0 || !aligned(cu_q, 4) || !aligned(k_cache, 16) ||
        !aligned(v_cache, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(block_table, 4) ||
        !aligned(seq_lens, 4) || !aligned(out_bf16, 16) || !aligned(lse, 4) || !aligned(workspace, 16))
        return FP8BS_ERR_ALIGN;
    if (workspace_bytes < kv4_attention_ws_bytes(head_dim)) return FP8BS_ERR_SHAPE;
    Kv4AttnArgs a = {};
    a.q = q_bf16, a.cu_q = cu_q, a.k_cache = k_cache, a.v_cache = v_cache, a.k_scale = k_scale, a.v_scale = v_scale;
    a.block_table = block_table, a.seq_lens = seq_lens, a.out = out_bf16, a.lse = lse, a.workspace = workspace;
    a.q_stride = q_stride, a.tokens = num_q_tokens, a.max_q = max_q, a.batch = batch, a.q_heads = num_q_heads;
    a.kv_heads = num_kv_heads, a.head_dim = head_dim, a.page_size = page_size, a.num_blocks = num_blocks;
    a.max_blocks = max_blocks_per_seq, a.max_seq_len = max_seq_len, a.window = window, a.sm_scale = sm_scale;
    return cuda_status(launch_kv4_attention(a, static_cast<cudaStream_t>(stream)));
}

namespace {

int check_rope(const KvRopeArgs &a) {
    if (a.tokens < 0 || a.tokens >= kMaxDim || a.q_heads <= 0 || a.q_heads >= 65536) return FP8BS_ERR_SHAPE;
    if (a.tokens * a.q_heads >= (int64_t{1} << 40) || a.tokens * (a.q_heads + 2 * a.kv_heads) >= (int64_t{1} << 33))
        return FP8BS_ERR_SHAPE;
    if (a.max_pos <= 0 || a.max_pos >= kMaxDim || a.rot_dim < 16 || a.rot_dim % 16 != 0 || a.rot_dim > a.head_dim)
        return FP8BS_ERR_SHAPE;
    if (!stride_ok(a.q_stride, a.q_heads * a.head_dim) || !stride_ok(a.k_stride, a.kv_heads * a.head_dim) ||
        !stride_ok(a.v_stride, a.kv_heads * a.head_dim))
        return FP8BS_ERR_SHAPE;
    if (!(a.eps >= 0.0f) || a.eps > 3.0e38f) return FP8BS_ERR_SHAPE;
    if (a.tokens == 0) return FP8BS_OK;
    if (!a.q || !a.k || !a.v || !a.positions || !a.slots || !a.cos_sin || !a.q_out || !a.k_scale || !a.v_scale ||
        !a.k_cache || !a.v_cache)
        return FP8BS_ERR_NULL;
    if (!aligned(a.q, 16) || !aligned(a.k, 16) || !aligned(a.v, 16) || a.q_stride % 8 != 0 || a.k_stride % 8 != 0 ||
        a.v_stride % 8 != 0 || !aligned(a.positions, 4) || !aligned(a.slots, 4) || !aligned(a.cos_sin, 16) ||
        !aligned(a.q_weight, 16) || !aligned(a.k_weight, 16) || !aligned(a.q_out, 16) || !aligned(a.k_scale, 4) ||
        !aligned(a.v_scale, 4) || !aligned(a.k_cache, 16) || !aligned(a.v_cache, 16))
        return FP8BS_ERR_ALIGN;
    return FP8BS_OK;
}

int run_rope(const KvRopeArgs &a, bool four_bit, void *stream) {
    const int st = check_rope(a);
    if (st != FP8BS_OK || a.tokens == 0) return st;
    return cuda_status(launch_kv_rope(a, four_bit, static_cast<cudaStream_t>(stream)));
}

}  // namespace

int fp8kv_rope_append(const void *q_bf16, int64_t q_stride, const void *k_bf16, int64_t k_stride, const void *v_bf16,
                      int64_t v_stride, int64_t num_tokens, int64_t num_q_heads, int64_t num_kv_heads,
                      int64_t head_dim, const int32_t *positions, const int32_t *slots, const float *cos_sin,
                      int64_t max_pos, int64_t rot_dim, int interleaved, const void *q_weight, const void *k_weight,
                      float eps, void *q_out, const float *k_scale, const float *v_scale, uint8_t *k_cache,
                      uint8_t *v_cache, int64_t num_slots, void *stream) {
    if (num_kv_heads <= 0 || num_kv_heads >= 4096 || num_slots <= 0 || head_dim != 128) return FP8BS_ERR_SHAPE;
    if (num_slots >= kMaxDim || num_slots * num_kv_heads * head_dim >= (int64_t{1} << 40)) return FP8BS_ERR_SHAPE;
    const KvRopeArgs a{q_bf16, k_bf16, v_bf16, positions, slots, cos_sin, q_weight, k_weight, q_out, k_scale, v_scale,
                       k_cache, v_cache, q_stride, k_stride, v_stride, num_tokens, num_q_heads, num_kv_heads, head_dim,
                       max_pos, rot_dim, 0, num_slots, eps, interleaved != 0};
    return run_rope(a, false, stream);
}

int fp4kv_rope_append(const void *q_bf16, int64_t q_stride, const void *k_bf16, int64_t k_stride, const void *v_bf16,
                      int64_t v_stride, int64_t num_tokens, int64_t num_q_heads, int64_t num_kv_heads,
                      int64_t head_dim, const int32_t *positions, const int32_t *slots, const float *cos_sin,
                      int64_t max_pos, int64_t rot_dim, int interleaved, const void *q_weight, const void *k_weight,
                      float eps, void *q_out, const float *k_scale, const float *v_scale, uint8_t *k_cache,
                      uint8_t *v_cache, int64_t page_size, int64_t num_blocks, void *stream) {
    const int st = check_kv4_cache(num_kv_heads, head_dim, page_size, num_blocks);
    if (st != FP8BS_OK) return st;
    const KvRopeArgs a{q_bf16, k_bf16, v_bf16, positions, slots, cos_sin, q_weight, k_weight, q_out, k_scale, v_scale,
                       k_cache, v_cache, q_stride, k_stride, v_stride, num_tokens, num_q_heads, num_kv_heads, head_dim,
                       max_pos, rot_dim, page_size, num_blocks * page_size, eps, interleaved != 0};
    return run_rope(a, true, stream);
}

int fp8bs_moe_route(const void *logits, int logits_f32, int64_t row_stride, int64_t num_tokens, int64_t num_experts,
                    int64_t topk, int scoring, const float *bias, int64_t groups, int64_t topk_groups,
                    int64_t group_top, int renormalize, float scale, int32_t *expert_ids, float *weights,
                    void *stream) {
    if (num_tokens < 0 || num_tokens >= kMaxDim || num_experts < 1 || num_experts > kRouteMaxExperts || topk < 1 ||
        topk > kRouteMaxTopk || num_tokens * topk >= kMaxDim)
        return FP8BS_ERR_SHAPE;
    if ((row_stride < num_experts && row_stride != 0) || row_stride >= (int64_t{1} << 40)) return FP8BS_ERR_SHAPE;
    if (groups < 1 || groups > kRouteMaxGroups || num_experts % groups != 0 || topk_groups < 1 || topk_groups > groups ||
        group_top < 1 || group_top > 2 || group_top > num_experts / groups ||
        topk > topk_groups * (num_experts / groups))
        return FP8BS_ERR_SHAPE;
    if (scoring != FP8BS_SCORE_SOFTMAX && scoring != FP8BS_SCORE_SIGMOID) return FP8BS_ERR_SHAPE;
    if (!(scale == scale) || scale > 3.0e38f || scale < -3.0e38f) return FP8BS_ERR_SHAPE;
    if (num_tokens == 0) return FP8BS_OK;
    if (!logits || !expert_ids || !weights) return FP8BS_ERR_NULL;
    if (!aligned(logits, logits_f32 ? 4 : 2) || !aligned(bias, 4) || !aligned(expert_ids, 4) || !aligned(weights, 4))
        return FP8BS_ERR_ALIGN;
    const MoeScoreArgs a{logits, logits_f32 != 0, scoring == FP8BS_SCORE_SOFTMAX, renormalize != 0, bias, expert_ids,
                         weights, row_stride, num_tokens, num_experts, topk, groups, topk_groups, group_top, scale};
    return cuda_status(launch_moe_scores(a, static_cast<cudaStream_t>(stream)));
}

int fp8bs_moe_combine(const void *y_bf16, const float *weights, const int32_t *expert_ids, int64_t num_experts,
                      const void *residual_bf16, int64_t num_tokens, int64_t topk, int64_t n, void *out_bf16,
                      void *stream) {
    if (num_tokens < 0 || num_tokens >= kMaxDim || topk < 1 || topk > 1024 || n < 1 || n >= kMaxDim ||
        num_experts < 0 || num_experts >= kMaxDim || num_tokens * topk >= kMaxDim)
        return FP8BS_ERR_SHAPE;
    if (num_tokens * ((n + 1023) / 1024) >= kMaxDim) return FP8BS_ERR_SHAPE;  // CTAs of 1024 columns of a token
    if (num_tokens == 0) return FP8BS_OK;
    if (!y_bf16 || !weights || !out_bf16) return FP8BS_ERR_NULL;
    if (!aligned(y_bf16, 2) || !aligned(weights, 4) || !aligned(expert_ids, 4) || !aligned(residual_bf16, 2) ||
        !aligned(out_bf16, 2))
        return FP8BS_ERR_ALIGN;
    const MoeCombineArgs a{y_bf16, weights, expert_ids, residual_bf16, out_bf16, num_tokens, topk, n, num_experts};
    return cuda_status(launch_moe_combine(a, static_cast<cudaStream_t>(stream)));
}

int fp8bs_token_logprobs(const void *logits, int logits_f32, int64_t row_stride, int64_t rows, int64_t vocab,
                         const int32_t *targets, int64_t top, float *logprobs, float *entropy, int32_t *top_ids,
                         float *top_logprobs, void *stream) {
    if (rows < 0 || rows >= kMaxDim || vocab <= 0 || vocab >= kMaxDim || (row_stride < vocab && row_stride != 0) ||
        row_stride >= (int64_t{1} << 40) || top < 0 || top > kLogprobsMaxTop || top > vocab)
        return FP8BS_ERR_SHAPE;
    if (rows == 0) return FP8BS_OK;
    if (!logits || !targets || !logprobs || !entropy || (top > 0 && (!top_ids || !top_logprobs)))
        return FP8BS_ERR_NULL;
    if (!aligned(logits, logits_f32 ? 4 : 2) || !aligned(targets, 4) || !aligned(logprobs, 4) ||
        !aligned(entropy, 4) || !aligned(top_ids, 4) || !aligned(top_logprobs, 4))
        return FP8BS_ERR_ALIGN;
    const LogprobArgs a{logits, logits_f32 != 0, targets, logprobs, entropy, top_ids, top_logprobs,
                        row_stride, rows, vocab, top};
    return cuda_status(launch_token_logprobs(a, static_cast<cudaStream_t>(stream)));
}

int fp8bs_sample_tokens(const void *logits, int logits_f32, int64_t row_stride, int64_t rows, int64_t vocab,
                        const float *u, const float *temperature, const int32_t *top_k, const float *top_p,
                        const float *min_p, int32_t *tokens, float *logprobs, void *stream) {
    if (rows < 0 || rows >= (int64_t{1} << 28) || vocab <= 0 || vocab > kSampleMaxVocab ||
        (row_stride < vocab && row_stride != 0) || row_stride >= (int64_t{1} << 40))
        return FP8BS_ERR_SHAPE;
    if (rows == 0) return FP8BS_OK;
    if (!logits || !u || !tokens) return FP8BS_ERR_NULL;
    if (!aligned(logits, logits_f32 ? 4 : 2) || !aligned(u, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) ||
        !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(tokens, 4) || !aligned(logprobs, 4))
        return FP8BS_ERR_ALIGN;
    const SampleArgs a{logits, logits_f32 != 0, u, temperature, top_k, top_p, min_p, tokens, logprobs, row_stride, rows, vocab};
    return cuda_status(launch_sample(a, static_cast<cudaStream_t>(stream)));
}

int fp8bs_select_path(int64_t m, int64_t n, int64_t k, const void *x_bf16, const void *codes, int mx) {
    (void)n;
    if (m <= 0 || k <= 0) return FP8BS_ERR_SHAPE;
    return select_path(m, k, x_bf16, codes, mx != 0);
}

int fp8bs_debug_wait_expiry(void *stream) {
    return cuda_status(launch_wait_expiry_probe(static_cast<cudaStream_t>(stream)));
}

int fp8bs_debug_encode_f32(uint32_t first_bits, int64_t count, uint8_t *codes_u8, void *stream) {
    if (!codes_u8) return FP8BS_ERR_NULL;
    if (count <= 0 || count % 4 != 0 || static_cast<uint64_t>(first_bits) + static_cast<uint64_t>(count) > (1ull << 32))
        return FP8BS_ERR_SHAPE;
    if (!aligned(codes_u8, 4)) return FP8BS_ERR_ALIGN;
    return cuda_status(launch_encode_probe(first_bits, count, codes_u8, static_cast<cudaStream_t>(stream)));
}

int fp8bs_check_device_error(void *stream, uint32_t *word_out) {
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return FP8BS_ERR_CUDA;
    const uint32_t w = take_decode_error() | take_prefill_error() | take_w8a8_error() | take_kv_error() |
                       take_moe_error() | take_plan_error() | take_kv4_error() | take_logprobs_error() |
                       take_rope_error() | take_sample_error();
    if (word_out) *word_out = w;
    return w ? FP8BS_ERR_DEVICE : FP8BS_OK;
}

}  // extern "C"
