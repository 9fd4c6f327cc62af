// route.cu -- the two ends of a layer of routed experts: which experts a token
// goes to and with which weights, and the weighted sum of what they gave.
//
// Route, a warp a token.  s = softmax(x) or 1 / (1 + e^-x); experts are chosen
// by c = s + bias.  Whole numbers come out, so near ties have to be decided as
// the definition decides them: c is compared in multiples of 2^-44.
#include "twofloat.cuh"

#include "serving.cuh"
#include "internal.h"

namespace fp8bs {

namespace {

constexpr int kRouteWarps = 8;
constexpr float kMostBias = 65536.0f;
constexpr float kNoScore = -104.0f;  // e^x below two_exp2's range

// Order of the values as unsigned integers above 0: -0 is +0, NaN below everything.
__device__ __forceinline__ uint32_t logit_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    return x != x ? 1u : u & 0x80000000u ? ~u : u | 0x80000000u;
}

// c in multiples of 2^-44, above 0, for |c| < 2^17; NaN below everything.
__device__ __forceinline__ uint64_t score_key(Two c) {
    if (c.h != c.h) return 1;
    const float h = c.h * 0x1p44f, l = c.l * 0x1p44f;
    const long long v = fabsf(h) < 0x1p23f ? __float2ll_rn(h + l) : __float2ll_rn(h) + __float2ll_rn(l);
    return static_cast<uint64_t>(v + (1ll << 62));
}

__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
    const uint32_t hi = static_cast<uint32_t>(v >> 32), top = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t lo = __reduce_max_sync(0xffffffffu, hi == top ? static_cast<uint32_t>(v) : 0u);
    return static_cast<uint64_t>(top) << 32 | lo;
}

template <bool F32>
__device__ __forceinline__ float load_logit(const void *row, int e) {
    if constexpr (F32) return static_cast<const float *>(row)[e];
    else return __bfloat162float(static_cast<const __nv_bfloat16 *>(row)[e]);
}

// Lane l has experts l * EPL .. l * EPL + EPL - 1, so that the lowest lane among
// equals has the lowest expert.
template <bool F32, int EPL>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const MoeScoreArgs a) {
    extern __shared__ uint64_t sh_scores[];  // [warps][experts], with groups
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t token = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp;
    pdl_wait();
    if (token >= a.tokens) return;
    const int experts = static_cast<int>(a.experts), topk = static_cast<int>(a.topk), e0 = lane * EPL;
    const void *row = static_cast<const char *>(a.logits) + token * a.row_stride * (F32 ? 4 : 2);
    float x[EPL];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        x[i] = e0 + i < experts ? load_logit<F32>(row, e0 + i) : -INFINITY;
        m = fmaxf(m, x[i]);
    }
    // ---- scores
    Two s[EPL];
    if (a.softmax) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        Two z{0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            // -inf and experts that are not there add nothing, also where there is nothing else
            const float d = m == -INFINITY && x[i] == -INFINITY ? -INFINITY : x[i] - m;
            s[i] = d > kNoScore ? two_exp2(times_log2e(two_sum(x[i], -m))) : Two{d != d ? d : 0.0f, 0.0f};
            z = add(z, s[i]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            z = add(z, Two{__shfl_xor_sync(0xffffffffu, z.h, o), __shfl_xor_sync(0xffffffffu, z.l, o)});
        if (z.h == 0.0f) z.h = 1.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) s[i] = div(s[i], z);
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const float d = -fabsf(x[i]);
            const Two e = d > kNoScore ? two_exp2(times_log2e(Two{d, 0.0f})) : Two{d != d ? d : 0.0f, 0.0f};
            const Two one{1.0f, 0.0f};
            s[i] = div(x[i] < 0.0f ? e : one, add(e, 1.0f));
        }
    }
    // ---- what the experts are ordered by
    uint64_t key[EPL];
    uint32_t mine = 0;  // of this lane's experts, those that may be chosen
    if (a.groups > 1 || a.bias) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            float b = 0.0f;
            if (a.bias && e0 + i < experts) b = fminf(fmaxf(a.bias[e0 + i], -kMostBias), kMostBias);
            key[i] = score_key(add(s[i], b));
        }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) mine |= e0 + i < experts ? 1u << i : 0u;
    if (a.groups > 1) {
        const int groups = static_cast<int>(a.groups), per = experts / groups;
        uint64_t *sc = sh_scores + static_cast<int64_t>(warp) * experts;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (e0 + i < experts) sc[e0 + i] = key[i];
        __syncwarp();
        uint64_t best = 0;  // lane g: the score of group g, of its one or two best experts
        if (lane < groups) {
            uint64_t b1 = 0, b2 = 0;
            for (int j = 0; j < per; ++j) {
                const uint64_t v = sc[lane * per + j];
                if (v > b1) b2 = b1, b1 = v;
                else if (v > b2) b2 = v;
            }
            best = a.group_top == 2 ? b1 + b2 : b1;
        }
        int before = 0;
        for (int g = 0; g < groups; ++g) {
            const uint64_t other = __shfl_sync(0xffffffffu, best, g);
            before += other > best || (other == best && g < lane) ? 1 : 0;
        }
        const uint32_t open = __ballot_sync(0xffffffffu, lane < groups && before < static_cast<int>(a.topk_groups));
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (e0 + i < experts && !((open >> ((e0 + i) / per)) & 1)) mine &= ~(1u << i);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        if (!a.bias) key[i] = logit_key(x[i]);
        if (!((mine >> i) & 1)) key[i] = 0;
    }
    // ---- the best that is left, topk times; lane j keeps the j-th
    int id = 0;
    float w = 0.0f;
    for (int j = 0; j < topk; ++j) {
        uint64_t best = 0;
        int at = 0;
        float sc = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (key[i] > best) best = key[i], at = i, sc = s[i].h;
        const uint64_t top = warp_max(best);
        const int winner = __ffs(__ballot_sync(0xffffffffu, best == top)) - 1;
        const int e = __shfl_sync(0xffffffffu, e0 + at, winner);
        const float ws = __shfl_sync(0xffffffffu, sc, winner);
        if (lane == j) id = e, w = ws;
        if (lane == winner) {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (i == at) key[i] = 0;
        }
    }
    if (a.renormalize) {
        float sum = lane < topk ? w : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        w = sum == 0.0f ? 0.0f : w / sum;
    }
    if (lane < topk) {
        a.ids[token * topk + lane] = id;
        a.weights[token * topk + lane] = w * a.scale;
    }
}

template <bool F32, int EPL>
cudaError_t launch_route_t(const MoeScoreArgs &a, cudaStream_t stream) {
    const int64_t blocks = (a.tokens + kRouteWarps - 1) / kRouteWarps;
    const size_t smem = a.groups > 1 ? static_cast<size_t>(kRouteWarps * a.experts * 8) : 0;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(route_kernel<F32, EPL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(kRouteWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, route_kernel<F32, EPL>, a);
}

template <bool F32>
cudaError_t launch_route_epl(const MoeScoreArgs &a, cudaStream_t stream) {
    if (a.experts <= 32) return launch_route_t<F32, 1>(a, stream);
    if (a.experts <= 64) return launch_route_t<F32, 2>(a, stream);
    if (a.experts <= 128) return launch_route_t<F32, 4>(a, stream);
    if (a.experts <= 256) return launch_route_t<F32, 8>(a, stream);
    if (a.experts <= 512) return launch_route_t<F32, 16>(a, stream);
    return launch_route_t<F32, 32>(a, stream);
}

// --------------------------------------------------------------- combination
// A thread has 8 consecutive columns of a token, 16 bytes of each of its
// slots; kInFlight of them are loaded before the first is used.
constexpr int kCombineThreads = 256;
constexpr int kInFlight = 4;

template <bool VEC>
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, int n, float (&x)[8]) {
    if constexpr (VEC) {
        const uint4 v = ld_v4(p);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) x[2 * j] = bf16lo_to_f32(u[j]), x[2 * j + 1] = bf16hi_to_f32(u[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = j < n ? __bfloat162float(p[j]) : 0.0f;
    }
}

template <bool VEC>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const MoeCombineArgs a, int64_t per_row) {
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kCombineThreads + threadIdx.x;
    const int64_t token = item / per_row, col = 8 * (item - token * per_row);
    pdl_wait();
    if (token >= a.tokens) return;
    const int topk = static_cast<int>(a.topk), cols = static_cast<int>(a.n - col < 8 ? a.n - col : 8);
    const __nv_bfloat16 *y = static_cast<const __nv_bfloat16 *>(a.y) + token * topk * a.n + col;
    float acc[8] = {};
    if (a.residual) load8<VEC>(static_cast<const __nv_bfloat16 *>(a.residual) + token * a.n + col, cols, acc);
    for (int j0 = 0; j0 < topk; j0 += kInFlight) {
        float w[kInFlight], x[kInFlight][8];
        bool live[kInFlight];
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            live[i] = j0 + i < topk;
            if (live[i] && a.ids) {
                const int id = a.ids[token * topk + j0 + i];
                live[i] = id >= 0 && id < a.experts;
            }
            if (live[i]) {
                w[i] = a.weights[token * topk + j0 + i];
                load8<VEC>(y + (j0 + i) * a.n, cols, x[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < kInFlight; ++i)
            if (live[i])
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] = fmaf(w[i], x[i][j], acc[j]);
    }
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + token * a.n + col;
    if constexpr (VEC) {
        *reinterpret_cast<uint4 *>(out) = make_uint4(f32x2_to_bf16x2(acc[0], acc[1]), f32x2_to_bf16x2(acc[2], acc[3]),
                                                     f32x2_to_bf16x2(acc[4], acc[5]), f32x2_to_bf16x2(acc[6], acc[7]));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < cols) out[j] = __float2bfloat16_rn(acc[j]);
    }
}

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

cudaError_t launch_moe_scores(const MoeScoreArgs &a, cudaStream_t stream) {
    return a.f32 ? launch_route_epl<true>(a, stream) : launch_route_epl<false>(a, stream);
}

cudaError_t launch_moe_combine(const MoeCombineArgs &a, cudaStream_t stream) {
    const int64_t per_row = (a.n + 7) / 8, items = a.tokens * per_row;
    const int64_t blocks = (items + kCombineThreads - 1) / kCombineThreads;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    const bool vec = a.n % 8 == 0 && aligned16(a.y) && aligned16(a.residual) && aligned16(a.out);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(kCombineThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return vec ? cudaLaunchKernelEx(&cfg, combine_kernel<true>, a, per_row)
               : cudaLaunchKernelEx(&cfg, combine_kernel<false>, a, per_row);
}

}  // namespace fp8bs
