// kvrope.cu -- the rows of a fused q, k, v projection on their way to the
// attention: norm of each query and key head, rotation by position, q out in
// bf16, k and v into the paged cache (FP8 or 4-bit).
//
// Of a head vector a of D elements with norm weights w, at a position's (c, s):
//   r = fl(1 / sqrt(mean a^2 + eps)),  n_i = fl(fl(a_i r) w_i)  (n = a without weights),
//   o1 = fl(fl(n1 c) - fl(n2 s)),  o2 = fl(fl(n2 c) + fl(n1 s))
// over the rotated pairs, each fl one fp32 rounding, so that the bytes of the
// cache are defined exactly.  r is the rounding of the exact value but for one
// head in about 2^17: a key's sum of squares is carried in two fp32 numbers (a
// square of a bf16 number is exact in one), and a step of Newton's method with
// an exact residual corrects the square root's reciprocal.  With a plain fp32
// sum r is off by a unit in the last place for every third head, and a 4-bit
// code in some ten million with it.
#include "serving.cuh"
#include "internal.h"

namespace fp8bs {

namespace {

__device__ uint32_t g_rope_err;

constexpr int kRopeThreads = 256;

// a + b = s + e exactly (Knuth's two-sum).
__device__ __forceinline__ void two_sum(float a, float b, float &s, float &e) {
    s = __fadd_rn(a, b);
    const float t = __fsub_rn(s, a);
    e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
}

// 1 / sqrt(h + l), |l| <= ulp(h): one rounding of y + y (1 - (h + l) y^2) / 2,
// with y = rsqrtf(h) and the residual exact to 2^-24 of itself.
__device__ __forceinline__ float rsqrt_once(float h, float l) {
    const float y = rsqrtf(h);
    const float p = __fmul_rn(y, y), pe = __fmaf_rn(y, y, -p);
    float e = __fmaf_rn(-h, p, 1.0f);
    e = __fmaf_rn(-h, pe, e);
    e = __fmaf_rn(-l, p, e);
    return __fmaf_rn(__fmul_rn(0.5f, y), e, y);
}

enum RopeKind : int { kRopeQ = 0, kRopeK = 1, kRopeV = 2 };

// Heads of one kind of one token: N for each team of D / 8 lanes of the warp.
// A lane has 8 consecutive elements of each, 16 bytes of bf16.
template <int D, int N, bool F4>
__device__ __forceinline__ void rope_heads(const KvRopeArgs &a, int kind, int64_t token, int64_t slot, int position,
                                           int head0) {
    constexpr int kLanes = D / 8, kTeams = 32 / kLanes;
    const int lane = threadIdx.x & 31, l = lane % kLanes, team = lane / kLanes;
    const int heads = static_cast<int>(kind == kRopeQ ? a.q_heads : a.kv_heads);
    const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(kind == kRopeQ ? a.q : kind == kRopeK ? a.k : a.v) +
                               token * (kind == kRopeQ ? a.q_stride : kind == kRopeK ? a.k_stride : a.v_stride);
    uint4 raw[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int h = head0 + i * kTeams + team;
        raw[i] = h < heads ? ld_v4(src + h * D + 8 * l) : make_uint4(0, 0, 0, 0);
    }
    // ---- what the heads share: norm weights, cos and sin
    const void *wp = kind == kRopeQ ? a.q_weight : kind == kRopeK ? a.k_weight : nullptr;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (wp) w = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(wp) + 8 * l);
    const int rot = static_cast<int>(a.rot_dim), half = rot / 2;
    const bool turns = kind != kRopeV && 8 * l < rot, first = 8 * l < half;
    float c[8], s[8];
    if (turns) {
        const float *row = a.cos_sin + static_cast<int64_t>(position) * rot;
        if (a.interleaved) {
            const float4 cc = *reinterpret_cast<const float4 *>(row + 4 * l);
            const float4 ss = *reinterpret_cast<const float4 *>(row + half + 4 * l);
            const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) c[j] = cv[j / 2], s[j] = (j & 1) ? sv[j / 2] : -sv[j / 2];
        } else {
            const float *p = row + (first ? 8 * l : 8 * l - half);
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
                const float4 cc = *reinterpret_cast<const float4 *>(p + j);
                const float4 ss = *reinterpret_cast<const float4 *>(p + half + j);
                c[j] = cc.x, c[j + 1] = cc.y, c[j + 2] = cc.z, c[j + 3] = cc.w;
                s[j] = ss.x, s[j + 1] = ss.y, s[j + 2] = ss.z, s[j + 3] = ss.w;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] = first ? -s[j] : s[j];
        }
    }
    // the lane with the other elements of this lane's pairs
    const int partner = !turns ? lane : first ? lane + half / 8 : lane - half / 8;
    float scale = 1.0f;
    if (kind != kRopeQ) scale = *(kind == kRopeK ? a.k_scale : a.v_scale);

#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int h = head0 + i * kTeams + team;
        const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        float x[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[2 * j] = bf16lo_to_f32(u[j]), x[2 * j + 1] = bf16hi_to_f32(u[j]);
        if (wp) {
            float sum = 0.0f, rest = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float sq = __fmul_rn(x[j], x[j]);
                if (kind == kRopeQ) {
                    sum = __fadd_rn(sum, sq);
                } else {
                    float e;
                    two_sum(sum, sq, sum, e);
                    rest += e;
                }
            }
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) {
                const float os = __shfl_xor_sync(0xffffffffu, sum, o);
                if (kind == kRopeQ) {
                    sum = __fadd_rn(sum, os);
                } else {
                    const float oe = __shfl_xor_sync(0xffffffffu, rest, o);
                    float e;
                    two_sum(sum, os, sum, e);
                    rest = (rest + oe) + e;
                }
            }
            float vh, vl;
            two_sum(sum * (1.0f / D), a.eps, vh, vl);
            vl += rest * (1.0f / D);
            const float r = rsqrt_once(vh, vl);
            const uint32_t wu[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float wj = j & 1 ? bf16hi_to_f32(wu[j / 2]) : bf16lo_to_f32(wu[j / 2]);
                x[j] = __fmul_rn(__fmul_rn(x[j], r), wj);
            }
        }
        if (kind != kRopeV) {
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float other = a.interleaved ? x[j ^ 1] : __shfl_sync(0xffffffffu, x[j], partner);
                o[j] = turns ? __fadd_rn(__fmul_rn(x[j], c[j]), __fmul_rn(other, s[j])) : x[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = o[j];
        }
        if (kind == kRopeQ) {
            if (h < heads)
                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.q_out) + (token * heads + h) * D + 8 * l) =
                    make_uint4(f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]), f32x2_to_bf16x2(x[4], x[5]),
                               f32x2_to_bf16x2(x[6], x[7]));
            continue;
        }
        uint8_t *cache = kind == kRopeK ? a.k_cache : a.v_cache;
        if constexpr (F4) {
            // a group is two lanes; NaN is above every magnitude
            uint32_t mx = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) mx = max(mx, __float_as_uint(x[j]) & 0x7FFFFFFFu);
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            const uint32_t sc = f32x2_to_e4m3x2(__uint_as_float(mx) / (6.0f * scale), 0.0f) & 0xFFu;
            const float den = f16x2_to_f32x2(e4m3x2_to_f16x2(sc)).x * scale;
            uint32_t codes = 0;
            if (den > 0.0f) {
                float q[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) q[j] = x[j] / den;
                codes = f32x8_to_e2m1x8(q);
            }
            if (h < heads && slot >= 0) {
                const uint32_t tpp = static_cast<uint32_t>(a.page_size / kKv4Tile);
                const uint32_t tile = static_cast<uint32_t>(slot) / kKv4Tile, row = static_cast<uint32_t>(slot) % kKv4Tile;
                const uint32_t blk = tile / tpp;
                uint8_t *t = cache + ((static_cast<int64_t>(blk) * heads + h) * tpp + (tile - blk * tpp)) * kv4_tile_bytes(D);
                *reinterpret_cast<uint32_t *>(t + row * (D / 2) + 4 * l) = codes;
                if ((l & 1) == 0) t[8 * D + row * (D / 16) + l / 2] = static_cast<uint8_t>(sc);
            }
        } else {
            uint32_t out[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                out[j] = f32x2_to_e4m3x2(x[4 * j] / scale, x[4 * j + 1] / scale) |
                         static_cast<uint32_t>(f32x2_to_e4m3x2(x[4 * j + 2] / scale, x[4 * j + 3] / scale)) << 16;
            if (h < heads && slot >= 0)
                *reinterpret_cast<uint2 *>(cache + (slot * heads + h) * D + 8 * l) = make_uint2(out[0], out[1]);
        }
    }
}

// A warp has up to N * (256 / D) heads of one kind of one token; q_warps and
// kv_warps of them make a token's q, k and v.
template <int D, int N, bool F4>
__global__ void __launch_bounds__(kRopeThreads) kv_rope_kernel(const KvRopeArgs a, int q_warps, int kv_warps) {
    constexpr int kHeads = N * (256 / D);
    const int per_token = q_warps + 2 * kv_warps;
    const int64_t warp = static_cast<int64_t>(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5);
    const int64_t token = warp / per_token;
    const int part = static_cast<int>(warp - token * per_token);
    pdl_wait();
    if (token >= a.tokens) return;
    const int position = a.positions[token];
    const int64_t slot = a.slots[token];
    if (position < 0 || position >= a.max_pos) {
        if (position != -1 && part == 0 && (threadIdx.x & 31) == 0) atomicOr(&g_rope_err, ERRBIT_INDEX);
        return;
    }
    const int kind = part < q_warps ? kRopeQ : part < q_warps + kv_warps ? kRopeK : kRopeV;
    const int at = kind == kRopeQ ? part : kind == kRopeK ? part - q_warps : part - q_warps - kv_warps;
    if (kind == kRopeQ) {
        rope_heads<D, N, F4>(a, kRopeQ, token, slot, position, at * kHeads);
        return;
    }
    if (slot < 0 || slot >= a.num_slots) {
        if (slot != -1 && at == 0 && kind == kRopeK && (threadIdx.x & 31) == 0) atomicOr(&g_rope_err, ERRBIT_INDEX);
        return;
    }
    if (kind == kRopeK) rope_heads<D, N, F4>(a, kRopeK, token, slot, position, at * kHeads);
    else rope_heads<D, N, F4>(a, kRopeV, token, slot, position, at * kHeads);
}

template <int D, int N, bool F4>
cudaError_t launch_rope(const KvRopeArgs &a, cudaStream_t stream) {
    constexpr int64_t kHeads = N * (256 / D);
    const int64_t q_warps = (a.q_heads + kHeads - 1) / kHeads, kv_warps = (a.kv_heads + kHeads - 1) / kHeads;
    const int64_t warps = a.tokens * (q_warps + 2 * kv_warps), per = kRopeThreads / 32;
    const int64_t blocks = (warps + per - 1) / per;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(kRopeThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_rope_kernel<D, N, F4>, a, static_cast<int>(q_warps), static_cast<int>(kv_warps));
}

template <int D, bool F4>
cudaError_t launch_rope_split(const KvRopeArgs &a, cudaStream_t stream) {
    return launch_rope<D, 2, F4>(a, stream);
}

}  // namespace

cudaError_t launch_kv_rope(const KvRopeArgs &a, bool four_bit, cudaStream_t stream) {
    if (!four_bit) return launch_rope_split<128, false>(a, stream);
    return a.head_dim == 128 ? launch_rope_split<128, true>(a, stream) : launch_rope_split<64, true>(a, stream);
}

uint32_t take_rope_error() {
    uint32_t v = 0;
    if (cudaMemcpyFromSymbol(&v, g_rope_err, sizeof v) != cudaSuccess) return 0xFFFFFFFFu;
    const uint32_t zero = 0;
    cudaMemcpyToSymbol(g_rope_err, &zero, sizeof zero);
    return v;
}

}  // namespace fp8bs
