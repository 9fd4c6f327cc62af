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
#include "twofloat.cuh"

#include "serving.cuh"
#include "internal.h"

namespace fp8bs {

namespace {

__device__ uint32_t g_rope_err;

constexpr int kRopeThreads = 256;

// 1 / sqrt(h + l), |l| <= ulp(h): one rounding of y + y (1 - (h + l) y^2) / 2,
// with y = rsqrtf(h) and the residual exact to 2^-24 of itself.
__device__ __forceinline__ float rsqrt_once(float h, float l) {
    const float y = rsqrtf(h);
    const Two p = two_prod(y, y);
    float e = fma1(-h, p.h, 1.0f);
    e = fma1(-h, p.l, e);
    e = fma1(-l, p.h, e);
    return fma1(mul1(0.5f, y), e, y);
}

__device__ __forceinline__ uint2 ld_v2(const void *p) {
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

// The codes of x / s without a division: q = x (1 / s) is within 2^-23 of the
// quotient, so if q (1 - 2^-21) and q (1 + 2^-21) have one code, the rounded
// quotient has it too; a value near a border between codes is divided (one in
// some hundred thousand).  encode(v) gives the codes of v[0 .. 7]; `recip` is RN(1 / s) for
// s in [2^-100, 2^100], or 0: every value is divided.
template <class Word, class Encode>
__device__ __forceinline__ Word codes_of(const float (&x)[8], float s, float recip, Encode encode) {
    float lo[8], hi[8];
    if (recip != 0.0f) {
        const uint64_t y2 = pair(recip, recip), down = pair(1.0f - 0x1p-21f, 1.0f - 0x1p-21f);
        const uint64_t up = pair(1.0f + 0x1p-21f, 1.0f + 0x1p-21f);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const uint64_t q = mul2(pair(x[j], x[j + 1]), y2);
            unpair(mul2(q, down), lo[j], lo[j + 1]);
            unpair(mul2(q, up), hi[j], hi[j + 1]);
        }
        const Word a = encode(lo), b = encode(hi);
        if (a == b) return a;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) lo[j] = __fdiv_rn(x[j], s);
    return encode(lo);
}
__device__ __forceinline__ float safe_reciprocal(float s) { return s >= 0x1p-100f && s <= 0x1p100f ? __frcp_rn(s) : 0.0f; }

enum RopeKind : int { kRopeQ = 0, kRopeK = 1, kRopeV = 2 };

// A lane has 8 elements of each of its heads, in pairs of four: of a query, or
// of pairs that are neighbours, the elements that turn together; of a key with
// halves, and of a value, 8 consecutive ones, because a group of a 4-bit cache
// is 16.  first, second: where the lane's two fours begin.
struct Fours {
    int first, second;
    bool turns;
};
template <int D, bool NEXT>
__device__ __forceinline__ Fours fours_of(int kind, int l, int rot) {
    const int half = rot / 2;
    if (kind == kRopeQ && !NEXT) {
        if (4 * l < half) return Fours{4 * l, half + 4 * l, true};
        return Fours{8 * l, 8 * l + 4, false};  // 8 (l - half / 4) past the rotated ones
    }
    return Fours{8 * l, 8 * l + 4, 8 * l < rot};
}

__device__ __forceinline__ void unpack4(uint2 u, uint64_t &a, uint64_t &b) {
    a = pair(bf16lo_to_f32(u.x), bf16hi_to_f32(u.x));
    b = pair(bf16lo_to_f32(u.y), bf16hi_to_f32(u.y));
}
__device__ __forceinline__ uint32_t pack2(uint64_t v) {
    float a, b;
    unpair(v, a, b);
    return f32x2_to_bf16x2(a, b);
}
__device__ __forceinline__ uint64_t neg2(uint64_t v) { return v ^ 0x8000000080000000ull; }

// The sums of two products, each rounded before: as a pair's addition the
// assembler joins it with one of the products, whatever its rounding is said to be.
__device__ __forceinline__ uint64_t add_apart(uint64_t a, uint64_t b) {
    float a0, a1, b0, b1;
    unpair(a, a0, a1);
    unpair(b, b0, b1);
    return pair(add1(a0, b0), add1(a1, b1));
}

// Queries.  x: the pairs' first elements, y: their second ones, two and two.
template <int D, int N, bool NEXT>
__device__ __forceinline__ void rope_queries(const KvRopeArgs &a, const uint4 (&raw)[N], const uint4 weights, const Fours at,
                                             int64_t token, int position, int head0) {
    constexpr int kLanes = D / 8, kTeams = 32 / kLanes;
    const int lane = threadIdx.x & 31, l = lane % kLanes, team = lane / kLanes;
    const int heads = static_cast<int>(a.q_heads), rot = static_cast<int>(a.rot_dim);
    uint64_t c[2] = {}, s[2] = {}, wx[2] = {}, wy[2] = {};
    if (at.turns) {
        const float *row = a.cos_sin + static_cast<int64_t>(position) * rot + 4 * l;
        const float4 cc = *reinterpret_cast<const float4 *>(row), ss = *reinterpret_cast<const float4 *>(row + rot / 2);
        c[0] = pair(cc.x, cc.y), c[1] = pair(cc.z, cc.w), s[0] = pair(ss.x, ss.y), s[1] = pair(ss.z, ss.w);
    }
    // neighbours: (x0, y0), (x1, y1), ... to (x0, x1), (y0, y1), ...
    auto split = [&](uint4 u, uint64_t (&x)[2], uint64_t (&y)[2]) {
        if constexpr (NEXT) {
            x[0] = pair(bf16lo_to_f32(u.x), bf16lo_to_f32(u.y)), y[0] = pair(bf16hi_to_f32(u.x), bf16hi_to_f32(u.y));
            x[1] = pair(bf16lo_to_f32(u.z), bf16lo_to_f32(u.w)), y[1] = pair(bf16hi_to_f32(u.z), bf16hi_to_f32(u.w));
        } else {
            unpack4(make_uint2(u.x, u.y), x[0], x[1]);
            unpack4(make_uint2(u.z, u.w), y[0], y[1]);
        }
    };
    const bool norm = a.q_weight != nullptr;
    if (norm) split(weights, wx, wy);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int h = head0 + i * kTeams + team;
        uint64_t x[2], y[2];
        split(raw[i], x, y);
        if (norm) {
            const uint64_t sq = fma2(y[1], y[1], fma2(y[0], y[0], fma2(x[1], x[1], mul2(x[0], x[0]))));
            float s0, s1;
            unpair(sq, s0, s1);
            float sum = s0 + s1;
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float r = rsqrt_once(fmaf(sum, 1.0f / D, a.eps), 0.0f);
            const uint64_t r2 = pair(r, r);
#pragma unroll
            for (int j = 0; j < 2; ++j) x[j] = mul2(mul2(x[j], r2), wx[j]), y[j] = mul2(mul2(y[j], r2), wy[j]);
        }
        if (at.turns) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint64_t o1 = add_apart(mul2(x[j], c[j]), neg2(mul2(y[j], s[j])));
                y[j] = add_apart(mul2(y[j], c[j]), mul2(x[j], s[j]));
                x[j] = o1;
            }
        }
        if (h < heads) {
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.q_out) + (token * heads + h) * D;
            if constexpr (NEXT) {
                float x0, x1, x2, x3, y0, y1, y2, y3;
                unpair(x[0], x0, x1), unpair(x[1], x2, x3), unpair(y[0], y0, y1), unpair(y[1], y2, y3);
                *reinterpret_cast<uint4 *>(out + at.first) =
                    make_uint4(f32x2_to_bf16x2(x0, y0), f32x2_to_bf16x2(x1, y1), f32x2_to_bf16x2(x2, y2), f32x2_to_bf16x2(x3, y3));
            } else {
                *reinterpret_cast<uint2 *>(out + at.first) = make_uint2(pack2(x[0]), pack2(x[1]));
                *reinterpret_cast<uint2 *>(out + at.second) = make_uint2(pack2(y[0]), pack2(y[1]));
            }
        }
    }
}

// Keys and values: 8 consecutive elements a lane.
template <int D, int N, bool F4, bool KEYS, bool NEXT>
__device__ __forceinline__ void rope_cached(const KvRopeArgs &a, const uint4 (&raw)[N], const uint4 weights, float scale,
                                            int64_t token, int64_t slot, int position, int head0) {
    constexpr int kLanes = D / 8, kTeams = 32 / kLanes;
    const int lane = threadIdx.x & 31, l = lane % kLanes, team = lane / kLanes;
    const int heads = static_cast<int>(a.kv_heads), rot = static_cast<int>(a.rot_dim), half = rot / 2;
    const bool norm = KEYS && a.k_weight != nullptr, turns = KEYS && 8 * l < rot, low = 8 * l < half;
    uint64_t w[4] = {}, c[4] = {}, s[4] = {};
    if (norm) {
        unpack4(make_uint2(weights.x, weights.y), w[0], w[1]);
        unpack4(make_uint2(weights.z, weights.w), w[2], w[3]);
    }
    if (turns) {
        const float *row = a.cos_sin + static_cast<int64_t>(position) * rot;
        if constexpr (NEXT) {
            const float4 cc = *reinterpret_cast<const float4 *>(row + 4 * l);
            const float4 ss = *reinterpret_cast<const float4 *>(row + half + 4 * l);
            const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) c[j] = pair(cv[j], cv[j]), s[j] = pair(-sv[j], sv[j]);
        } else {
            const float *p = row + (low ? 8 * l : 8 * l - half);
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                const float4 cc = *reinterpret_cast<const float4 *>(p + 2 * j);
                const float4 ss = *reinterpret_cast<const float4 *>(p + half + 2 * j);
                c[j] = pair(cc.x, cc.y), c[j + 1] = pair(cc.z, cc.w);
                s[j] = pair(ss.x, ss.y), s[j + 1] = pair(ss.z, ss.w);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] = low ? neg2(s[j]) : s[j];
        }
    }
    // the lane with the other elements of this lane's pairs
    const int partner = !turns ? lane : low ? lane + half / 8 : lane - half / 8;
    uint8_t *cache = KEYS ? a.k_cache : a.v_cache;
    const float recip = safe_reciprocal(scale);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int h = head0 + i * kTeams + team;
        uint64_t v[4];
        unpack4(make_uint2(raw[i].x, raw[i].y), v[0], v[1]);
        unpack4(make_uint2(raw[i].z, raw[i].w), v[2], v[3]);
        if (norm) {
            // two sums of exact squares, each with what its roundings lost
            uint64_t sum = mul2(v[0], v[0]), rest = 0;
#pragma unroll
            for (int j = 1; j < 4; ++j) {
                const uint64_t t = fma2(v[j], v[j], sum), z = add2(t, neg2(sum));
                rest = add2(rest, add2(add2(sum, neg2(add2(t, neg2(z)))), fma2(v[j], v[j], neg2(z))));
                sum = t;
            }
            float s0, s1, r0, r1;
            unpair(sum, s0, s1);
            unpair(rest, r0, r1);
            Two all = two_sum(s0, s1);
            all.l += r0 + r1;
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) {
                const float oh = __shfl_xor_sync(0xffffffffu, all.h, o), ol = __shfl_xor_sync(0xffffffffu, all.l, o);
                const Two t = two_sum(all.h, oh);
                all = Two{t.h, add1(add1(all.l, ol), t.l)};
            }
            const Two m = two_sum(mul1(all.h, 1.0f / D), a.eps);
            const float r = rsqrt_once(m.h, fma1(all.l, 1.0f / D, m.l));
            const uint64_t r2 = pair(r, r);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = mul2(mul2(v[j], r2), w[j]);
        }
        float x[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) unpair(v[j], x[2 * j], x[2 * j + 1]);
        if (KEYS) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint64_t other;
                if constexpr (NEXT) other = pair(x[2 * j + 1], x[2 * j]);
                else other = pair(__shfl_sync(0xffffffffu, x[2 * j], partner), __shfl_sync(0xffffffffu, x[2 * j + 1], partner));
                v[j] = turns ? add_apart(mul2(v[j], c[j]), mul2(other, s[j])) : v[j];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) unpair(v[j], x[2 * j], x[2 * j + 1]);
        }
        if constexpr (F4) {
            // a group is two lanes; NaN is above every magnitude
            uint32_t mx = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) mx = max(mx, __float_as_uint(x[j]) & 0x7FFFFFFFu);
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            const uint32_t sc = f32x2_to_e4m3x2(__fdiv_rn(__uint_as_float(mx), mul1(6.0f, scale)), 0.0f) & 0xFFu;
            const float den = mul1(f16x2_to_f32x2(e4m3x2_to_f16x2(sc)).x, scale);
            uint32_t codes = 0;
            if (den > 0.0f)
                codes = codes_of<uint32_t>(x, den, safe_reciprocal(den), [](const float (&q)[8]) { return f32x8_to_e2m1x8(q); });
            if (h < heads) {
                const uint32_t tpp = static_cast<uint32_t>(a.page_size / kKv4Tile);
                const uint32_t tile = static_cast<uint32_t>(slot) / kKv4Tile, row = static_cast<uint32_t>(slot) % kKv4Tile;
                const uint32_t blk = tile / tpp;
                uint8_t *t = cache + ((static_cast<int64_t>(blk) * heads + h) * tpp + (tile - blk * tpp)) * kv4_tile_bytes(D);
                *reinterpret_cast<uint32_t *>(t + row * (D / 2) + 4 * l) = codes;
                if ((l & 1) == 0) t[8 * D + row * (D / 16) + l / 2] = static_cast<uint8_t>(sc);
            }
        } else {
            const uint64_t codes = codes_of<uint64_t>(x, scale, recip, [](const float (&q)[8]) {
                uint32_t o[2];
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    o[j] = f32x2_to_e4m3x2(q[4 * j], q[4 * j + 1]) |
                           static_cast<uint32_t>(f32x2_to_e4m3x2(q[4 * j + 2], q[4 * j + 3])) << 16;
                return static_cast<uint64_t>(o[1]) << 32 | o[0];
            });
            if (h < heads) *reinterpret_cast<uint64_t *>(cache + (slot * heads + h) * D + 8 * l) = codes;
        }
    }
}

// A warp has up to N * (256 / D) heads of one kind of one token; q_warps and
// kv_warps of them make a token's q, k and v.  `inverse` = ceil(2^64 / warps a
// token) divides every warp number below 2^47 exactly by a multiplication.  The
// heads are loaded before the token's place is known: two loads one after the
// other to the cos and sin instead of three.
template <int D, int N, bool F4, bool NEXT>
__global__ void __launch_bounds__(kRopeThreads, 6) kv_rope_kernel(const KvRopeArgs a, uint64_t inverse, int q_warps, int kv_warps) {
    constexpr int kHeads = N * (256 / D), kLanes = D / 8, kTeams = 32 / kLanes;
    const int lane = threadIdx.x & 31, l = lane % kLanes, team = lane / kLanes;
    const uint64_t warp = static_cast<uint64_t>(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5);
    const int64_t token = static_cast<int64_t>(__umul64hi(warp, inverse));
    const int part = static_cast<int>(warp - token * (q_warps + 2 * kv_warps));
    const int kind = part < q_warps ? kRopeQ : part < q_warps + kv_warps ? kRopeK : kRopeV;
    const int at = kind == kRopeQ ? part : kind == kRopeK ? part - q_warps : part - q_warps - kv_warps;
    pdl_wait();
    if (token >= a.tokens) return;
    const int heads = static_cast<int>(kind == kRopeQ ? a.q_heads : a.kv_heads), head0 = at * kHeads;
    const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(kind == kRopeQ ? a.q : kind == kRopeK ? a.k : a.v) +
                               token * (kind == kRopeQ ? a.q_stride : kind == kRopeK ? a.k_stride : a.v_stride);
    const int position = a.positions[token];
    const int64_t slot = a.slots[token];
    const Fours f = fours_of<D, NEXT>(kind, l, static_cast<int>(a.rot_dim));
    uint4 raw[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int h = head0 + i * kTeams + team;
        raw[i] = make_uint4(0, 0, 0, 0);
        if (h < heads) {
            if (f.second == f.first + 4) {
                raw[i] = ld_v4(src + h * D + f.first);
            } else {
                const uint2 u = ld_v2(src + h * D + f.first), v = ld_v2(src + h * D + f.second);
                raw[i] = make_uint4(u.x, u.y, v.x, v.y);
            }
        }
    }
    // what all tokens share, in the same round trip
    const __nv_bfloat16 *wp = static_cast<const __nv_bfloat16 *>(kind == kRopeQ ? a.q_weight : kind == kRopeK ? a.k_weight : nullptr);
    uint4 weights = make_uint4(0, 0, 0, 0);
    if (wp) {
        const uint2 u = *reinterpret_cast<const uint2 *>(wp + f.first), v = *reinterpret_cast<const uint2 *>(wp + f.second);
        weights = make_uint4(u.x, u.y, v.x, v.y);
    }
    const float scale = *(kind == kRopeV ? a.v_scale : a.k_scale);
    if (position < 0 || position >= a.max_pos) {
        if (position != -1 && part == 0 && lane == 0) atomicOr(&g_rope_err, ERRBIT_INDEX);
        return;
    }
    if (kind == kRopeQ) {
        rope_queries<D, N, NEXT>(a, raw, weights, f, token, position, head0);
        return;
    }
    if (slot < 0 || slot >= a.num_slots) {
        if (slot != -1 && at == 0 && kind == kRopeK && lane == 0) atomicOr(&g_rope_err, ERRBIT_INDEX);
        return;
    }
    if (kind == kRopeK) rope_cached<D, N, F4, true, NEXT>(a, raw, weights, scale, token, slot, position, head0);
    else rope_cached<D, N, F4, false, NEXT>(a, raw, weights, scale, token, slot, position, head0);
}

template <int D, int N, bool F4, bool NEXT>
cudaError_t launch_rope(const KvRopeArgs &a, cudaStream_t stream) {
    constexpr int64_t kHeads = N * (256 / D);
    const int64_t q_warps = (a.q_heads + kHeads - 1) / kHeads, kv_warps = (a.kv_heads + kHeads - 1) / kHeads;
    const int64_t per_token = q_warps + 2 * kv_warps, warps = a.tokens * per_token, per = kRopeThreads / 32;
    const int64_t blocks = (warps + per - 1) / per;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    const uint64_t inverse = ~uint64_t{0} / static_cast<uint64_t>(per_token) + 1;  // per_token >= 3
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(kRopeThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_rope_kernel<D, N, F4, NEXT>, a, inverse, static_cast<int>(q_warps),
                              static_cast<int>(kv_warps));
}

template <int D, bool F4, bool NEXT>
cudaError_t launch_rope_split(const KvRopeArgs &a, cudaStream_t stream) {
    return a.tokens >= 512 ? launch_rope<D, 2, F4, NEXT>(a, stream) : launch_rope<D, 1, F4, NEXT>(a, stream);
}

}  // namespace

cudaError_t launch_kv_rope(const KvRopeArgs &a, bool four_bit, cudaStream_t stream) {
    if (!four_bit) return a.interleaved ? launch_rope_split<128, false, true>(a, stream) : launch_rope_split<128, false, false>(a, stream);
    if (a.head_dim == 128)
        return a.interleaved ? launch_rope_split<128, true, true>(a, stream) : launch_rope_split<128, true, false>(a, stream);
    return a.interleaved ? launch_rope_split<64, true, true>(a, stream) : launch_rope_split<64, true, false>(a, stream);
}

uint32_t take_rope_error() {
    uint32_t v = 0;
    if (cudaMemcpyFromSymbol(&v, g_rope_err, sizeof v) != cudaSuccess) return 0xFFFFFFFFu;
    const uint32_t zero = 0;
    cudaMemcpyToSymbol(g_rope_err, &zero, sizeof zero);
    return v;
}

}  // namespace fp8bs
