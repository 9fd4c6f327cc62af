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
// an exact residual corrects the square root's reciprocal; for |a| below 2^50 and
// mean a^2 + eps from 2^-100 on, beyond which the low parts are subnormal.  With a
// plain fp32 sum r is off by a unit in the last place for every third head, and a
// 4-bit code in some ten million with it; queries, which end in bf16, have that.
#include "twofloat.cuh"

#include "serving.cuh"
#include "internal.h"

namespace fp8bs {

namespace {

__device__ uint32_t g_rope_err;

constexpr int kRopeThreads = 128;

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

// The codes of x / s without a division: q = x (1 / s) is within 2^-23 of the
// quotient, so if q (1 - 2^-21) and q (1 + 2^-21) have one code, the rounded
// quotient has it too; a value near a border between codes is divided (one in
// some hundred thousand).  encode(v) gives the codes of v[0 .. 7]; `recip` is RN(1 / s) for
// s in [2^-100, 2^100], or 0: every value is divided.
template <class Word, class Encode>
__device__ __forceinline__ Word codes_of(const uint64_t *x, float s, float recip, Encode encode) {
    float lo[8], hi[8];
    if (recip != 0.0f) {
        const uint64_t y2 = pair(recip, recip), down = pair(1.0f - 0x1p-21f, 1.0f - 0x1p-21f);
        const uint64_t up = pair(1.0f + 0x1p-21f, 1.0f + 0x1p-21f);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const uint64_t q = mul2(x[j / 2], y2);
            unpair(mul2(q, down), lo[j], lo[j + 1]);
            unpair(mul2(q, up), hi[j], hi[j + 1]);
        }
        const Word a = encode(lo), b = encode(hi);
        if (a == b) return a;
    }
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        float a, b;
        unpair(x[j / 2], a, b);
        lo[j] = __fdiv_rn(a, s), lo[j + 1] = __fdiv_rn(b, s);
    }
    return encode(lo);
}
__device__ __forceinline__ float safe_reciprocal(float s) { return s >= 0x1p-100f && s <= 0x1p100f ? __frcp_rn(s) : 0.0f; }

enum RopeKind : int { kRopeQ = 0, kRopeK = 1, kRopeV = 2 };

// Eight bf16 numbers to pairs of fp32: (0, 1), (2, 3), ...
__device__ __forceinline__ void unpack8(uint4 u, uint64_t *x) {
    x[0] = pair(bf16lo_to_f32(u.x), bf16hi_to_f32(u.x)), x[1] = pair(bf16lo_to_f32(u.y), bf16hi_to_f32(u.y));
    x[2] = pair(bf16lo_to_f32(u.z), bf16hi_to_f32(u.z)), x[3] = pair(bf16lo_to_f32(u.w), bf16hi_to_f32(u.w));
}
// Sixteen to the even ones, (0, 2), (4, 6), ..., and the odd ones.
__device__ __forceinline__ void unpack_apart(uint4 u, uint4 v, uint64_t *even, uint64_t *odd) {
    even[0] = pair(bf16lo_to_f32(u.x), bf16lo_to_f32(u.y)), odd[0] = pair(bf16hi_to_f32(u.x), bf16hi_to_f32(u.y));
    even[1] = pair(bf16lo_to_f32(u.z), bf16lo_to_f32(u.w)), odd[1] = pair(bf16hi_to_f32(u.z), bf16hi_to_f32(u.w));
    even[2] = pair(bf16lo_to_f32(v.x), bf16lo_to_f32(v.y)), odd[2] = pair(bf16hi_to_f32(v.x), bf16hi_to_f32(v.y));
    even[3] = pair(bf16lo_to_f32(v.z), bf16lo_to_f32(v.w)), odd[3] = pair(bf16hi_to_f32(v.z), bf16hi_to_f32(v.w));
}
__device__ __forceinline__ uint32_t pack2(uint64_t v) {
    float a, b;
    unpair(v, a, b);
    return f32x2_to_bf16x2(a, b);
}
__device__ __forceinline__ uint4 pack8(const uint64_t *x) {
    return make_uint4(pack2(x[0]), pack2(x[1]), pack2(x[2]), pack2(x[3]));
}
// (x0, y0), (x1, y1) of the pairs (x0, x1), (y0, y1)
__device__ __forceinline__ void pack_together(uint64_t x, uint64_t y, uint32_t &a, uint32_t &b) {
    float x0, x1, y0, y1;
    unpair(x, x0, x1);
    unpair(y, y0, y1);
    a = f32x2_to_bf16x2(x0, y0), b = f32x2_to_bf16x2(x1, y1);
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
__device__ __forceinline__ uint64_t sub_apart(uint64_t a, uint64_t b) {
    float a0, a1, b0, b1;
    unpair(a, a0, a1);
    unpair(b, b0, b1);
    return pair(sub1(a0, b0), sub1(a1, b1));
}
__device__ __forceinline__ void load_pairs8(const float *p, uint64_t *x) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    x[0] = pair(a.x, a.y), x[1] = pair(a.z, a.w), x[2] = pair(b.x, b.y), x[3] = pair(b.z, b.w);
}

// A head is D / 16 lanes' of 16 elements each.  With halves a lane whose elements
// turn has eight and the eight that turn with them; else 16 consecutive ones,
// neighbours that turn together or, of a value, a group of the 4-bit cache.
template <int D>
struct Lanes {
    static constexpr int kPerHead = D / 16, kHeads = 32 / kPerHead;
    int l, head;  // lane of the head, head of the warp
    __device__ __forceinline__ Lanes() : l(threadIdx.x % kPerHead), head((threadIdx.x & 31) / kPerHead) {}
};

template <int D, bool NEXT>
__device__ __forceinline__ void rope_queries(const KvRopeArgs &a, int64_t token, int part) {
    using L = Lanes<D>;
    const L me;
    const int heads = static_cast<int>(a.q_heads), h = part * L::kHeads + me.head, rot = static_cast<int>(a.rot_dim);
    const int half = rot / 2;
    const bool turns = 8 * me.l < half, there = h < heads;
    const int first = NEXT || !turns ? 16 * me.l : 8 * me.l, second = NEXT || !turns ? first + 8 : half + 8 * me.l;
    const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.q) + token * a.q_stride + h * D;
    const int position = a.positions[token];
    uint4 u = make_uint4(0, 0, 0, 0), v = u, wu = u, wv = u;
    if (there) u = ld_v4(src + first), v = ld_v4(src + second);
    const __nv_bfloat16 *wp = static_cast<const __nv_bfloat16 *>(a.q_weight);
    if (wp) wu = *reinterpret_cast<const uint4 *>(wp + first), wv = *reinterpret_cast<const uint4 *>(wp + second);
    if (position < 0 || position >= a.max_pos) {
        if (position != -1 && part == 0 && (threadIdx.x & 31) == 0) atomicOr(&g_rope_err, ERRBIT_INDEX);
        return;
    }
    uint64_t c[4], s[4], x[4], y[4];
    if (turns) {
        const float *row = a.cos_sin + static_cast<int64_t>(position) * rot + 8 * me.l;
        load_pairs8(row, c);
        load_pairs8(row + half, s);
    }
    if constexpr (NEXT) {
        unpack_apart(u, v, x, y);
    } else {
        unpack8(u, x);
        unpack8(v, y);
    }
    if (wp) {
        uint64_t sq = mul2(x[0], x[0]);
#pragma unroll
        for (int j = 1; j < 4; ++j) sq = fma2(x[j], x[j], sq);
#pragma unroll
        for (int j = 0; j < 4; ++j) sq = fma2(y[j], y[j], sq);
        float s0, s1;
        unpair(sq, s0, s1);
        float sum = s0 + s1;
#pragma unroll
        for (int o = L::kPerHead / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float r = rsqrt_once(fmaf(sum, 1.0f / D, a.eps), 0.0f);
        const uint64_t r2 = pair(r, r);
        uint64_t wx[4], wy[4];
        if constexpr (NEXT) {
            unpack_apart(wu, wv, wx, wy);
        } else {
            unpack8(wu, wx);
            unpack8(wv, wy);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = mul2(mul2(x[j], r2), wx[j]), y[j] = mul2(mul2(y[j], r2), wy[j]);
    }
    if (turns) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint64_t o1 = sub_apart(mul2(x[j], c[j]), mul2(y[j], s[j]));
            y[j] = add_apart(mul2(y[j], c[j]), mul2(x[j], s[j]));
            x[j] = o1;
        }
    }
    if (!there) return;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.q_out) + (token * heads + h) * D;
    if constexpr (NEXT) {
        pack_together(x[0], y[0], u.x, u.y), pack_together(x[1], y[1], u.z, u.w);
        pack_together(x[2], y[2], v.x, v.y), pack_together(x[3], y[3], v.z, v.w);
    } else {
        u = pack8(x), v = pack8(y);
    }
    *reinterpret_cast<uint4 *>(out + first) = u;
    *reinterpret_cast<uint4 *>(out + second) = v;
}

// KEYS with halves: a lane's eights can be of two groups of the 4-bit cache, whose
// other eights are another lane's; its largest magnitudes come by shuffles.
template <int D, bool F4, bool KEYS, bool NEXT>
__device__ __forceinline__ void rope_cached(const KvRopeArgs &a, int64_t token, int part) {
    using L = Lanes<D>;
    constexpr bool kApart = KEYS && !NEXT;
    const L me;
    const int heads = static_cast<int>(a.kv_heads), h = part * L::kHeads + me.head, rot = static_cast<int>(a.rot_dim);
    const int half = rot / 2, lane = threadIdx.x & 31;
    const bool there = h < heads, turns = KEYS && 8 * me.l < half;
    const int first = kApart && turns ? 8 * me.l : 16 * me.l, second = kApart && turns ? half + 8 * me.l : first + 8;
    const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(KEYS ? a.k : a.v) +
                               token * (KEYS ? a.k_stride : a.v_stride) + h * D;
    const int position = a.positions[token];
    const int64_t slot = a.slots[token];
    const float scale = *(KEYS ? a.k_scale : a.v_scale);
    uint4 u = make_uint4(0, 0, 0, 0), v = u, wu = u, wv = u;
    if (there) u = ld_v4(src + first), v = ld_v4(src + second);
    const __nv_bfloat16 *wp = KEYS ? static_cast<const __nv_bfloat16 *>(a.k_weight) : nullptr;
    if (wp) wu = *reinterpret_cast<const uint4 *>(wp + first), wv = *reinterpret_cast<const uint4 *>(wp + second);
    if (position < 0 || position >= a.max_pos) return;
    if (slot < 0 || slot >= a.num_slots) {
        if (KEYS && slot != -1 && part == 0 && lane == 0) atomicOr(&g_rope_err, ERRBIT_INDEX);
        return;
    }
    uint64_t x[8];  // what turns together: x[j] and x[j + 4]
    if (KEYS && NEXT) {
        unpack_apart(u, v, x, x + 4);
    } else {
        unpack8(u, x);
        unpack8(v, x + 4);
    }
    if (KEYS) {
        uint64_t c[4], s[4];
        if (turns) {
            const float *row = a.cos_sin + static_cast<int64_t>(position) * rot + 8 * me.l;
            load_pairs8(row, c);
            load_pairs8(row + half, s);
        }
        if (wp) {
            // two sums of exact squares, each with what its roundings lost
            uint64_t sum = mul2(x[0], x[0]), rest = 0;
#pragma unroll
            for (int j = 1; j < 8; ++j) {
                const uint64_t t = fma2(x[j], x[j], sum), z = add2(t, neg2(sum));
                rest = add2(rest, add2(add2(sum, neg2(add2(t, neg2(z)))), fma2(x[j], x[j], neg2(z))));
                sum = t;
            }
            float s0, s1, r0, r1;
            unpair(sum, s0, s1);
            unpair(rest, r0, r1);
            Two all = two_sum(s0, s1);
            all.l += r0 + r1;
#pragma unroll
            for (int o = L::kPerHead / 2; o > 0; o >>= 1) {
                const float oh = __shfl_xor_sync(0xffffffffu, all.h, o), ol = __shfl_xor_sync(0xffffffffu, all.l, o);
                const Two t = two_sum(all.h, oh);
                all = Two{t.h, add1(add1(all.l, ol), t.l)};
            }
            const Two m = two_sum(mul1(all.h, 1.0f / D), a.eps);
            const float r = rsqrt_once(m.h, fma1(all.l, 1.0f / D, m.l));
            const uint64_t r2 = pair(r, r);
            uint64_t w[8];
            if (NEXT) {
                unpack_apart(wu, wv, w, w + 4);
            } else {
                unpack8(wu, w);
                unpack8(wv, w + 4);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = mul2(mul2(x[j], r2), w[j]);
        }
        if (turns) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint64_t o1 = sub_apart(mul2(x[j], c[j]), mul2(x[j + 4], s[j]));
                x[j + 4] = add_apart(mul2(x[j + 4], c[j]), mul2(x[j], s[j]));
                x[j] = o1;
            }
        }
        if constexpr (NEXT) {
            // back to the elements' order
            uint64_t t[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float x0, x1, y0, y1;
                unpair(x[j], x0, x1);
                unpair(x[j + 4], y0, y1);
                t[2 * j] = pair(x0, y0), t[2 * j + 1] = pair(x1, y1);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = t[j];
        }
    }
    uint8_t *cache = KEYS ? a.k_cache : a.v_cache;
    if constexpr (F4) {
        // NaN is above every magnitude
        uint32_t mx[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float a0, a1;
            unpair(x[j], a0, a1);
            mx[j / 4] = max(mx[j / 4], max(__float_as_uint(a0) & 0x7FFFFFFFu, __float_as_uint(a1) & 0x7FFFFFFFu));
        }
        if constexpr (kApart) {
            const int firsts = turns ? half / 8 : 0;  // eights that are lanes' first ones
            uint32_t other[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int eight = (turns ? (k ? second : first) / 8 : 2 * me.l + k) ^ 1;
                const bool is_second = turns ? eight >= firsts : k == 0;
                const int from = lane - me.l + (turns ? eight - (is_second ? firsts : 0) : me.l);
                const uint32_t m0 = __shfl_sync(0xffffffffu, mx[0], from), m1 = __shfl_sync(0xffffffffu, mx[1], from);
                other[k] = is_second ? m1 : m0;
            }
            mx[0] = max(mx[0], other[0]), mx[1] = max(mx[1], other[1]);
        } else {
            mx[0] = mx[1] = max(mx[0], mx[1]);
        }
        const float scale6 = mul1(6.0f, scale);
        uint32_t sc[2], codes[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (k == 0 || kApart) sc[k] = f32x2_to_e4m3x2(__fdiv_rn(__uint_as_float(mx[k]), scale6), 0.0f) & 0xFFu;
            else sc[k] = sc[0];
            const float den = mul1(f16x2_to_f32x2(e4m3x2_to_f16x2(sc[k])).x, scale);
            codes[k] = 0;
            if (den > 0.0f)
                codes[k] = codes_of<uint32_t>(x + 4 * k, den, safe_reciprocal(den),
                                              [](const float (&q)[8]) { return f32x8_to_e2m1x8(q); });
        }
        if (there) {
            const uint32_t tpp = static_cast<uint32_t>(a.page_size / kKv4Tile);
            const uint32_t tile = static_cast<uint32_t>(slot) / kKv4Tile, row = static_cast<uint32_t>(slot) % kKv4Tile;
            const uint32_t blk = tile / tpp;
            uint8_t *t = cache + ((static_cast<int64_t>(blk) * heads + h) * tpp + (tile - blk * tpp)) * kv4_tile_bytes(D);
            uint8_t *to = t + row * (D / 2), *to_scale = t + 8 * D + row * (D / 16);
            if constexpr (kApart) {
                *reinterpret_cast<uint32_t *>(to + first / 2) = codes[0];
                *reinterpret_cast<uint32_t *>(to + second / 2) = codes[1];
                if (first % 16 == 0) to_scale[first / 16] = static_cast<uint8_t>(sc[0]);
                if (second % 16 == 0) to_scale[second / 16] = static_cast<uint8_t>(sc[1]);
            } else {
                *reinterpret_cast<uint2 *>(to + 8 * me.l) = make_uint2(codes[0], codes[1]);
                to_scale[me.l] = static_cast<uint8_t>(sc[0]);
            }
        }
    } else {
        const float recip = safe_reciprocal(scale);
        auto encode = [](const float (&q)[8]) {
            uint32_t o[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                o[j] = f32x2_to_e4m3x2(q[4 * j], q[4 * j + 1]) |
                       static_cast<uint32_t>(f32x2_to_e4m3x2(q[4 * j + 2], q[4 * j + 3])) << 16;
            return static_cast<uint64_t>(o[1]) << 32 | o[0];
        };
        const uint64_t c0 = codes_of<uint64_t>(x, scale, recip, encode), c1 = codes_of<uint64_t>(x + 4, scale, recip, encode);
        if (there) {
            uint8_t *to = cache + (slot * heads + h) * D;
            if constexpr (kApart) {
                *reinterpret_cast<uint64_t *>(to + first) = c0;
                *reinterpret_cast<uint64_t *>(to + second) = c1;
            } else {
                *reinterpret_cast<uint4 *>(to + first) =
                    make_uint4(static_cast<uint32_t>(c0), static_cast<uint32_t>(c0 >> 32), static_cast<uint32_t>(c1),
                               static_cast<uint32_t>(c1 >> 32));
            }
        }
    }
}

// A warp has 512 / D heads of one kind of one token: 2 * kv_blocks CTAs of keys
// and values, which take longer, come before those of queries.  The inverses are
// ceil(2^64 / warps a token), which divide every warp number below 2^47 exactly by
// a multiplication (0: one warp).  A token's place, its heads and the weights are
// one round trip, cos and sin the second.
//
// Floor: every byte of q, k, v read once, q's written, the cache's rows written.
// At D = 128, 32 query and 8 key and value heads, 8191 tokens into the FP8 cache
// (189 MB): 43.7 us, 4.3 TB/s; 4099 tokens of 64 and 8, half of each rotated, no norms (161 MB): 32.9 us, 4.9 TB/s;
// 64 tokens 2.15 us.  What bounds it is latency: two dependent round
// trips and some 200 instructions a warp, 32 warps an SM.  Warps an SM, at 8191
// tokens: 24 53.6 us, 32 45.8, 40 47.0 (48 registers, which spill).  Threads a CTA:
// 64 43.3 us, 128 43.7, 256 45.8, 512 49.6, since a CTA's registers are free when
// its last warp is done; at 64 tokens 64 takes 2.3 us, 128 2.15.  A lane with 8
// elements (a third more instructions a byte, 48 warps an SM) took 51.6 us, a warp
// with several tokens one after the other, the next one's heads loaded ahead into
// registers 44 to 106, into shared memory 59 to 86.
template <int D, bool F4, bool NEXT>
__global__ void __launch_bounds__(kRopeThreads, 8) kv_rope_kernel(const __grid_constant__ KvRopeArgs a, uint32_t kv_blocks,
                                                                  uint64_t kv_inverse, uint64_t q_inverse) {
    using L = Lanes<D>;
    const bool q = blockIdx.x >= 2 * kv_blocks;
    const uint32_t block = q ? blockIdx.x - 2 * kv_blocks : blockIdx.x >> 1;
    const uint64_t warp = static_cast<uint64_t>(block) * (kRopeThreads / 32) + (threadIdx.x >> 5);
    const uint64_t inverse = q ? q_inverse : kv_inverse;
    const int64_t token = static_cast<int64_t>(inverse ? __umul64hi(warp, inverse) : warp);
    const uint32_t heads = static_cast<uint32_t>(q ? a.q_heads : a.kv_heads), per = (heads + L::kHeads - 1) / L::kHeads;
    const int part = static_cast<int>(warp - token * per);
    pdl_wait();
    if (token >= a.tokens) return;
    if (q) rope_queries<D, NEXT>(a, token, part);
    else if (blockIdx.x & 1) rope_cached<D, F4, false, NEXT>(a, token, part);
    else rope_cached<D, F4, true, NEXT>(a, token, part);
}

template <int D, bool F4, bool NEXT>
cudaError_t launch_rope_t(const KvRopeArgs &a, cudaStream_t stream) {
    constexpr int64_t kHeads = Lanes<D>::kHeads, kWarps = kRopeThreads / 32;
    const int64_t q_per = (a.q_heads + kHeads - 1) / kHeads, kv_per = (a.kv_heads + kHeads - 1) / kHeads;
    const int64_t q_blocks = (a.tokens * q_per + kWarps - 1) / kWarps, kv_blocks = (a.tokens * kv_per + kWarps - 1) / kWarps;
    if (q_blocks + 2 * kv_blocks > 0x7fffffff) return cudaErrorInvalidValue;
    auto inverse = [](int64_t per) { return per == 1 ? uint64_t{0} : ~uint64_t{0} / static_cast<uint64_t>(per) + 1; };
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(q_blocks + 2 * kv_blocks), 1, 1);
    cfg.blockDim = dim3(kRopeThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_rope_kernel<D, F4, NEXT>, a, static_cast<uint32_t>(kv_blocks), inverse(kv_per),
                              inverse(q_per));
}

template <int D, bool F4>
cudaError_t launch_rope(const KvRopeArgs &a, cudaStream_t stream) {
    return a.interleaved ? launch_rope_t<D, F4, true>(a, stream) : launch_rope_t<D, F4, false>(a, stream);
}

}  // namespace

cudaError_t launch_kv_rope(const KvRopeArgs &a, bool four_bit, cudaStream_t stream) {
    if (!four_bit) return launch_rope<128, false>(a, stream);
    return a.head_dim == 128 ? launch_rope<128, true>(a, stream) : launch_rope<64, true>(a, stream);
}

uint32_t take_rope_error() {
    uint32_t v = 0;
    if (cudaMemcpyFromSymbol(&v, g_rope_err, sizeof v) != cudaSuccess) return 0xFFFFFFFFu;
    const uint32_t zero = 0;
    cudaMemcpyToSymbol(g_rope_err, &zero, sizeof zero);
    return v;
}

}  // namespace fp8bs
