// route.cu -- the two ends of a layer of routed experts: which experts a token
// goes to and with which weights, and the weighted sum of what they gave.
//
// Route, a warp a token.  s = softmax(x) or 1 / (1 + e^-x); experts are chosen
// by c = s + bias.  Whole numbers come out, so near ties have to be decided as
// the definition decides them: c is compared in multiples of 2^-44.  The choice
// is made in fp32 first, and stands if what it told apart is further apart than
// c can be off; else (one token in some thousands) it is made again with pairs
// of fp32.  Without a bias or groups it goes by the logits themselves.
//
// Floor: the logits read once (8192 tokens of 256 experts in fp32: 8.9 MB, 1.3 us).
// Measured 14.6 us (sigmoid, bias, the best 4 of 8 groups; 8 of 256), 9.7 (softmax,
// 12 of 256, no bias), 14.6 (softmax, 3 of 8 groups, 6 of 160) and 3.3 for 32 tokens,
// most of it the launch and the chain of dependent steps.  What bounds the prompt is
// instructions, 1090 and 860 a token, ALU first: the scores, the groups, the order
// keys.  With pairs of fp32 for every token it took 36.5 us; with the largest left
// taken topk times in place of a rank among the few that can be chosen 18.9, 13.8 and
// 4.2.  Warps an SM: 16 20.0 us (with those rounds), 32 16.9 and 9.8, 40 17.1 and 9.7,
// 48 17.8 and 9.9.
#include "twofloat.cuh"

#include "serving.cuh"
#include "internal.h"

namespace fp8bs {

namespace {

constexpr int kRouteWarps = 4;
constexpr float kMostBias = 65536.0f;
constexpr float kNoScore = -104.0f;  // e^x below two_exp2's range

// Order of the values as unsigned integers above 0: -0 is +0, NaN below everything.
__device__ __forceinline__ uint32_t logit_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    return x != x ? 1u : u & 0x80000000u ? ~u : u | 0x80000000u;
}

// To the nearest whole number, for a number below 2^62.
__device__ __forceinline__ long long to_whole(float h, float l) {
    return fabsf(h) < 0x1p23f ? __float2ll_rn(h + l) : __float2ll_rn(h) + __float2ll_rn(l);
}
// c = s + bias in multiples of 2^-44, above 0, for s in [0, 1] and a bias of at most 2^16; NaN below everything.  A
// bias of 2^-20 and more is a whole number of them and added as one: a pair of fp32 near 65536 resolves 2^-32 only.
__device__ __forceinline__ uint64_t score_key(Two s, float bias) {
    long long v = 0;
    if (fabsf(bias) < 0x1p-20f) s = add(s, bias);
    else v = __float2ll_rn(bias * 0x1p44f);
    if (s.h != s.h || bias != bias) return 1;
    v += to_whole(s.h * 0x1p44f, s.l * 0x1p44f);
    return static_cast<uint64_t>(v + (1ll << 62));
}

// A bias as it counts: in [-kMostBias, kMostBias]; NaN stays NaN, as its c then is.
__device__ __forceinline__ float bias_of(float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(b), "f"(-kMostBias));
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(r) : "f"(kMostBias));
    return r;
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
// equals has the lowest expert.  sc: [experts] in shared memory, with groups.
template <bool F32, int EPL>
__device__ __noinline__ void route_exactly(const MoeScoreArgs &a, int64_t token, uint64_t *sc) {
    const int lane = threadIdx.x & 31;
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
            if (a.bias && e0 + i < experts) b = bias_of(a.bias[e0 + i]);
            key[i] = score_key(s[i], b);
        }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) mine |= e0 + i < experts ? 1u << i : 0u;
    if (a.groups > 1) {
        const int groups = static_cast<int>(a.groups), per = experts / groups;
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

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float reciprocal(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// e^(x - m) within 2^-21 of itself, x - m in [-104, 0]: the exponent's own error goes back in.
__device__ __forceinline__ float exp_near(float x, float m) {
    const Two t = times_log2e(two_sum(x, -m));
    const float e = ex2(t.h);
    return fmaf(e, t.l * 0.6931471805599453f, e);
}

struct Candidates {  // of a warp
    alignas(16) uint32_t key[32];
    int id[32];
};

// A token's experts by fp32 scores; false if they do not tell them apart.
template <bool F32, int EPL>
__device__ __forceinline__ bool route_quickly(const MoeScoreArgs &a, int64_t token, Candidates &sh) {
    constexpr float kLog2e = 1.4426950408889634f;
    const int lane = threadIdx.x & 31, experts = static_cast<int>(a.experts), topk = static_cast<int>(a.topk);
    const int groups = static_cast<int>(a.groups), per = groups > 1 ? experts / groups : experts;
    const int lanes = groups > 1 ? 32 >> (32 - __clz(groups - 1)) : 32;  // of a group, a power of two
    if (lanes * EPL < per) return false;
    // this lane's experts, e0 .. e0 + mine - 1: they rise with the lanes
    const int group = lane / lanes, begin = (lane % lanes) * EPL, left = group < groups ? per - begin : 0;
    const int e0 = group * per + begin, mine = left < 0 ? 0 : left < EPL ? left : EPL;
    const char *row = static_cast<const char *>(a.logits) + token * a.row_stride * (F32 ? 4 : 2);
    float x[EPL];
    constexpr int kBytes = EPL * (F32 ? 4 : 2);
    bool vector = false;
    if constexpr (kBytes >= 16) vector = (reinterpret_cast<uintptr_t>(row + e0 * (F32 ? 4 : 2)) & 15) == 0 && mine == EPL;
    if (vector) {
        if constexpr (kBytes >= 16) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i) {
                const uint4 v = ld_v4(row + e0 * (F32 ? 4 : 2) + 16 * i);
                const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (F32) x[4 * i + j] = __uint_as_float(u[j]);
                    else x[8 * i + 2 * j] = bf16lo_to_f32(u[j]), x[8 * i + 2 * j + 1] = bf16hi_to_f32(u[j]);
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) x[i] = i < mine ? load_logit<F32>(row, e0 + i) : -INFINITY;
    }
    float m = 0.0f, z = 1.0f;
    if (a.softmax) {
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i) m = fmaxf(m, x[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (!(fabsf(m) < INFINITY)) return false;
    }
    // ---- what the experts are ordered by: c, or the logit itself; 0: not there, or its group is not open
    const bool scored = a.bias != nullptr || groups > 1;
    uint32_t key[EPL];
    float c[EPL];
    float slack = 0.0f;  // c is within slack + 2^-22 |c|
    if (a.softmax || scored) {
        z = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            if (a.softmax) {
                c[i] = ex2((x[i] - m) * kLog2e);
                z += c[i];
            } else {
                c[i] = reciprocal(1.0f + ex2(-x[i] * kLog2e));
            }
        }
        if (a.softmax) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        }
        if (z != z) return false;
    }
    if (scored) {
        // Softmax: e^-d, d = m - x, is off by 2.5 2^-24 d and ex2's 2^-22 of itself, below 2^-21 of the largest; z by 2^-22,
        // 2^-23 and half a step for each of EPL + 5 additions; the quotient by 2^-22: to 256 experts 2^-19 of the largest
        // score.  Sigmoid, with u = e^-x: u / (1 + u) of u's 2.2 2^-24 |x| + 2^-22 reach s, 1 + u rounds once, the
        // reciprocal is within 2^-23: below 2^-21.
        const float to_score = a.softmax ? __fdividef(1.0f, z) : 1.0f;
        slack = a.softmax ? (EPL <= 8 ? 0x1p-19f : 0x1p-18f) * to_score : 0x1p-21f;
        float b[EPL] = {};
        bool wide = false;
        if constexpr (EPL >= 4) wide = a.bias && (reinterpret_cast<uintptr_t>(a.bias + e0) & 15) == 0 && mine == EPL;
        if (wide) {
            if constexpr (EPL >= 4) {
#pragma unroll
                for (int i = 0; i < EPL; i += 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(a.bias + e0 + i);
                    b[i] = v.x, b[i + 1] = v.y, b[i + 2] = v.z, b[i + 3] = v.w;
                }
            }
        } else if (a.bias) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) b[i] = i < mine ? a.bias[e0 + i] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) c[i] = fmaf(c[i], to_score, bias_of(b[i]));
    }
    bool open = true;
    if (groups > 1) {
        // ---- the groups' scores: the two best of the lane's experts, then of the group's lanes
        float b1 = -INFINITY, b2 = -INFINITY;
        bool nan = false;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const float v = i < mine ? c[i] : -INFINITY;
            nan |= v != v;
            b2 = fmaxf(b2, fminf(b1, v));
            b1 = fmaxf(b1, v);
        }
        if (__any_sync(0xffffffffu, nan)) return false;
        for (int o = 1; o < lanes; o <<= 1) {
            const float o1 = __shfl_xor_sync(0xffffffffu, b1, o), o2 = __shfl_xor_sync(0xffffffffu, b2, o);
            b2 = fmaxf(fmaxf(b2, o2), fminf(b1, o1));
            b1 = fmaxf(b1, o1);
        }
        const bool two = a.group_top == 2;
        const float score = two ? b1 + b2 : b1;
        int before = 0;
        for (int g = 0; g < groups; ++g) {
            const float other = __shfl_sync(0xffffffffu, score, g * lanes);
            before += other > score || (other == score && g < group) ? 1 : 0;
        }
        open = group < groups && before < static_cast<int>(a.topk_groups);
        if (a.topk_groups < a.groups) {
            // A score is off by what its parts are, which the sum does not tell: a large c and its opposite may cancel.
            // The last that is open, at its least, and the first that is not, at its most.
            const float off = 2.0f * (slack + 0x1p-22f * (fabsf(b1) + (two ? fabsf(b2) : 0.0f)));
            const uint32_t in = __reduce_min_sync(0xffffffffu, open ? logit_key(score - off) : 0xFFFFFFFFu);
            const uint32_t out = __reduce_max_sync(0xffffffffu, group < groups && !open ? logit_key(score + off) : 0u);
            if (in <= out) return false;
        }
    }
    const bool by_score = a.bias != nullptr;
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = open && i < mine ? logit_key(by_score ? c[i] : x[i]) : 0u;
    // ---- candidates: what is not below the topk-th largest of the lanes' largest, which is no larger than the topk-th of
    // all, or where those are fewer of all; by scores not below what may yet be before it.  To lane j the j-th of them by
    // key, then expert.
    auto value = [](uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); };
    uint32_t best = 0, least = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) best = max(best, key[i]);
    int seen = 0;
    for (; seen < topk;) {
        least = __reduce_max_sync(0xffffffffu, best);
        if (least == 0) break;
        seen += __popc(__ballot_sync(0xffffffffu, best == least));
        if (best == least) best = 0;
    }
    if (seen < topk) {
        // the largest left, topk times (8192 x 256, bias, the top 16 in 3 of 8 groups 20.3 us, by pairs of fp32 52.9), unless
        // all that are open will do
        int open_ones = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) open_ones += key[i] != 0 ? 1 : 0;
        const bool all_do = !by_score && __reduce_add_sync(0xffffffffu, open_ones) <= 32;
        uint32_t under = 0xFFFFFFFFu;  // what lanes have below it is not seen
        for (seen = all_do ? topk : 0; seen < topk;) {
            best = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) best = key[i] < under ? max(best, key[i]) : best;
            under = least = __reduce_max_sync(0xffffffffu, best);
            if (least == 0) break;
            seen += __popc(__ballot_sync(0xffffffffu, best == least));
        }
    }
    if (by_score) {
        if (least <= 1) return false;  // fewer that differ in their lanes than topk, or NaN
        const float v = value(least);
        least = logit_key(v - 4.0f * (slack + 0x1p-21f * fabsf(v)));
    }
    if (least == 0) least = 1;
    int some = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) some += key[i] >= least ? 1 : 0;
    int upto = some;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    const int n = __shfl_sync(0xffffffffu, upto, 31);
    if (n > 32) return false;
    sh.key[lane] = 0;
    __syncwarp();
    int to = upto - some;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (key[i] >= least) {
            sh.key[to] = key[i];
            sh.id[to++] = e0 + i;
        }
    __syncwarp();
    uint32_t got = sh.key[lane];
    int id = sh.id[lane], rank = 0;
    for (int k = 0; k < n; k += 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(sh.key + k);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) rank += u[q] > got || (u[q] == got && k + q < lane) ? 1 : 0;
    }
    __syncwarp();
    if (lane < n) {
        sh.key[rank] = got;
        sh.id[rank] = id;
    }
    __syncwarp();
    got = sh.key[lane];
    id = sh.id[lane];
    int place = lane < n ? lane : 32;
    bool close = false;
    if (by_score) {
        const float v = value(got), above = value(sh.key[lane > 0 ? lane - 1 : 0]);
        const bool apart = above - v > 2.0f * (slack + 0x1p-22f * (fabsf(above) + fabsf(v)));
        close = __any_sync(0xffffffffu, lane > 0 && lane <= topk && lane < n && !apart);
    }
    if (close) {
        // ---- scores that fp32 does not tell apart: those of the candidates again, and their places by them
        if (a.softmax) return false;  // would need the sum of all again
        uint64_t exact = 0;
        if (lane < n) {
            const float v = load_logit<F32>(row, id), d = -fabsf(v);
            const Two u = d > kNoScore ? two_exp2(times_log2e(Two{d, 0.0f})) : Two{0.0f, 0.0f}, one{1.0f, 0.0f};
            exact = score_key(div(v < 0.0f ? u : one, add(u, 1.0f)), bias_of(a.bias[id]));
        }
        place = 0;
        for (int j = 0; j < n; ++j) {
            const uint64_t other = __shfl_sync(0xffffffffu, exact, j);
            const int other_id = __shfl_sync(0xffffffffu, id, j);
            place += other > exact || (other == exact && other_id < id) ? 1 : 0;
        }
        if (lane >= n) place = 32;
    }
    // ---- the weights, from the chosen experts' logits
    float w = 0.0f;
    if (place < topk) {
        float v = value(got);
        if (by_score) v = load_logit<F32>(row, id);
        if (a.softmax) {
            w = v - m > kNoScore ? exp_near(v, m) / z : 0.0f;
        } else {
            const float e = fabsf(v) < -kNoScore ? exp_near(-fabsf(v), 0.0f) : 0.0f;
            w = (v < 0.0f ? e : 1.0f) / (1.0f + e);
        }
        if (v != v) w = v;
    }
    if (a.renormalize) {
        float sum = w;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        w = sum == 0.0f ? 0.0f : w / sum;
    }
    if (place < topk) {
        a.ids[token * topk + place] = id;
        a.weights[token * topk + place] = w * a.scale;
    }
    return true;
}

// CTAs an SM: 32 warps to 8 experts a lane (64 registers); 28 for 16 (8192 x 512, softmax top 10: 12.8 us, 16 warps
// 15.4), 16 for 32 (1024 experts: 24.7 us, 8 warps 36.7).
template <bool F32, int EPL>
__global__ void __launch_bounds__(kRouteWarps * 32, EPL <= 8 ? 8 : EPL == 16 ? 7 : 4)
    route_kernel(const __grid_constant__ MoeScoreArgs a) {
    extern __shared__ uint64_t sh_scores[];  // [warps][experts], with groups
    const int64_t token = static_cast<int64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
    __shared__ Candidates candidates[kRouteWarps];
    pdl_wait();
    if (token >= a.tokens) return;
    if (!route_quickly<F32, EPL>(a, token, candidates[threadIdx.x >> 5]))
        route_exactly<F32, EPL>(a, token, sh_scores + (threadIdx.x >> 5) * a.experts);
}

template <bool F32, int EPL>
cudaError_t launch_route_t(const MoeScoreArgs &a, cudaStream_t stream) {
    const int64_t blocks = (a.tokens + kRouteWarps - 1) / kRouteWarps;
    static_assert(kRouteWarps * kRouteMaxExperts * 8 <= 48 * 1024, "shared memory of a launch");
    const size_t smem = a.groups > 1 ? static_cast<size_t>(kRouteWarps * a.experts * 8) : 0;
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

// Experts a lane: what a group's lanes, or all, have to hold.  Where 32 a lane are not enough (a group has a power of
// two of the lanes: 1023 experts in 3 groups are 341 on 8 lanes) every token is left to pairs of fp32: 8192 tokens 244
// us, 32 tokens 47, against 58 and 7 for 1024 in 4 groups, the best 2 of them open.
template <bool F32>
cudaError_t launch_route_epl(const MoeScoreArgs &a, cudaStream_t stream) {
    int64_t lanes = 32;
    for (int64_t g = 1; g < a.groups; g *= 2) lanes /= 2;
    const int64_t all = (a.experts + 31) / 32, group = (a.experts / a.groups + lanes - 1) / lanes;
    const int64_t need = group > 32 || all > group ? all : group;
    if (need <= 1) return launch_route_t<F32, 1>(a, stream);
    if (need <= 2) return launch_route_t<F32, 2>(a, stream);
    if (need <= 4) return launch_route_t<F32, 4>(a, stream);
    if (need <= 8) return launch_route_t<F32, 8>(a, stream);
    if (need <= 16) return launch_route_t<F32, 16>(a, stream);
    return launch_route_t<F32, 32>(a, stream);
}

// --------------------------------------------------------------- combination
// A thread has 8 consecutive columns of a token, 16 bytes of each of its
// slots.  A warp's lanes load the token's ids and weights, a slot each, at
// once; kInFlight slots are loaded before the first is used.
//
// Floor: y, the residual and the result once.  2048 tokens of 12 x 4096 (235 MB):
// 36.2 us, 6.5 TB/s, 0.97 of a copy's rate; 512 of 8 x 7168 (73 MB, within L2) 13.4;
// 32 tokens 2.4.  DRAM bounds it.  Slots in flight, for these three: 2 38.7, 15.2, 3.1
// (CTAs of 256); 4 36.2, 13.4, 2.4; 6 35.8, 14.1, 2.2; 8 36.6, 13.0, 2.3: 6 and 8 each
// gain where they divide topk and lose elsewhere.  Threads a CTA: 64 36.2, 13.4, 2.7;
// 128 36.2, 13.4, 2.4; 256 36.8, 13.7, 2.9; 512 39.7, 15.5, 3.1.  With branches around
// the loads, which the compiler then waits for one by one, 51.
constexpr int kCombineThreads = 128;
constexpr int kInFlight = 4;

// The 8 columns from p on, of which `cols` are there, as bf16; no load unless `want`.  Without a branch, so that
// several are in flight.
template <bool VEC>
__device__ __forceinline__ uint4 load8(const __nv_bfloat16 *p, int cols, bool want) {
    if constexpr (VEC) {
        uint4 v;
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
            "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
            "@p ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];\n\t}"
            : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
            : "l"(p), "r"(want ? 1u : 0u));
        return v;
    } else {
        const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t lo = want && 2 * j < cols ? q[2 * j] : 0u, hi = want && 2 * j + 1 < cols ? q[2 * j + 1] : 0u;
            w[j] = lo | hi << 16;
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}
__device__ __forceinline__ void add8(const uint4 v, float w, float (&acc)[8]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        acc[2 * j] = fmaf(w, bf16lo_to_f32(u[j]), acc[2 * j]);
        acc[2 * j + 1] = fmaf(w, bf16hi_to_f32(u[j]), acc[2 * j + 1]);
    }
}

template <bool VEC>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const MoeCombineArgs a, uint32_t chunks) {
    const int lane = threadIdx.x & 31;
    const int64_t token = blockIdx.x / chunks;
    const int64_t col = 8 * (static_cast<int64_t>(blockIdx.x - token * chunks) * blockDim.x + threadIdx.x);
    pdl_wait();
    const int topk = static_cast<int>(a.topk), cols = static_cast<int>(a.n - col < 8 ? a.n - col : 8);
    const bool in = cols > 0;
    const __nv_bfloat16 *y = static_cast<const __nv_bfloat16 *>(a.y) + token * topk * a.n + col;
    const uint4 base = load8<VEC>(static_cast<const __nv_bfloat16 *>(a.residual) + token * a.n + col, cols, in && a.residual);
    float acc[8];
    for (int j0 = 0; j0 < topk; j0 += 32) {
        // lane j: slot j0 + j
        const bool there = j0 + lane < topk;
        const int id = there && a.ids ? a.ids[token * topk + j0 + lane] : 0;
        const float weight = there ? a.weights[token * topk + j0 + lane] : 0.0f;
        const uint32_t live = __ballot_sync(0xffffffffu, there && (!a.ids || (id >= 0 && id < a.experts)));
        const int slots = topk - j0 < 32 ? topk - j0 : 32;
        for (int j = 0; j < slots; j += kInFlight) {
            uint4 x[kInFlight];
#pragma unroll
            for (int i = 0; i < kInFlight; ++i)
                x[i] = load8<VEC>(y + (j0 + j + i) * a.n, cols, in && j + i < slots && ((live >> ((j + i) & 31)) & 1));
            if (j0 + j == 0) {
                const uint32_t u[4] = {base.x, base.y, base.z, base.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[2 * k] = bf16lo_to_f32(u[k]), acc[2 * k + 1] = bf16hi_to_f32(u[k]);
            }
#pragma unroll
            for (int i = 0; i < kInFlight; ++i) {
                const float w = __shfl_sync(0xffffffffu, weight, (j + i) & 31);
                if (j + i < slots && ((live >> ((j + i) & 31)) & 1)) add8(x[i], w, acc);  // the same for the whole warp
            }
        }
    }
    if (!in) return;
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
    // a CTA has one token's columns: as few warps as hold a short row
    const int64_t per_row = (a.n + 7) / 8;
    const int64_t threads = per_row >= kCombineThreads ? kCombineThreads : (per_row + 31) / 32 * 32;
    const int64_t chunks = (per_row + threads - 1) / threads, blocks = a.tokens * chunks;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    const bool vec = a.n % 8 == 0 && aligned16(a.y) && aligned16(a.residual) && aligned16(a.out);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return vec ? cudaLaunchKernelEx(&cfg, combine_kernel<true>, a, static_cast<uint32_t>(chunks))
               : cudaLaunchKernelEx(&cfg, combine_kernel<false>, a, static_cast<uint32_t>(chunks));
}

}  // namespace fp8bs
