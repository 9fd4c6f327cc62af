// sample.cu -- the next token of each row of logits, drawn with given random
// numbers from what temperature, top-k, top-p and min-p leave.
//
// With m the row's largest logit, w_j = 2^(c (x_j - m)), c = log2(e) / T.  Kept
// are the first tokens of the order by value, then index: as many as top-k, top-p
// (of the top-k's mass) and min-p all allow, which is a cut, a value and how many
// of its equals.  The first random number picks a block of 1024 tokens by the
// kept mass, the second a token of the block.
//
// Whole numbers come out, so masses are whole numbers too, in units of 2^-41 of
// the largest weight: their sums and comparisons are exact and do not depend on
// an order.  What rounds is a weight (ex2's 2^-22, with the exponent's own error
// taken back out, so that the errors of different values do not add up) and a
// lane's fp32 sum of 32; the drawn block's weights are pairs of fp32 (2^-44).
//
// The CTAs of a cluster (one CTA when there are many rows) have consecutive
// blocks of a row each, a warp a block at a time.  One pass over the row gives the
// largest logit and every block's mass.  A cut takes two more: a histogram over
// the exponents of the weights, 32 bins to a factor of 2, whose masses are each
// bin's count times its weight plus what its tokens differ from that; and, for the
// bin that holds the cut, the tokens above it summed by block and its own tokens
// gathered in shared memory, where histograms over their values end the search.
// A bin that holds too many is first cut by histograms over its values.
//
// Floor: the logits once.  512 rows of 152064 (bf16, 156 MB) by temperature 38.6 us,
// 4.0 TB/s; by top-p 163, by top-k 103; 64 rows of mixed settings 37; 256 fp32 rows
// of 32003 44.1; one row by top-p 21.8, by temperature 8.4.  The passes are bound by the
// instructions they issue, 512 rows also by their count on 152 SMs (400 rows 33 us, 600
// 40.1); what lies between the passes by the latency of steps that a whole CTA or
// cluster takes together, about 0.7 us for each exchange in a cluster.
#include "twofloat.cuh"
#include "samplebins.cuh"

#include "serving.cuh"
#include "internal.h"

#include <cstddef>
#include <cstring>
#include <mutex>

namespace fp8bs {

namespace {

__device__ uint32_t g_sample_err;

constexpr int kBlock = 1024;                    // tokens of a block
constexpr int kMaxBlocks = kSampleMaxVocab / kBlock;
constexpr int kMaxSplit = 8;                    // CTAs a row
constexpr int kFine = 512;                      // of the values in a range
constexpr int kGather = 2048;                   // tokens that the last histograms can take
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMagic = 12582912.0f;           // 1.5 * 2^23: adding it rounds to whole numbers
constexpr uint32_t kMagicBits = 0x4B400000u;
constexpr float kUnit = 0x1p41f;                // of masses

// 2^(62 - j / 32): a bin's weight
__constant__ uint64_t kBinWeight[32] = {
    0x4000000000000000ull, 0x3EA0ECB6DC8A80CFull, 0x3D495F454921B30Bull, 0x3BF92E66F736BD73ull,
    0x3AB031B9F7490E4Cull, 0x396E41B9DF20D22Aull, 0x383337BB0AA53844ull, 0x36FEEDE5F6BC8DD5ull,
    0x35D13F32B5A75ABDull, 0x34AA07647C4AB917ull, 0x3389230547E12039ull, 0x326E6F619B8BC9E9ull,
    0x3159CA845541B6B7ull, 0x304B1332999C2516ull, 0x2F4228E7D6030DB0ull, 0x2E3EEBD1D8BEE7BAull,
    0x2D413CCCFE779921ull, 0x2C48FD6074AB0964ull, 0x2B560FBA90A852B2ull, 0x2A6856AD3A9F03BEull,
    0x297FB5AA6C544E3Bull, 0x289C10C0C3125A06ull, 0x27BD4C982468446Bull, 0x26E34E6E7553954Eull,
    0x260DFC14636E2A5Cull, 0x253D3BEA3FBDC258ull, 0x2470F4DCEAC470CEull, 0x23A90E62D17354F0ull,
    0x22E57078FAA2F5BAull, 0x222603A024B6A14Aull, 0x216AB0D9F3121EC5ull, 0x20B361A62B0AE876ull,
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Order of the values as unsigned integers, of 16 bits for bf16: -0 is +0, NaN
// above everything.
template <bool F32>
struct Key {
    static constexpr uint32_t kInf = F32 ? 0xFF800000u : 0xFF80u, kNegInf = F32 ? 0x007FFFFFu : 0x007Fu;
    static constexpr uint32_t kNegZero = F32 ? 0x7FFFFFFFu : 0x7FFFu;  // no value's
    static __device__ __forceinline__ uint32_t of(float x) {
        const uint32_t u = __float_as_uint(x + 0.0f);
        const uint32_t k = x != x ? 0xFFFFFFFFu : u & 0x80000000u ? ~u : u | 0x80000000u;
        return F32 ? k : k >> 16;
    }
    static __device__ __forceinline__ float value(uint32_t k) {
        if (!F32) k = k & 0x8000u ? k << 16 : k << 16 | 0xFFFFu;
        return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
    }
    // Of the least value that is not below x, a finite fp32.
    static __device__ __forceinline__ uint32_t from(float x) {
        const uint32_t u = __float_as_uint(x + 0.0f);
        if (F32) return of(x);
        const uint32_t k = u & 0x80000000u ? ~u >> 16 : ((u | 0x80000000u) + 0xFFFFu) >> 16;
        return k == kNegZero ? k + 1 : k;
    }
};

template <class T>
__device__ __forceinline__ T warp_inclusive(T v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// 0xFFFF in the halves where a's number is at least b's.
__device__ __forceinline__ uint32_t at_least_bf16x2(uint32_t a, uint32_t b) {
    __nv_bfloat162 x, y;
    memcpy(&x, &a, 4);
    memcpy(&y, &b, 4);
    return __hge2_mask(x, y);
}
// v's two numbers and c, each sum one fp32 rounding.
__device__ __forceinline__ void add_bf16x2(uint32_t v, float c, float &lo, float &hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "add.rn.f32.bf16 %0, l, %3;\n\tadd.rn.f32.bf16 %1, h, %3;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(v), "f"(c));
}
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Elements e0 .. of a row, 16 bytes of them, -inf past it: what the ends of a row that is off a boundary need.  One copy
// of its code, which every pass would have for each of a lane's vectors.
template <bool F32>
__device__ __noinline__ uint4 one_by_one(const char *base, int vocab, int e0) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (F32) {
            w[j] = e0 + j < vocab ? reinterpret_cast<const uint32_t *>(base)[e0 + j] : 0xFF800000u;
        } else {
            const uint16_t *p = reinterpret_cast<const uint16_t *>(base);
            const uint32_t lo = e0 + 2 * j < vocab ? p[e0 + 2 * j] : 0xFF80u;
            const uint32_t hi = e0 + 2 * j + 1 < vocab ? p[e0 + 2 * j + 1] : 0xFF80u;
            w[j] = lo | hi << 16;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A row of logits by blocks: lane l of the warp that has block b holds NV vectors
// of VE elements, of element b * 1024 + (l + 32 i) * VE on, or turned; -inf past the
// row.  Turned rows read as many vectors as others: 2048 bf16 rows of 32003 by
// temperature 50.7 us, 57.8 with each vector put together from two; 256 fp32 rows of
// 32003 with cuts 44.4 and 48.8.  With the next block's loads ahead in registers (bf16)
// the first took 54.0, 512 rows of 152064 42.6 and not 39.2, 64 of them 11.6 and not 12.1.
template <bool F32>
struct Row {
    static constexpr int VE = F32 ? 4 : 8, NV = kBlock / (32 * VE), ES = F32 ? 4 : 2;
    const char *base;
    int vocab, off;  // off: bytes that the row is past a 16-byte boundary

    __device__ __forceinline__ Row(const void *p, int v)
        : base(static_cast<const char *>(p)), vocab(v), off(static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15)) {}
    __device__ __forceinline__ float at(int e) const {
        if constexpr (F32) return reinterpret_cast<const float *>(base)[e];
        else return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(base)[e]);
    }
    // Elements by which a lane's vectors of block b are turned: where the row is off a boundary they are taken as they
    // lie in memory, and the first one's elements before the block are those after its last vector instead.
    __device__ __forceinline__ int turn(int b) const {
        return off != 0 && b > 0 && (b + 1) * kBlock + VE <= vocab ? off / ES : 0;
    }
    __device__ __forceinline__ void load(int b, uint4 (&w)[NV]) const {
        const int first = b * kBlock + (threadIdx.x & 31) * VE;
        if (off == 0 && (b + 1) * kBlock <= vocab) {  // a whole block: the most
            const char *p = base + static_cast<int64_t>(first) * ES;
#pragma unroll
            for (int i = 0; i < NV; ++i) w[i] = ld_v4(p + i * 512);
            return;
        }
        if (turn(b) != 0) {
            const char *p = base + static_cast<int64_t>(first) * ES - off;
#pragma unroll
            for (int i = 0; i < NV; ++i) w[i] = ld_v4(p + i * 512);
            const uint4 e = ld_v4(base + static_cast<int64_t>(b + 1) * kBlock * ES - off);
            const int from = (threadIdx.x & 31) == 0 ? off : 0;  // bytes that are those of e
            auto join = [&](uint32_t mine, uint32_t behind, int at) {
                const uint32_t mask = (from > at ? 0xFFFFu : 0u) | (from > at + 2 ? 0xFFFF0000u : 0u);
                return (behind & mask) | (mine & ~mask);
            };
            w[0] = make_uint4(join(w[0].x, e.x, 0), join(w[0].y, e.y, 4), join(w[0].z, e.z, 8), join(w[0].w, e.w, 12));
            return;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e0 = first + i * 32 * VE;
            const char *p = base + static_cast<int64_t>(e0) * ES;
            if (e0 >= vocab) w[i] = F32 ? make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u)
                                        : make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
            else if (off == 0 && e0 + VE <= vocab) w[i] = ld_v4(p);
            else w[i] = one_by_one<F32>(base, vocab, e0);
        }
    }
    static __device__ __forceinline__ void unpack(const uint4 v, float (&x)[VE]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (F32) {
                x[j] = __uint_as_float(w[j]);
            } else {
                x[2 * j] = bf16lo_to_f32(w[j]);
                x[2 * j + 1] = bf16hi_to_f32(w[j]);
            }
        }
    }
    // The largest of a vector's elements, none of which is NaN.
    static __device__ __forceinline__ float largest(const uint4 v) {
        if constexpr (F32) {
            return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
        } else {
            const uint32_t m = max_bf16x2(max_bf16x2(v.x, v.y), max_bf16x2(v.z, v.w));
            return fmaxf(bf16lo_to_f32(m), bf16hi_to_f32(m));
        }
    }
    static __device__ __forceinline__ float smallest(const uint4 v) {
        if constexpr (F32) {
            return fminf(fminf(__uint_as_float(v.x), __uint_as_float(v.y)), fminf(__uint_as_float(v.z), __uint_as_float(v.w)));
        } else {
            const uint32_t m = min_bf16x2(min_bf16x2(v.x, v.y), min_bf16x2(v.z, v.w));
            return fminf(bf16lo_to_f32(m), bf16hi_to_f32(m));
        }
    }
    // Which of a lane's elements, none of which is NaN, are in [lo, hi], a bit each; and the element of a bit.
    static __device__ __forceinline__ uint32_t between(const uint4 (&w)[NV], float lo, float hi) {
        uint32_t in = 0;
        const uint32_t l = __float_as_uint(lo) >> 16, h = __float_as_uint(hi) >> 16, low = l << 16 | l, high = h << 16 | h;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (F32) {
                    const float x = __uint_as_float(u[j]);
                    in |= x >= lo && x <= hi ? 1u << (4 * i + j) : 0u;
                } else {
                    in |= at_least_bf16x2(u[j], low) & at_least_bf16x2(high, u[j]) & (0x10001u << (4 * i + j));
                }
            }
        }
        return in;
    }
    static __device__ __forceinline__ int element(int bit) { return F32 ? bit : 2 * (bit & 15) + (bit >> 4); }
    // The largest of a lane's elements; NaN if there is one.
    static __device__ __forceinline__ float most(const uint4 (&w)[NV]) {
        if constexpr (F32) {
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                m = max_nan(m, max_nan(max_nan(__uint_as_float(w[i].x), __uint_as_float(w[i].y)),
                                       max_nan(__uint_as_float(w[i].z), __uint_as_float(w[i].w))));
            return m;
        } else {
            uint32_t m = w[0].x;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                m = max_nan_bf16x2(max_nan_bf16x2(m, w[i].x), max_nan_bf16x2(max_nan_bf16x2(w[i].y, w[i].z), w[i].w));
            return max_nan(bf16lo_to_f32(m), bf16hi_to_f32(m));
        }
    }
};

// The values of keys lo .. hi, where the cut lies: `equals` tokens, under `count`
// of them with `mass` above.
struct Range {
    uint32_t lo, hi;
    int count, equals;
    uint64_t mass;
    int none;      // not 0: there is no cut
    int pad;
};

template <int TH>
struct Shared {
    static constexpr int kWarps = TH / 32;
    uint64_t block_mass[kMaxBlocks];  // the first CTA has all blocks' in the end
    uint32_t block_key[kMaxBlocks];   // of the block's largest logit
    int block_equals[kMaxBlocks];     // tokens at the cut's value
    Range range, inbox[2];
    uint64_t warp_sum[kWarps], part_mass[kMaxSplit], part_in[kMaxSplit];
    double log_min_p;
    int warp_int[kWarps];
    uint64_t went_in[kWarps];         // of count_exponents, which no barrier parts from the sums before it
    uint32_t warp_key[kWarps], part_key[kMaxSplit], part_bound[kMaxSplit], bound, min_key;
    uint64_t bin_weight[32];          // kBinWeight: lanes ask for different ones
    int listed, collected, last, block, allowed;
    uint64_t beside;                  // the mass outside the drawn block
    // from here on for the search of a cut only
    alignas(16) uint32_t n[kBins], q[kBins];  // tokens of a bin, and what they weigh beside its weight
    union {
        struct {
            uint32_t fine_n[kFine], fine_q[kFine];
        };
        uint64_t list_weight[kFine];  // of a short list's tokens
    };
    uint32_t list_key[kGather], list_id[kGather];
};

// To the shared memory of CTA `rank` of the cluster, at the place of *local.
template <class T>
__device__ __forceinline__ void dsmem_put(T *local, int rank, const T &v) {
    static_assert(sizeof(T) % 4 == 0, "words");
    const uint32_t to = dsmem_map(smem_u32(local), rank);
    const float *w = reinterpret_cast<const float *>(&v);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 4); ++i) dsmem_st_f32(to + 4 * i, w[i]);
}
__device__ __forceinline__ void dsmem_add(uint32_t *local, int rank, uint32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(dsmem_map(smem_u32(local), rank)), "r"(v)
                 : "memory");
}
__device__ __forceinline__ uint32_t dsmem_next(int *local, int rank, uint32_t n) {
    uint32_t r;
    asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;"
                 : "=r"(r)
                 : "r"(dsmem_map(smem_u32(local), rank)), "r"(n)
                 : "memory");
    return r;
}

// The sum of the values of the threads before this one, and of all.  It ends with every thread reading `warps`, and no
// barrier after that: whoever writes one of the arrays that are given here, warp_int and warp_sum, has a barrier before.
template <class T, int TH>
__device__ __forceinline__ T cta_exclusive(T v, T *warps, T &all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T upto = warp_inclusive(v);
    __syncthreads();
    if (lane == 31) warps[warp] = upto;
    __syncthreads();
    T before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < TH / 32; ++w) {
        if (w == warp) before = sum;
        sum += warps[w];
    }
    all = sum;
    return before + upto - v;
}
// The same of a count and a mass at once: n and v become the sums before.
template <int TH>
__device__ __forceinline__ void cta_exclusive2(int &n, uint64_t &v, int *warps_n, uint64_t *warps_v, uint64_t &all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int upto_n = warp_inclusive(n);
    const uint64_t upto = warp_inclusive(v);
    __syncthreads();
    if (lane == 31) warps_n[warp] = upto_n, warps_v[warp] = upto;
    __syncthreads();
    int before_n = 0, sum_n = 0;
    uint64_t before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < TH / 32; ++w) {
        if (w == warp) before_n = sum_n, before = sum;
        sum_n += warps_n[w];
        sum += warps_v[w];
    }
    all = sum;
    n = before_n + upto_n - n;
    v = before + upto - v;
}

// 2^(c (x - m)).  One copy of its code: what runs once waits for its instructions.
__device__ __noinline__ Two weight(float x, float m, Two c) {
    if (!(x > -INFINITY)) return Two{0.0f, 0.0f};
    const Two d = two_sum(x, -m);
    const float t = d.h * c.h;
    return t > -125.0f ? two_exp2(mul(d, c)) : Two{0.0f, 0.0f};
}
// v * unit to the nearest whole number.
__device__ __forceinline__ uint64_t fixed(Two v, float unit) {
    const float h = v.h * unit, l = v.l * unit;
    return h < 0x1p23f ? __float2ull_rn(h + l) : __float2ull_rn(h) + static_cast<uint64_t>(__float2ll_rn(l));
}
__device__ __forceinline__ uint64_t at_least_one(uint64_t v) { return v > 0 ? v : 1; }
// floor(share * mass), for a share in [0, 1].
__device__ __forceinline__ uint64_t part_of(uint64_t mass, float share) {
    return share >= 1.0f ? mass : __umul64hi(mass, __float2ull_rz(share * 0x1p64f));
}

// A lane's sum of 2^(c (x - m)), m the block's largest, of its elements with x
// above `least`.  t = d c.h rounds; what it lost and d c.l, e together, come
// back as the factor 1 + e ln 2, its second part summed apart.
template <bool F32, bool ALL>
__device__ __forceinline__ float block_sum(const uint4 (&w)[Row<F32>::NV], uint32_t m_key, Two c, float reach, float least) {
    const float m = Key<F32>::value(m_key);
    if (!(fabsf(m) < 1e37f && fabsf(m) * c.h < 1e30f)) {  // d c may not fit fp32
        constexpr int VE = Row<F32>::VE;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < Row<F32>::NV; ++i) {
            float x[VE];
            Row<F32>::unpack(w[i], x);
            for (int j = 0; j < VE; ++j)
                if (ALL || x[j] > least) sum += ex2(fmaxf(x[j] - m, -reach) * c.h);
        }
        return sum;
    }
    // below this a weight is none, but d c still a number; less than m itself
    float floor = fminf(m - reach, Key<F32>::value(m_key - 1));
    const uint32_t fb = __float_as_uint(floor);
    const uint32_t low = fb & 0x80000000u ? (fb + 0xFFFFu) >> 16 : fb >> 16;  // the next bf16 down
    const uint64_t neg_m = pair(-m, -m), ch = pair(c.h, c.h), neg_ch = pair(-c.h, -c.h), neg_cl = pair(-c.l, -c.l);
    uint64_t sum = 0, missing = 0;
#pragma unroll
    for (int i = 0; i < Row<F32>::NV; ++i) {
        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int j = 0; j < (F32 ? 2 : 4); ++j) {
            float x0, x1, d0 = 0.0f, d1 = 0.0f;
            if constexpr (F32) {
                x0 = fmaxf(__uint_as_float(u[2 * j]), floor), x1 = fmaxf(__uint_as_float(u[2 * j + 1]), floor);
            } else {
                const uint32_t v = max_bf16x2(u[j], low | low << 16);
                x0 = bf16lo_to_f32(v), x1 = bf16hi_to_f32(v);
                add_bf16x2(v, -m, d0, d1);
            }
            const uint64_t d = F32 ? add2(pair(x0, x1), neg_m) : pair(d0, d1), t = mul2(d, ch);
            const uint64_t e = fma2(d, neg_cl, fma2(d, neg_ch, t));  // minus what is missing
            float t0, t1;
            unpair(t, t0, t1);
            float w0 = ex2(t0), w1 = ex2(t1);
            if constexpr (!ALL) {
                w0 = x0 > least ? w0 : 0.0f;
                w1 = x1 > least ? w1 : 0.0f;
            }
            const uint64_t v = pair(w0, w1);
            sum = add2(sum, v);
            missing = fma2(v, e, missing);
        }
    }
    float a, b, p, q;
    unpair(sum, a, b);
    unpair(missing, p, q);
    return fmaf(p + q, -kLn2, a + b);
}

struct Job {
    float m;       // the row's largest logit
    uint32_t m_key, lowest;  // no token below `lowest` is kept
    Two c;
    float reach;   // 124 / c: a weight that far below another is none beside it
    int b0, b1, blocks, part, splits;
    int bits;      // of a residual in a histogram of the row
    int turn;      // of share_range's boxes
};

// The n-th token, or the first whose mass to it reaches `mass`.
struct Target {
    bool by_mass;
    int count;
    uint64_t mass;
    __device__ __forceinline__ bool reached(int n, uint64_t v) const { return by_mass ? v >= mass : n >= count; }
};

// Among the bins of the threads in order, PER each (n tokens of mass v), the one
// that reaches the target, or with MUST the last that holds a token: tell(bin of
// the thread, tokens before, mass before) by the one thread that has it.  Returns
// whether there is one.
template <bool MUST, int PER, int TH, class Tell>
__device__ __forceinline__ bool find_bin(const int (&n)[PER], const uint64_t (&v)[PER], int at_n, uint64_t at,
                                         const Target &target, Shared<TH> &sh, Tell tell) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int hit = -1, last = -1, last_n = 0;
    uint64_t last_at = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (hit < 0 && n[i] > 0) {
            if (target.reached(at_n + n[i], at + v[i])) {
                hit = i;
            } else {
                if (MUST) last = i, last_n = at_n, last_at = at;
                at_n += n[i], at += v[i];
            }
        }
    }
    const uint32_t have = __ballot_sync(0xffffffffu, hit >= 0);
    const uint32_t any = MUST ? __ballot_sync(0xffffffffu, last >= 0) : 0;
    __syncthreads();
    if (lane == 0) {
        sh.warp_int[warp] = have ? __ffs(have) - 1 : -1;
        sh.warp_key[warp] = any ? 31 - __clz(any) : 0xFFFFFFFFu;
    }
    __syncthreads();
    int who = -1;
#pragma unroll
    for (int i = TH / 32 - 1; i >= 0; --i) who = sh.warp_int[i] >= 0 ? i * 32 + sh.warp_int[i] : who;
    if (MUST && who < 0) {
        for (int i = 0; i < TH / 32; ++i) who = sh.warp_key[i] != 0xFFFFFFFFu ? i * 32 + static_cast<int>(sh.warp_key[i]) : who;
        hit = last, at_n = last_n, at = last_at;
    }
    if (static_cast<int>(threadIdx.x) == who) tell(hit, at_n, at);
    __syncthreads();
    return who >= 0;
}

// What a token of a range of values whose weights are within 2^-5 of the range's
// largest weighs less than that, in units of 2^-25.
__device__ __forceinline__ uint32_t fine_rest(float top, float x, Two c, float scale) {
    const float d = top - x, f = fmaf(d, c.l, d * c.h) * kLn2;
    return static_cast<uint32_t>(__float2int_rn(f * fmaf(f, fmaf(f, 1.0f / 6.0f, -0.5f), 1.0f) * scale));
}

// No number is -0's: ranges leave its key out, so that their ends compare as floats do.
template <bool F32>
__device__ __forceinline__ Range tidy(Range r) {
    if (r.hi == Key<F32>::kNegZero) --r.hi;
    if (r.lo == Key<F32>::kNegZero) ++r.lo;
    return r;
}

// From the histogram fine_n, fine_q of sh.range's values: the bin with the target
// becomes sh.range.  By the first CTA.
template <bool F32, int TH>
__device__ void narrow(const Job &job, Shared<TH> &sh, const Target &target, int shift, int bits) {
    constexpr int kPer = kFine / TH > 0 ? kFine / TH : 1;
    const Range r = sh.range;
    const uint64_t w = fixed(weight(Key<F32>::value(r.hi), job.m, job.c), 0x1p62f);
    int n[kPer], sum_n = 0;
    uint64_t v[kPer], sum = 0, all;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int bin = threadIdx.x * kPer + i;
        n[i] = bin < kFine ? static_cast<int>(sh.fine_n[bin]) : 0;
        // (n - q 2^-(5 + bits)) w
        v[i] = n[i] ? __umul64hi(((static_cast<uint64_t>(n[i]) << (5 + bits)) - sh.fine_q[bin]) << (38 - bits), w) : 0;
        sum_n += n[i], sum += v[i];
    }
    cta_exclusive2<TH>(sum_n, sum, sh.warp_int, sh.warp_sum, all);
    const int at_n = r.count + sum_n;
    const uint64_t at = r.mass + sum;
    // the bins' masses can miss by their units what their sum was one histogram before: the last bin has the cut then
    const bool found = find_bin<true, kPer, TH>(n, v, at_n, at, target, sh, [&](int i, int before_n, uint64_t before) {
        const uint32_t hi = r.hi - (static_cast<uint32_t>(threadIdx.x * kPer + i) << shift);
        const uint32_t lo = hi - r.lo < (1u << shift) ? r.lo : hi - (1u << shift) + 1;
        sh.range = tidy<F32>(Range{lo, hi, before_n, n[i], before, 0, 0});
    });
    if (!found) {  // a range holds a token; were it not so, this ends the search
        if (threadIdx.x == 0) sh.range.lo = sh.range.hi;
        __syncthreads();
    }
}

// What the first CTA has found to all of the row's.  The boxes take turns: the
// one that is written has been read before the last barrier.
template <int TH>
__device__ __forceinline__ void share_range(Job &job, Shared<TH> &sh) {
    __syncthreads();
    if (job.splits > 1) {
        Range *box = &sh.inbox[job.turn];
        job.turn ^= 1;
        if (job.part == 0 && threadIdx.x > 0 && static_cast<int>(threadIdx.x) < job.splits)
            dsmem_put(box, threadIdx.x, sh.range);
        cluster_sync_all();
        if (job.part != 0 && threadIdx.x == 0) sh.range = *box;
    }
    __syncthreads();
}

__device__ __forceinline__ int fine_shift(uint32_t lo, uint32_t hi) {
    const uint32_t over = (hi - lo) / kFine;  // bins of 1 << shift values: ((hi - lo) >> shift) < kFine
    return over ? 32 - __clz(over) : 0;
}

// A CTA's histogram into the first one's.
template <int TH>
__device__ __forceinline__ void collect(const Job &job, uint32_t *n, uint32_t *q, int bins) {
    if (job.splits > 1) {
        cluster_sync_all();
        if (job.part != 0)
            for (int i = threadIdx.x; i < bins; i += TH)
                if (n[i]) {
                    dsmem_add(n + i, 0, n[i]);
                    dsmem_add(q + i, 0, q[i]);
                }
        cluster_sync_all();
    }
}

// What a row's histogram has to tell.  Two atomics a token where both are wanted;
// for masses alone one does, a token's weight beside its bin's in units of 2^-20.
// 4000 tokens of a bin fit 32 bits so, and if more wrap (rows of equals, far
// temperatures) the bins do not add up to what went in: then both are counted.
enum Counting : int { kCounts = 1, kMasses = 2, kBoth = 3 };
constexpr int kMassBits = 20;

template <int MODE>
__device__ __forceinline__ void count_one(uint32_t at, uint32_t q) {
    if constexpr (MODE == kCounts) {
        asm volatile("red.shared.add.u32 [%0], 1;" ::"r"(at));
    } else if constexpr (MODE == kMasses) {
        asm volatile("red.shared.add.u32 [%0 + %2], %1;" ::"r"(at), "r"(q), "n"(kBins * 4));
    } else {
        asm volatile("red.shared.add.u32 [%0], 1;\n\tred.shared.add.u32 [%0 + %2], %1;" ::"r"(at), "r"(q), "n"(kBins * 4));
    }
}

// The histogram of the row's exponents, in the first CTA's n and q; they are
// zero in all CTAs before a cluster barrier before this.
template <bool F32, int TH, int MODE>
__device__ void count_exponents(const Row<F32> &row, const Job &job, Shared<TH> &sh) {
    constexpr int NV = Row<F32>::NV, VE = Row<F32>::VE;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float least = Key<F32>::value(job.lowest), m = job.m;
    // d = x - m; bin = round(-32 c d), f the rest in [-1/2, 1/2]; weight / bin's = 2^(-f / 32), with the counts less 63/64
    // and in units of 2^-(5 + bits): below 2^bits.  The low bits of r are the bin, those of q the units
    const float unit = static_cast<float>(1 << (MODE == kMasses ? kMassBits : 5 + job.bits)), y = kLn2 / kPerUnit;
    const float whole = (MODE == kMasses ? unit : unit / 64.0f) + 0x1p23f;
    const uint64_t neg_m = pair(-m, -m), minus = pair(-1.0f, -1.0f), magic = pair(kMagic, kMagic);
    const float chf = -job.c.h * kPerUnit, clf = -job.c.l * kPerUnit;
    const uint64_t ch = pair(chf, chf), cl = pair(clf, clf);
    const uint64_t q0 = pair(whole, whole), q1 = pair(-unit * y, -unit * y);
    const uint64_t q2 = pair(unit * y * y / 2.0f, unit * y * y / 2.0f);
    const uint32_t base = smem_u32(sh.n) - (kMagicBits << 2);
    uint64_t went_in = 0;
    for (int b = job.b0 + warp; b < job.b1; b += TH / 32) {
        if (sh.block_key[b] < job.lowest) continue;
        uint4 w[NV];
        row.load(b, w);
        uint32_t sum = 0;  // 32 tokens of 2^20 and a hundredth more
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (Row<F32>::largest(w[i]) < least) continue;
            float x[VE];
            uint32_t at[VE], v[VE];
            Row<F32>::unpack(w[i], x);
            const uint32_t words[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int j = 0; j < VE; j += 2) {
                float d0 = 0.0f, d1 = 0.0f;
                if constexpr (!F32) add_bf16x2(words[j / 2], -m, d0, d1);
                const uint64_t d = F32 ? add2(pair(x[j], x[j + 1]), neg_m) : pair(d0, d1), r = fma2(d, ch, magic);
                float r0, r1, u0 = 0.0f, u1 = 0.0f;
                unpair(r, r0, r1);
                if constexpr (MODE != kCounts) {
                    // -32 c d - n, of which the product's part is exact but for one rounding; the third power of
                    // f ln 2 / 32 is at most 2^-22, as often up as down
                    const uint64_t f = fma2(d, cl, fma2(d, ch, fma2(r, minus, magic)));
                    unpair(fma2(f, fma2(f, q2, q1), q0), u0, u1);
                }
                at[j] = base + (__float_as_uint(r0) << 2), at[j + 1] = base + (__float_as_uint(r1) << 2);
                v[j] = __float_as_uint(u0) & 0x7FFFFFu, v[j + 1] = __float_as_uint(u1) & 0x7FFFFFu;
            }
            if (MODE == kMasses && Row<F32>::smallest(w[i]) >= least) {
#pragma unroll
                for (int j = 0; j < VE; ++j) {
                    count_one<MODE>(at[j], v[j]);
                    sum += v[j];
                }
            } else {
#pragma unroll
                for (int j = 0; j < VE; ++j)
                    if (x[j] >= least) {
                        count_one<MODE>(at[j], v[j]);
                        sum += v[j];
                    }
            }
        }
        went_in += sum;
    }
    if constexpr (MODE == kMasses) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) went_in += __shfl_xor_sync(0xffffffffu, went_in, o);
        if (lane == 0) sh.went_in[warp] = went_in;
    }
    __syncthreads();
    if constexpr (MODE == kMasses) {
        if (tid == 0) {
            went_in = 0;
            for (int i = 0; i < TH / 32; ++i) went_in += sh.went_in[i];
            if (job.splits > 1) dsmem_put(&sh.part_in[job.part], 0, went_in);
            else sh.part_in[0] = went_in;
        }
    }
    if (job.splits > 1) {
        if (job.part != 0)
            for (int i = tid; i < kBins; i += TH) {
                if (MODE != kMasses && sh.n[i]) dsmem_add(&sh.n[i], 0, sh.n[i]);
                if (MODE != kCounts && sh.q[i]) dsmem_add(&sh.q[i], 0, sh.q[i]);
            }
        cluster_sync_all();
    }
}

// The range of values of the exponents' bin that holds the target: sh.range, the
// same in all the row's CTAs; `none` is 1 if all the bins together do not reach
// it, 2 if masses alone did not fit their bins.
template <bool F32, int TH>
__device__ void find_exponent(Job &job, Shared<TH> &sh, const Target &target, int mode) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (job.part == 0) {
        constexpr int kPer = kBins / TH;
        int n[kPer], sum_n = 0;
        uint64_t v[kPer], sum = 0, all, in_bins = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int bin = tid * kPer + i;
            const uint32_t q = sh.q[bin];
            const uint64_t w = sh.bin_weight[bin & 31] >> (bin >> 5);
            if (mode == kMasses) {
                n[i] = static_cast<int>(q / ((1u << kMassBits) * 63 / 64)) + (q > 0 ? 1 : 0);  // no fewer than there are
                v[i] = __umul64hi(static_cast<uint64_t>(q) << (43 - kMassBits), w);
                in_bins += q;
            } else {
                n[i] = static_cast<int>(sh.n[bin]);
                const uint64_t units = static_cast<uint64_t>(n[i]) * (63u << (job.bits - 1)) + q;
                v[i] = n[i] && mode == kBoth ? __umul64hi(units << (38 - job.bits), w) : 0;
            }
            sum_n += n[i], sum += v[i];
        }
        cta_exclusive2<TH>(sum_n, sum, sh.warp_int, sh.warp_sum, all);
        const int at_n = sum_n;
        const uint64_t at = sum;
        bool wrapped = false;
        if (mode == kMasses) {
            // each thread's part of what is in the bins fits 35 bits, and their sum is off by a multiple of 2^32 or not at all
            uint64_t went_in = 0;
            for (int i = 0; i < job.splits; ++i) went_in += sh.part_in[i];
            const uint32_t low = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(in_bins & 0xFFFFu));
            const uint32_t high = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(in_bins >> 16));
            __syncthreads();
            if (lane == 0) sh.warp_sum[warp] = (static_cast<uint64_t>(high) << 16) + low;
            __syncthreads();
            for (int i = 0; i < TH / 32; ++i) went_in -= sh.warp_sum[i];
            wrapped = went_in != 0;
        }
        bool found = false;
        if (!wrapped)
            found = find_bin<false, kPer, TH>(n, v, at_n, at, target, sh, [&](int i, int before_n, uint64_t before) {
                sh.range = Range{static_cast<uint32_t>(tid * kPer + i), 0, before_n, n[i], before, 0, 0};
            });
        if (found) {
            // the bin's least value (warp 0) and the next bin's above it (warp 1): the bins' numbers fall as values rise
            const float ch = job.c.h * kPerUnit;
            const int bin = static_cast<int>(sh.range.lo);
            if (warp < 2) {
                const int want = bin - warp;
                auto reached = [&](int64_t key) {
                    const float r = fmaf(job.m - Key<F32>::value(static_cast<uint32_t>(key)), ch, kMagic);
                    return static_cast<int>(__float_as_uint(r) - kMagicBits) <= want;
                };
                int64_t from = static_cast<int64_t>(job.lowest) - 1, to = static_cast<int64_t>(job.m_key) + 1;  // in (from, to]
                {
                    // most often it is near where the numbers say
                    const int64_t guess = Key<F32>::of(job.m - (want + 0.5f) / ch);
                    const int64_t probe = guess - 16 + lane;
                    const bool yes = probe >= to || (probe > from && reached(probe));
                    const uint32_t votes = __ballot_sync(0xffffffffu, yes);
                    if (votes & 1u) to = min(to, max(guess - 16, from + 1));
                    else if (votes) to = min(to, guess - 16 + (__ffs(votes) - 1)), from = max(from, to - 1);
                    else from = max(from, guess + 15);
                }
                while (to - from > 1) {
                    const int64_t step = ((to - from) >> 5) + 1, probe = from + step * (lane + 1);
                    const bool yes = probe >= to || reached(probe);
                    const int k = __ffs(__ballot_sync(0xffffffffu, yes)) - 1;  // the last probe is past the end
                    to = min(to, from + step * (k + 1));
                    from += step * k;
                }
                if (lane == 0) sh.warp_key[warp] = static_cast<uint32_t>(to);
            }
            __syncthreads();
            if (tid == 0) {
                sh.range.lo = sh.warp_key[0];
                sh.range.hi = sh.warp_key[1] - 1;
                sh.range = tidy<F32>(sh.range);
            }
        } else if (tid == 0) {
            sh.range.none = wrapped ? 2 : 1;
        }
        __syncthreads();
    }
    share_range(job, sh);
}

// By block, the mass of the tokens above value `hi`; and the tokens from `lo` to
// it: gathered in this CTA's list, or, one value, counted by block.
template <bool GATHER, bool F32, int TH>
__device__ void sum_blocks(const Row<F32> &row, const Job &job, Shared<TH> &sh, uint32_t lo, uint32_t hi) {
    constexpr int NV = Row<F32>::NV, VE = Row<F32>::VE;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float least = Key<F32>::value(lo), most = Key<F32>::value(hi);
    for (int b = job.b0 + warp; b < job.b1; b += TH / 32) {
        const uint32_t key = sh.block_key[b];
        float s = 0.0f;
        int n = 0;
        if (key >= lo) {
            uint4 w[NV];
            row.load(b, w);
            if (key > hi) s = block_sum<F32, false>(w, key, job.c, job.reach, most);
            const uint32_t in = Row<F32>::between(w, least, most);
            n = __popc(in);
            if constexpr (GATHER) {
                if (__any_sync(0xffffffffu, n > 0)) {
                    const int upto = warp_inclusive(n), turn = row.turn(b);
                    int at = 0;
                    if (lane == 31) at = atomicAdd(&sh.listed, upto);
                    at = __shfl_sync(0xffffffffu, at, 31) + upto - n;
                    for (uint32_t left = in; left; left &= left - 1, ++at) {
                        const int k = Row<F32>::element(__ffs(left) - 1);
                        const int id = b * kBlock + (((lane + 32 * (k / VE)) * VE + k % VE - turn) & (kBlock - 1));
                        if (at < kGather) {
                            sh.list_key[at] = Key<F32>::of(row.at(id));
                            sh.list_id[at] = id;
                        }
                    }
                }
            } else {
                n = __reduce_add_sync(0xffffffffu, n);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        }
        if (lane == 0) {
            sh.block_mass[b] = __float_as_uint(s);
            sh.block_equals[b] = GATHER ? 0 : n;
        }
    }
    __syncthreads();
}

// The CTAs' lists into the first one's, from its end down; its own are at its start.
template <int TH>
__device__ __forceinline__ void hand_over_list(const Job &job, Shared<TH> &sh) {
    if (job.splits > 1 && job.part != 0) {
        const int n = min(sh.listed, kGather);
        if (threadIdx.x == 0 && n > 0) sh.last = static_cast<int>(dsmem_next(&sh.collected, 0, n));
        __syncthreads();
        if (n > 0)
            for (int i = threadIdx.x; i < n && sh.last + i < kGather; i += TH) {
                dsmem_put(&sh.list_key[kGather - 1 - sh.last - i], 0, sh.list_key[i]);
                dsmem_put(&sh.list_id[kGather - 1 - sh.last - i], 0, sh.list_id[i]);
            }
    }
}

// sh.block_mass from sums relative to the block's largest logit to units of the row's.
template <bool F32, int TH>
__device__ __forceinline__ uint64_t weigh_blocks(const Job &job, Shared<TH> &sh) {
    uint64_t mine = 0;
    for (int b = job.b0 + threadIdx.x; b < job.b1; b += TH) {
        const float s = __uint_as_float(static_cast<uint32_t>(sh.block_mass[b]));
        uint64_t v = 0;
        if (s > 0.0f) v = fixed(mul(weight(Key<F32>::value(sh.block_key[b]), job.m, job.c), Two{s, 0.0f}), kUnit);
        sh.block_mass[b] = v;
        mine += v;
    }
    return mine;
}

template <int TH>
__device__ __forceinline__ void hand_over_blocks(const Job &job, Shared<TH> &sh) {
    if (job.splits > 1) {
        if (job.part != 0)
            for (int b = job.b0 + threadIdx.x; b < job.b1; b += TH) {
                dsmem_put(&sh.block_mass[b], 0, sh.block_mass[b]);
                dsmem_put(&sh.block_key[b], 0, sh.block_key[b]);
                dsmem_put(&sh.block_equals[b], 0, sh.block_equals[b]);
            }
        cluster_sync_all();
    }
    __syncthreads();
}

template <int TH, class Each>
__device__ __forceinline__ void for_list(const Shared<TH> &sh, Each each) {
    const int own = min(sh.listed, kGather), n = min(own + sh.collected, kGather);
    for (int i = threadIdx.x; i < n; i += TH) each(i < own ? i : kGather - 1 - (i - own));
}

// The list's tokens whose keys are in sh.range, down to one value.  By the first CTA.
template <bool F32, int TH>
__device__ void search_list(const Job &job, Shared<TH> &sh, const Target &target) {
    constexpr int kBits = 20;  // kGather residuals of 2^20 fit 32 bits
    while (sh.range.lo != sh.range.hi) {
        const uint32_t lo = sh.range.lo, hi = sh.range.hi;
        const int shift = fine_shift(lo, hi);
        const float top = Key<F32>::value(hi);
        for (int i = threadIdx.x; i < kFine; i += TH) sh.fine_n[i] = sh.fine_q[i] = 0;
        __syncthreads();
        for_list(sh, [&](int i) {
            const uint32_t key = sh.list_key[i];
            if (key >= lo && key <= hi) {
                const uint32_t bin = (hi - key) >> shift;
                atomicAdd(&sh.fine_n[bin], 1u);
                atomicAdd(&sh.fine_q[bin], fine_rest(top, Key<F32>::value(key), job.c, static_cast<float>(1 << (5 + kBits))));
            }
        });
        __syncthreads();
        narrow<F32>(job, sh, target, shift, kBits);
    }
}

// The same of a short list, to the end: every token's place among them and the
// mass to it, by comparing all.  The token with the target has the cut.
constexpr int kShort = 256;
static_assert(kShort <= kFine, "list_weight holds a short list");
template <bool F32, int TH>
__device__ void rank_list(const Job &job, Shared<TH> &sh, const Target &target) {
    static_assert(TH >= kShort, "a thread a token");
    const int own = min(sh.listed, kGather), n = own + sh.collected, i = threadIdx.x;
    auto at = [&](int j) { return j < own ? j : kGather - 1 - (j - own); };
    const Range r = sh.range;
    uint32_t key = 0, id = 0;
    uint64_t w = 0;
    if (i < n) {
        key = sh.list_key[at(i)], id = sh.list_id[at(i)];
        w = fixed(weight(Key<F32>::value(key), job.m, job.c), kUnit);
        sh.list_weight[i] = w;
    }
    __syncthreads();
    if (i < n) {
        int before = 0, equals = 0;
        uint64_t mass = 0;
        for (int j = 0; j < n; ++j) {
            const uint32_t k = sh.list_key[at(j)];
            const bool same = k == key && sh.list_id[at(j)] < id, ahead = k > key || same;
            before += ahead ? 1 : 0;
            equals += same ? 1 : 0;
            mass += ahead ? sh.list_weight[j] : 0;
        }
        mass += r.mass;
        const bool last = before == n - 1;
        const bool mine = target.by_mass ? (mass < target.mass || before == 0) && (mass + w >= target.mass || last)
                                         : r.count + before + 1 == target.count || (last && r.count + n < target.count);
        if (mine) sh.range = Range{key, key, r.count + before - equals, equals + 1, mass + w, 0, 0};
    }
    __syncthreads();
}

// From sh.range, the same in all the row's CTAs, to the cut: its value
// (lo = hi), how many of its equals are kept, the mass of all that is.
// `list`: the range whose tokens are gathered and above which blocks are summed.
// After the last search only the first CTA has more than the range that it began
// with, or the one that is in the list.
template <bool F32, int TH>
__device__ void find_cut(const Row<F32> &row, Job &job, Shared<TH> &sh, const Target &target, Range &list, bool last) {
    const int tid = threadIdx.x, warp = tid >> 5;
    const bool listed = list.lo == sh.range.lo && list.hi == sh.range.hi;
    while (!listed && sh.range.equals > kGather && sh.range.lo != sh.range.hi) {
        const uint32_t lo = sh.range.lo, hi = sh.range.hi;
        const int shift = fine_shift(lo, hi);
        const float top = Key<F32>::value(hi), least = Key<F32>::value(lo);
        __syncthreads();
        for (int i = tid; i < kFine; i += TH) sh.fine_n[i] = sh.fine_q[i] = 0;
        __syncthreads();
        for (int b = job.b0 + warp; b < job.b1; b += TH / 32) {
            if (sh.block_key[b] < lo) continue;
            uint4 w[Row<F32>::NV];
            row.load(b, w);
#pragma unroll
            for (int i = 0; i < Row<F32>::NV; ++i) {
                float x[Row<F32>::VE];
                Row<F32>::unpack(w[i], x);
                for (int j = 0; j < Row<F32>::VE; ++j)
                    if (x[j] >= least && x[j] <= top) {
                        const uint32_t bin = (hi - Key<F32>::of(x[j])) >> shift;
                        atomicAdd(&sh.fine_n[bin], 1u);
                        atomicAdd(&sh.fine_q[bin], fine_rest(top, x[j], job.c, static_cast<float>(1 << (5 + job.bits))));
                    }
            }
        }
        __syncthreads();
        collect<TH>(job, sh.fine_n, sh.fine_q, kFine);
        if (job.part == 0) narrow<F32>(job, sh, target, shift, job.bits);
        share_range(job, sh);
    }
    if (!listed && sh.range.lo != sh.range.hi) {
        const bool again = list.lo <= list.hi;
        list = sh.range;
        if (tid == 0) {
            sh.listed = 0;
            if (again) sh.collected = 0;
        }
        __syncthreads();
        if (again && job.splits > 1) cluster_sync_all();
        sum_blocks<true, F32, TH>(row, job, sh, list.lo, list.hi);
        hand_over_list(job, sh);
        weigh_blocks<F32>(job, sh);
        hand_over_blocks(job, sh);
    }
    if (job.part == 0 && sh.range.lo != sh.range.hi && sh.listed + sh.collected <= kShort) {
        rank_list<F32>(job, sh, target);
    } else if (job.part == 0) {
        search_list<F32>(job, sh, target);
        __syncthreads();
        if (tid == 0) {
            const uint64_t w = fixed(weight(Key<F32>::value(sh.range.lo), job.m, job.c), kUnit);
            int kept = target.count - sh.range.count;
            if (target.by_mass) {
                // the fewest whose mass reaches what is missing: a quotient in fp32, put right by products
                const uint64_t miss = target.mass > sh.range.mass ? target.mass - sh.range.mass : 0;
                const uint64_t most = static_cast<uint64_t>(sh.range.equals);
                uint64_t need = most;
                if (w > 0 && miss < most * w) {
                    need = static_cast<uint64_t>(__fdividef(__ull2float_rn(miss), __ull2float_rn(w)));
                    while (need * w < miss) ++need;
                    while (need > 0 && (need - 1) * w >= miss) --need;
                }
                kept = need < 1 ? 1 : static_cast<int>(need < most ? need : most);
            }
            sh.range.equals = kept;
            sh.range.mass += w * static_cast<uint64_t>(kept);
        }
    }
    if (!last) share_range(job, sh);
    else __syncthreads();
}

// ------------------------------------------------------------------ the kernel
// PLAIN: nothing but temperatures are given.
template <bool F32, int TH, bool PLAIN>
__global__ void __launch_bounds__(TH, 1024 / TH) sample_kernel(const SampleArgs a, int splits) {
    extern __shared__ uint4 sample_smem[];
    Shared<TH> &sh = *reinterpret_cast<Shared<TH> *>(sample_smem);
    using K = Key<F32>;
    constexpr int kWarps = TH / 32, kBoundShift = F32 ? 21 : 5;  // keys to kBins
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t r = blockIdx.x / splits;
    Job job;
    job.splits = splits;
    job.turn = 0;
    job.part = static_cast<int>(blockIdx.x - r * splits);
    if (splits > 1) cluster_arrive();  // shared memory of the others is there once all have
    pdl_wait();
    const int vocab = static_cast<int>(a.vocab);
    job.blocks = (vocab + kBlock - 1) / kBlock;
    job.b0 = static_cast<int>(static_cast<int64_t>(job.blocks) * job.part / splits);
    job.b1 = static_cast<int>(static_cast<int64_t>(job.blocks) * (job.part + 1) / splits);
    const Row<F32> row(static_cast<const char *>(a.logits) + r * a.row_stride * (F32 ? 4 : 2), vocab);
    const float temperature = a.temperature ? a.temperature[r] : 1.0f;
    const float top_p = !PLAIN && a.top_p ? a.top_p[r] : 1.0f, min_p = !PLAIN && a.min_p ? a.min_p[r] : 0.0f;
    const float u0 = fminf(fmaxf(a.u[2 * r], 0.0f), 1.0f), u1 = fminf(fmaxf(a.u[2 * r + 1], 0.0f), 1.0f);
    int top_k = !PLAIN && a.top_k ? a.top_k[r] : 0;
    if (top_k <= 0 || top_k > vocab) top_k = vocab;
    const bool greedy = temperature == 0.0f;
    bool bad = !(greedy || (temperature >= 1e-30f && temperature <= 1e30f)) || top_p != top_p || min_p != min_p;
    job.c = div(Two{0x1.715476p+0f, 0x1.4ae0cp-26f}, Two{greedy || bad ? 1.0f : temperature, 0.0f});
    if (!PLAIN && tid < 32) sh.bin_weight[tid] = kBinWeight[tid];
    if (!PLAIN && min_p > 0.0f && tid == TH - 1) sh.log_min_p = log(static_cast<double>(fminf(min_p, 1.0f)));

    const bool by_p = !PLAIN && top_p < 1.0f, by_k = !PLAIN && top_k < vocab && top_k > 1 && !greedy && !bad;
    if (!PLAIN && by_k) {
        for (int i = tid; i < kBins; i += TH) sh.n[i] = 0;
        if (tid == 0) sh.bound = 0;
        __syncthreads();
    }
    // ---- the blocks' largest logits and their masses relative to those
    job.reach = 124.0f / job.c.h;
    for (int b = job.b0 + warp; b < job.b1; b += kWarps) {
        uint4 w[Row<F32>::NV];
        row.load(b, w);
        const uint32_t lane_key = K::of(Row<F32>::most(w)), key = __reduce_max_sync(0xffffffffu, lane_key);
        if (!PLAIN && by_k) atomicAdd(&sh.n[lane_key >> kBoundShift], 1u);
        float s = 0.0f;
        if (key > K::kNegInf && key < K::kInf && !greedy) s = block_sum<F32, true>(w, key, job.c, job.reach, 0.0f);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) {
            sh.block_key[b] = key;
            sh.block_mass[b] = __float_as_uint(s);
            sh.block_equals[b] = 0;
        }
    }
    __syncthreads();
    uint32_t key = 0;
    for (int b = job.b0 + tid; b < job.b1; b += TH) key = max(key, sh.block_key[b]);
    key = __reduce_max_sync(0xffffffffu, key);
    if (lane == 0) sh.warp_key[warp] = key;
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) key = max(key, sh.warp_key[i]);
    uint32_t bound = 0;
    if (!PLAIN && by_k) {
        // the top_k-th largest of the lanes' largest is no larger than the top_k-th of all: the least of its bin
        constexpr int kPer = kBins / TH;
        int n[kPer], sum = 0, all;
        uint64_t none[kPer] = {};
#pragma unroll
        for (int i = 0; i < kPer; ++i) n[i] = static_cast<int>(sh.n[kBins - 1 - (tid * kPer + i)]), sum += n[i];
        const int at = cta_exclusive<int, TH>(sum, sh.warp_int, all);
        find_bin<false, kPer, TH>(n, none, at, 0, Target{false, top_k, 0}, sh, [&](int i, int, uint64_t) {
            sh.bound = static_cast<uint32_t>(kBins - 1 - (tid * kPer + i)) << kBoundShift;
        });
        bound = sh.bound;
    }
    if (!PLAIN && (by_k || by_p)) {
        __syncthreads();
        for (int i = tid; i < kBins; i += TH) sh.n[i] = sh.q[i] = 0;
        if (tid == 0) sh.collected = 0;
        __syncthreads();
    }
    if (splits > 1) {
        cluster_wait();
        if (tid < splits) {
            dsmem_put(&sh.part_key[job.part], tid, key);
            dsmem_put(&sh.part_bound[job.part], tid, bound);
        }
        cluster_sync_all();
        for (int i = 0; i < splits; ++i) {
            key = max(key, sh.part_key[i]);
            bound = max(bound, sh.part_bound[i]);
        }
    }
    job.m_key = key;
    job.m = K::value(key);
    bad = bad || key >= K::kInf;
    if (!PLAIN && min_p > 0.0f && tid == 0)  // the least value whose weight is min_p or more
        sh.min_key = K::from(__double2float_ru(job.m + temperature * sh.log_min_p));
    if (bad || key == K::kNegInf) {  // the same in all of the row's CTAs
        if (job.part == 0 && tid == 0) {
            a.tokens[r] = -1;
            if (a.logprobs) a.logprobs[r] = 0.0f;
            if (bad) atomicOr(&g_sample_err, ERRBIT_INDEX);
        }
        return;
    }
    job.lowest = max(max(K::from(window_end(job.m, job.c.h)), K::kNegInf + 1), bound);
    job.bits = min(32 - (vocab > 1 ? 32 - __clz(vocab - 1) : 0), 18);  // 2^bits residuals of `vocab` tokens fit 32 bits

    // ---- the cut: tokens above its value are kept, and `ties` equal to it
    uint32_t cut = K::kNegInf;
    int ties = 0;
    Range list{1, 0, 0, 0, 0, 0, 0};
    if (greedy || top_k == 1) {
        cut = job.m_key;
        ties = 1;
    } else if (!PLAIN && (by_p || by_k)) {
        uint64_t whole = 0;  // the mass that top_p is a share of; the first CTA's counts
        const uint64_t mine = weigh_blocks<F32>(job, sh);
        cta_exclusive<uint64_t, TH>(mine, sh.warp_sum, whole);
        if (splits > 1 && tid == 0) dsmem_put(&sh.part_mass[job.part], 0, whole);
        int mode = !by_k ? kMasses : by_p ? kBoth : kCounts;
        if (mode == kMasses) count_exponents<F32, TH, kMasses>(row, job, sh);
        else if (mode == kBoth) count_exponents<F32, TH, kBoth>(row, job, sh);
        else count_exponents<F32, TH, kCounts>(row, job, sh);
        if (splits > 1) {
            whole = 0;
            for (int i = 0; i < splits; ++i) whole += sh.part_mass[i];
        }
        if (by_k) {
            const Target target{false, top_k, 0};
            find_exponent<F32>(job, sh, target, mode);
            if (!sh.range.none) {
                find_cut<F32, TH>(row, job, sh, target, list, !by_p);
                cut = sh.range.lo;
                ties = sh.range.equals;
                whole = sh.range.mass;
                __syncthreads();
            }
        }
        if (by_p) {
            const uint64_t share = __float2ull_rz(fmaxf(top_p, 0.0f) * 0x1p64f);
            const Target target{true, 0, at_least_one(__umul64hi(whole, share) + (whole * share != 0 ? 1 : 0))};
            find_exponent<F32>(job, sh, target, mode);
            if (sh.range.none == 2) {
                for (int i = tid; i < kBins; i += TH) sh.n[i] = sh.q[i] = 0;
                __syncthreads();
                if (splits > 1) cluster_sync_all();
                count_exponents<F32, TH, kBoth>(row, job, sh);
                mode = kBoth;
                find_exponent<F32>(job, sh, target, mode);
            }
            if (!sh.range.none) {
                find_cut<F32, TH>(row, job, sh, target, list, true);
                if (sh.range.lo > cut || (sh.range.lo == cut && sh.range.equals < ties))
                    cut = sh.range.lo, ties = sh.range.equals;
                __syncthreads();
            }
        }
    } else if (min_p <= 0.0f) {
        weigh_blocks<F32>(job, sh);
        __syncthreads();
        hand_over_blocks(job, sh);
    }
    if (!PLAIN && min_p > 0.0f && !greedy) {
        __syncthreads();
        const uint32_t k = sh.min_key;
        if (k > cut) cut = k, ties = 0x7FFFFFFF;
    }
    const bool filtered = cut > K::kNegInf;
    const float cut_value = K::value(cut);
    const bool in_list = !PLAIN && list.lo <= cut && cut <= list.hi;
    if (filtered && !in_list) {
        sum_blocks<false, F32, TH>(row, job, sh, cut, cut);
        weigh_blocks<F32>(job, sh);
        __syncthreads();
        hand_over_blocks(job, sh);
    } else if (!PLAIN && !filtered && (by_p || by_k)) {  // neither took a token away
        sum_blocks<false, F32, TH>(row, job, sh, K::kNegInf + 1, K::kNegInf);
        weigh_blocks<F32>(job, sh);
        __syncthreads();
        hand_over_blocks(job, sh);
    }
    if (job.part != 0) return;
    if (!PLAIN && filtered && in_list) {  // what the list holds above the cut, and the cut's equals
        for_list(sh, [&](int i) {
            const uint32_t k = sh.list_key[i], b = sh.list_id[i] / kBlock;
            if (k > cut)
                atomicAdd(reinterpret_cast<unsigned long long *>(&sh.block_mass[b]),
                          static_cast<unsigned long long>(fixed(weight(K::value(k), job.m, job.c), kUnit)));
            else if (k == cut) atomicAdd(&sh.block_equals[b], 1);
        });
        __syncthreads();
    }
    // ---- the block
    uint64_t total;
    {
        constexpr int kPer = kMaxBlocks / TH;
        const uint64_t cut_weight = filtered ? fixed(weight(cut_value, job.m, job.c), kUnit) : 0;
        const int per = (job.blocks + TH - 1) / TH, first = tid * per;  // of this thread
        int n[kPer], sum_n = 0, all_n;
        uint64_t v[kPer], sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const bool have = i < per && first + i < job.blocks;
            n[i] = have && filtered ? sh.block_equals[first + i] : 0;
            v[i] = have ? sh.block_mass[first + i] : 0;
            sum_n += n[i];
        }
        int seen = filtered ? cta_exclusive<int, TH>(sum_n, sh.warp_int, all_n) : 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int keep = min(max(ties - seen, 0), n[i]);
            seen += n[i];
            n[i] = keep;
            v[i] += cut_weight * static_cast<uint64_t>(keep);
            sum += v[i];
        }
        uint64_t at = cta_exclusive<uint64_t, TH>(sum, sh.warp_sum, total);
        uint64_t target = part_of(total, u0);
        if (target >= total) target = total - 1;  // u0 = 1: the last block
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (at <= target && at + v[i] > target) {  // one block
                sh.block = first + i;
                sh.allowed = n[i];
                sh.beside = total - v[i];
            }
            at += v[i];
        }
    }
    __syncthreads();
    // ---- the token: weights relative to the block's largest logit, which is kept if any of the block is
    constexpr int kPer = kBlock / TH;
    const float block_m = K::value(sh.block_key[sh.block]);
    const int e0 = sh.block * kBlock + tid * kPer;
    float x[kPer];
    int eq = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        x[j] = e0 + j < vocab ? row.at(e0 + j) : -INFINITY;
        eq += filtered && x[j] == cut_value ? 1 : 0;
    }
    int all_eq, rank = 0;
    if (filtered) rank = cta_exclusive<int, TH>(eq, sh.warp_int, all_eq);
    uint64_t w[kPer], sum = 0, all;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        bool keep = !filtered || x[j] > cut_value;
        if (filtered && x[j] == cut_value) keep = rank++ < sh.allowed;
        w[j] = keep ? fixed(weight(x[j], block_m, job.c), 0x1p45f) : 0;
        sum += w[j];
    }
    uint64_t at = cta_exclusive<uint64_t, TH>(sum, sh.warp_sum, all);
    uint64_t target = part_of(all, u1);
    if (target >= all) target = all - 1;  // u1 = 1: the last token
    int hit = -1;
    float x_hit = 0.0f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        if (at <= target && at + w[j] > target) hit = j, x_hit = x[j];
        at += w[j];
    }
    if (hit >= 0) {  // one token
        a.tokens[r] = e0 + hit;
        if (a.logprobs) {
            // (x - m) / T - log(mass / 2^41).  Of a mass near that of the largest logit, 2^41, the rest counts: if the
            // block has that logit, its own mass is taken from the weights here (2^-45)
            const uint64_t mass = block_m == job.m ? sh.beside + ((all + 8) >> 4) : total;
            const Two t = mul(mul(two_sum(x_hit, -job.m), job.c), Two{kLn2, -0x1.05c61p-29f});
            a.logprobs[r] = (t.h - log1pf(__ull2float_rn(mass - (1ull << 41)) * (1.0f / kUnit))) + t.l;
        }
    }
}

struct SampleSetup {
    std::mutex mu;
    bool done[64] = {};
    cudaError_t err[64] = {};
};

template <bool F32, int TH, bool PLAIN>
cudaError_t launch_rows(const SampleArgs &a, int splits, cudaStream_t stream) {
    static SampleSetup setup;
    constexpr int kSmem = static_cast<int>(PLAIN ? offsetof(Shared<TH>, n) : sizeof(Shared<TH>));
    static_assert(kSmem * (1024 / TH) <= 227 * 1024, "shared memory per SM");
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(setup.mu);
        if (!setup.done[dev]) {
            setup.err[dev] =
                cudaFuncSetAttribute(sample_kernel<F32, TH, PLAIN>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
            setup.done[dev] = true;
        }
        if (setup.err[dev] != cudaSuccess) return setup.err[dev];
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows * splits), 1, 1);
    cfg.blockDim = dim3(TH, 1, 1);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = static_cast<unsigned>(splits);
    attrs[1].val.clusterDim.y = 1;
    attrs[1].val.clusterDim.z = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = splits > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, sample_kernel<F32, TH, PLAIN>, a, splits);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, cudaStream_t stream) {
    const int64_t blocks = (a.vocab + kBlock - 1) / kBlock, sms = device_sm_count();
    const bool plain = !a.top_k && !a.top_p && !a.min_p;
    // CTAs a row: as many as still give each 8 blocks, and the SMs at most two CTAs, or one without a cut, whose one
    // pass gains less from a second than another exchange costs.  Rows of 152064, us at one CTA and at two an SM:
    // temperature alone 32 rows 9.5 and 11.2, 64 11.9 and 13.5, 100 14.4 and 16.9; with cuts 64 41.1 and 37.5, 100
    // 57.9 and 51.0 (four an SM: 50.6 for 64).  32 rows of 12000 with cuts: 8 blocks 19.7, 4 blocks 22.9; of 32003: 8
    // blocks 25.2, 16 blocks 26.2.
    int splits = 1;
    while (splits < kMaxSplit && 2 * splits * a.rows <= (plain ? sms : 2 * sms) && blocks / (2 * splits) >= 8) splits *= 2;
    // 512 threads a CTA, two an SM (registers).  Without a cut and with more rows than those, 256, four an SM: a row's
    // end leaves fewer idle, 2048 rows of 32003 57.6 and not 79.6 us, 512 of 152064 40.5 and not 43.2 (with the loads
    // ahead of then).  With cuts CTAs of 256 are slower: 64 rows 38.4 and not 37.5, 256 fp32 rows of 32003 53.9 and not
    // 49.7.
    if (plain) {
        if (splits == 1 && a.rows > 2 * sms)
            return a.f32 ? launch_rows<true, 256, true>(a, splits, stream) : launch_rows<false, 256, true>(a, splits, stream);
        return a.f32 ? launch_rows<true, 512, true>(a, splits, stream) : launch_rows<false, 512, true>(a, splits, stream);
    }
    return a.f32 ? launch_rows<true, 512, false>(a, splits, stream) : launch_rows<false, 512, false>(a, splits, stream);
}

uint32_t take_sample_error() {
    uint32_t v = 0;
    if (cudaMemcpyFromSymbol(&v, g_sample_err, sizeof v) != cudaSuccess) return 0xFFFFFFFFu;
    const uint32_t zero = 0;
    cudaMemcpyToSymbol(g_sample_err, &zero, sizeof zero);
    return v;
}

}  // namespace fp8bs
