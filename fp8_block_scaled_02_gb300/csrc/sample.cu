// sample.cu -- the next token of each row of logits, drawn with given random
// numbers from what temperature, top-k, top-p and min-p leave.
//
// With m the row's largest logit, w_j = 2^(c (x_j - m)), c = log2(e) / T.  Kept
// are the first tokens of the order by value, then index: as many as top-k, top-p
// (of the top-k's mass) and min-p all allow, which is a cut, a value and how many
// of its equals.  The first random number picks a block of 1024 tokens by the
// kept mass, the second a token of the block.
//
// Whole numbers come out, so sums are made as exact as it is cheap to.  In a
// block's fp32 sums the exponent is split into an integer and a rest below 1/2
// that is within 2^-25, so that a weight is within the 2^-22 of ex2 and errors of
// different values do not add up; blocks, cuts and the tokens of the drawn block
// go by pairs of fp32 (2^-44).
//
// The CTAs of a cluster (one CTA when there are many rows) have consecutive
// blocks of a row each, a warp a block at a time.  The cut comes from histograms
// over the values: counts, and the mass of each bin as its count times a weight of
// the bin plus what its tokens differ from that, in whole numbers, so that the
// order of the atomics does not matter.
#include "twofloat.cuh"

#include "serving.cuh"
#include "internal.h"

namespace fp8bs {

namespace {

__device__ uint32_t g_sample_err;

constexpr int kBlock = 1024;                    // tokens of a block
constexpr int kMaxBlocks = kSampleMaxVocab / kBlock;
constexpr int kMaxSplit = 8;                    // CTAs a row
constexpr int kBins = 2048;
constexpr float kPerUnit = 32.0f;               // first-level bins in a factor 2 of the weight
constexpr float kWindow = kBins / kPerUnit - 1; // in log2: lighter tokens are drawn with a chance below 2^-43
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMagic = 12582912.0f;           // 1.5 * 2^23: adding it rounds to whole numbers
constexpr float kResidual = 0.0225f;            // above 2^(1 / 32) - 1: what weights of one bin differ by

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Order of the values as unsigned integers: -0 is +0, NaN above everything.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    return x != x ? 0xFFFFFFFFu : u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
constexpr uint32_t kKeyInf = 0xFF800000u, kKeyNegInf = 0x007FFFFFu;

__device__ __forceinline__ Two neg(Two a) { return Two{-a.h, -a.l}; }
__device__ __forceinline__ bool above(Two a, Two b) { return add(a, neg(b)).h > 0.0f; }
__device__ __forceinline__ Two shfl(Two a, int lane) {
    return Two{__shfl_sync(0xffffffffu, a.h, lane), __shfl_sync(0xffffffffu, a.l, lane)};
}
__device__ __forceinline__ Two shfl_up(Two a, int o) {
    return Two{__shfl_up_sync(0xffffffffu, a.h, o), __shfl_up_sync(0xffffffffu, a.l, o)};
}
__device__ __forceinline__ Two warp_inclusive(Two v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Two y = shfl_up(v, o);
        if (lane >= o) v = add(y, v);
    }
    return v;
}
__device__ __forceinline__ int warp_inclusive(int v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
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

__device__ __forceinline__ uint4 ld_v4_cached(const void *p) {
    uint4 v;
    asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// A row of logits by blocks: lane l of the warp that has block b holds NV vectors
// of VE elements, of element b * 1024 + (l + 32 i) * VE on; -inf past the row.
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
    __device__ __forceinline__ uint4 slow(int e0) const {  // at the row's ends
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
    // Elements e0 .. e0 + VE - 1 of a row that is off a boundary, from the two vectors that hold them.
    __device__ __forceinline__ uint4 shifted(int e0) const {
        const char *p = base + static_cast<int64_t>(e0) * ES - off;
        const uint4 a = ld_v4_cached(p), b = ld_v4_cached(p + 16);
        uint32_t w[5];
        switch (off >> 2) {
            case 0: w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x; break;
            case 1: w[0] = a.y, w[1] = a.z, w[2] = a.w, w[3] = b.x, w[4] = b.y; break;
            case 2: w[0] = a.z, w[1] = a.w, w[2] = b.x, w[3] = b.y, w[4] = b.z; break;
            default: w[0] = a.w, w[1] = b.x, w[2] = b.y, w[3] = b.z, w[4] = b.w; break;
        }
        const int bits = (off & 3) * 8;
        return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                          __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
    }
    __device__ __forceinline__ void load(int b, uint4 (&w)[NV]) const {
        const int first = b * kBlock + (threadIdx.x & 31) * VE;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e0 = first + i * 32 * VE;
            if (off == 0) w[i] = e0 + VE <= vocab ? ld_v4(base + static_cast<int64_t>(e0) * ES) : slow(e0);
            else w[i] = e0 * ES >= off && e0 + 2 * VE <= vocab ? shifted(e0) : slow(e0);
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

// What a search for a cut has found so far: the tokens above value key_value(hi)
// are count and mass; the cut lies among the values of keys lo .. hi.
struct Found {
    uint32_t lo, hi;
    int count;     // of tokens above
    int equals;    // of tokens at the cut's value, once lo == hi
    Two mass;      // of tokens above
    int state;     // 0: go on, 1: found (lo == hi), 2: there is no cut, every token is kept
    int pad;
};

template <int TH>
struct Shared {
    static constexpr int kWarps = TH / 32;
    uint32_t n[kBins], q[kBins];  // a level's histogram: tokens, and what they weigh beside the bin's weight
    uint32_t block_key[kMaxBlocks];
    Two block_mass[kMaxBlocks];   // of the kept tokens above the cut's value; the first CTA has all blocks'
    int block_equals[kMaxBlocks]; // tokens at the cut's value
    Two fine[64], coarse[32];     // 2^-(j / 32), 2^-(2 i)
    Found found;
    Two c, warp_two[kWarps];
    int warp_int[kWarps];
    uint32_t part_key[kMaxSplit];
    Two part_mass[kMaxSplit];
    int bad, drawn, last, result_block, allowed;
    Two total;
    double log_min_p;
    uint32_t warp_key[kWarps];
};

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

// The sums of the threads' values before this thread's, and of all.
template <int TH>
__device__ __forceinline__ Two cta_exclusive(Two v, Shared<TH> &sh, Two &all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Two upto = warp_inclusive(v);
    __syncthreads();
    if (lane == 31) sh.warp_two[warp] = upto;
    __syncthreads();
    const Two w = warp_inclusive(lane < TH / 32 ? sh.warp_two[lane] : Two{0.0f, 0.0f});
    all = shfl(w, 31);
    const Two before = shfl(w, warp > 0 ? warp - 1 : 0);
    Two lanes = shfl_up(upto, 1);
    if (lane == 0) lanes = Two{0.0f, 0.0f};
    return warp > 0 ? add(before, lanes) : lanes;
}

template <int TH>
__device__ __forceinline__ int cta_exclusive(int v, Shared<TH> &sh, int &all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int upto = warp_inclusive(v);
    __syncthreads();
    if (lane == 31) sh.warp_int[warp] = upto;
    __syncthreads();
    const int w = warp_inclusive(lane < TH / 32 ? sh.warp_int[lane] : 0);
    all = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    return (warp > 0 ? before : 0) + upto - v;
}

// 2^(c (x - m)).
__device__ __forceinline__ Two weight(float x, float m, Two c) {
    if (!(x > -INFINITY)) return Two{0.0f, 0.0f};
    const Two d = two_sum(x, -m);
    const float t = d.h * c.h;
    return t > -125.0f ? two_exp2(mul(d, c)) : Two{0.0f, 0.0f};
}

// A lane's sum of 2^(c (x - m)) of its elements for which keep(x) holds.
template <bool F32, class Keep>
__device__ __forceinline__ float block_sum(const uint4 (&w)[Row<F32>::NV], float m, float floor, Two c, Keep keep) {
    constexpr int VE = Row<F32>::VE;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < Row<F32>::NV; ++i) {
        float x[VE], part = 0.0f;
        Row<F32>::unpack(w[i], x);
#pragma unroll
        for (int j = 0; j < VE; ++j) {
            const float d = fmaxf(x[j] - m, floor);
            const float r = fmaf(d, c.h, kMagic), n = r - kMagic;
            const float f = fmaf(d, c.l, fmaf(d, c.h, -n));
            // 2^n: the low bits of r are n; n >= -125 by the floor
            const float v = ex2(f) * __uint_as_float((__float_as_uint(r) << 23) + 0x3F800000u);
            part += keep(x[j]) ? v : 0.0f;
        }
        sum += part;
    }
    return sum;
}

struct Job {
    float m;       // the row's largest logit
    uint32_t m_key;
    Two c;
    float floor;   // of x - m: below it a weight counts as 2^-125 or less
    int b0, b1, blocks, part, splits;
    float inv_q;   // of the histogram's residuals
    float q_scale;
};

// ------------------------------------------------------------ the cut's search
// One level: a histogram of the tokens whose values' keys are in [lo, hi], over
// the row's CTAs, and the bin in which `count` (mass = false) or `mass` is reached.
// The first level has bins of equal ratio of weights, the others of equal numbers of values.
template <bool F32, int TH>
__device__ void level(const Row<F32> &row, const Job &job, Shared<TH> &sh, bool first, bool want_mass, bool by_mass,
                      int count, Two mass) {
    constexpr int VE = Row<F32>::VE, NV = Row<F32>::NV;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t lo = sh.found.lo, hi = sh.found.hi;
    const int count0 = sh.found.count;
    const Two mass0 = sh.found.mass;
    int shift = 0;
    while (((hi - lo) >> shift) >= kBins) ++shift;
    const float top = key_value(hi);
    const Two c = job.c;
    const Two c32{c.h * kPerUnit, c.l * kPerUnit};
    const float half_bin = 0.9892f;  // below 2^-(1 / 64), the lightest of a bin to its middle
    for (int i = tid; i < kBins; i += TH) sh.n[i] = sh.q[i] = 0;
    __syncthreads();
    for (int b = job.b0 + warp; b < job.b1; b += TH / 32) {
        if (sh.block_key[b] < lo) continue;
        uint4 w[NV];
        row.load(b, w);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float x[VE];
            Row<F32>::unpack(w[i], x);
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                const uint32_t key = order_key(x[j]);
                if (key < lo || key > hi) continue;
                uint32_t bin;
                float rest;  // weight / the bin's - its least, or 1 - weight / the range's largest
                if (first) {
                    const float d = job.m - x[j];
                    const float r = fmaf(d, c32.h, kMagic), n = r - kMagic;
                    const float f = fmaf(d, c32.l, fmaf(d, c32.h, -n)) * (kLn2 / kPerUnit);
                    bin = __float_as_uint(r) & 0xFFFFu;
                    rest = fmaf(f, fmaf(f, fmaf(f, -1.0f / 6.0f, 0.5f), -1.0f), 1.0f - half_bin);
                } else {
                    bin = (hi - key) >> shift;
                    const float d = top - x[j];
                    const float f = fmaf(d, c.l, d * c.h) * kLn2;
                    rest = f * fmaf(f, fmaf(f, 1.0f / 6.0f, -0.5f), 1.0f);
                }
                if (bin >= kBins) continue;
                atomicAdd(&sh.n[bin], 1u);
                if (want_mass) atomicAdd(&sh.q[bin], static_cast<uint32_t>(__float2int_rn(rest * job.q_scale)));
            }
        }
    }
    __syncthreads();
    if (job.splits > 1) {
        cluster_sync_all();
        if (job.part != 0) {
            for (int i = tid; i < kBins; i += TH) {
                const uint32_t n = sh.n[i];
                if (n) {
                    dsmem_add(&sh.n[i], 0, n);
                    if (want_mass) dsmem_add(&sh.q[i], 0, sh.q[i]);
                }
            }
        }
        cluster_sync_all();
    }
    if (job.part == 0) {
        constexpr int kPer = kBins / TH;
        Two bin_mass[kPer], sum{0.0f, 0.0f};
        int bin_n[kPer], sum_n = 0;
        const Two range_top = want_mass && !first ? weight(top, job.m, c) : Two{0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int bin = tid * kPer + i;
            bin_n[i] = static_cast<int>(sh.n[bin]);
            sum_n += bin_n[i];
            bin_mass[i] = Two{0.0f, 0.0f};
            if (want_mass && bin_n[i] > 0) {
                // the count (exact in fp32: at most 2^20) times the bin's weight, and the rest
                const Two rest = mul(two_prod(1.0f, static_cast<float>(sh.q[bin] >> 12) * 4096.0f), Two{job.inv_q, 0.0f});
                const Two rest2 = add(rest, static_cast<float>(sh.q[bin] & 4095u) * job.inv_q);
                if (first)
                    bin_mass[i] = mul(mul(sh.coarse[bin >> 6], sh.fine[bin & 63]),
                                      add(two_prod(static_cast<float>(bin_n[i]), half_bin), rest2));
                else
                    bin_mass[i] = mul(range_top, add(neg(rest2), static_cast<float>(bin_n[i])));
                sum = add(sum, bin_mass[i]);
            }
        }
        int all_n;
        Two all;
        int at_n = count0 + cta_exclusive(sum_n, sh, all_n);
        Two at{0.0f, 0.0f};
        if (want_mass) at = add(mass0, cta_exclusive(sum, sh, all));
        if (tid == 0) sh.found.state = 2;
        __syncthreads();
        int hit = -1;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (bin_n[i] > 0 && hit < 0) {
                const Two next = add(at, bin_mass[i]);
                if (by_mass ? !above(mass, next) : at_n + bin_n[i] >= count) {
                    hit = i;
                } else {
                    at_n += bin_n[i];
                    at = next;
                }
            }
        }
        // the first thread that has a hit; threads before it ended below the target, those after began above it
        const int hits = hit >= 0 ? tid : TH;
        const int lowest = __reduce_min_sync(0xffffffffu, hits);
        if (lane == 0) sh.warp_int[warp] = lowest;
        __syncthreads();
        int who = TH;
        for (int i = 0; i < TH / 32; ++i) who = min(who, sh.warp_int[i]);
        if (tid == who) {
            const int bin = tid * kPer + hit;
            Found f;
            f.count = at_n;
            f.mass = at;
            f.equals = bin_n[hit];
            f.pad = 0;
            if (first) {
                // the values of a bin: from its number's first key to its last (keys fall as bins rise)
                f.lo = f.hi = bin;  // resolved below
                f.state = 3;
            } else {
                f.hi = hi - (static_cast<uint32_t>(bin) << shift);
                f.lo = f.hi - lo < (1u << shift) ? lo : f.hi - (1u << shift) + 1;
                f.state = f.lo == f.hi ? 1 : 0;
            }
            sh.found = f;
        }
        __syncthreads();
        if (sh.found.state == 3) {
            // the first key from `lo` on whose bin is at most `bin` (warp 0), and the last whose bin is at least `bin`
            const int bin = static_cast<int>(sh.found.hi);
            __syncthreads();
            if (warp < 2) {
                const int want = warp == 0 ? bin : bin - 1;
                int64_t from = static_cast<int64_t>(lo) - 1, to = static_cast<int64_t>(hi) + 1;  // (from, to] holds it
                while (to - from > 1) {
                    const int64_t step = (to - from) / 33 + 1, probe = from + step * (lane + 1);
                    bool reached = true;
                    if (probe < to) {
                        const float d = job.m - key_value(static_cast<uint32_t>(probe));
                        const float r = fmaf(d, c32.h, kMagic);
                        reached = static_cast<int>(__float_as_uint(r) & 0xFFFFu) <= want;
                    }
                    const int k = __ffs(__ballot_sync(0xffffffffu, reached)) - 1;  // of the first, -1: none
                    const int64_t base = from;
                    from = k < 0 ? base + 32 * step : base + k * step;
                    if (k >= 0) to = min(to, base + (k + 1) * step);
                }
                if (lane == 0) sh.warp_key[warp] = static_cast<uint32_t>(to);
            }
            __syncthreads();
            if (tid == 0) {
                sh.found.lo = sh.warp_key[0];
                sh.found.hi = sh.warp_key[1] - 1;
                sh.found.state = sh.found.lo == sh.found.hi ? 1 : 0;
            }
            __syncthreads();
        }
        if (job.splits > 1 && tid > 0 && tid < job.splits) dsmem_put(&sh.found, tid, sh.found);
    }
    if (job.splits > 1) cluster_sync_all();
    __syncthreads();
}

template <bool F32, int TH>
__device__ Found search(const Row<F32> &row, const Job &job, Shared<TH> &sh, bool want_mass, bool by_mass, int count,
                        Two mass, uint32_t lowest) {
    __syncthreads();
    if (threadIdx.x == 0) sh.found = Found{lowest, job.m_key, 0, 0, Two{0.0f, 0.0f}, 0, 0};
    __syncthreads();
    bool first = true;
    while (sh.found.state == 0) {
        level<F32, TH>(row, job, sh, first, want_mass, by_mass, count, mass);
        first = false;
    }
    return sh.found;
}

// ------------------------------------------------------------------ the kernel
template <bool F32, int TH>
__global__ void __launch_bounds__(TH, 1024 / TH) sample_kernel(const SampleArgs a, int splits) {
    __shared__ Shared<TH> sh;
    constexpr int kWarps = TH / 32, NV = Row<F32>::NV;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t r = blockIdx.x / splits;
    Job job;
    job.splits = splits;
    job.part = static_cast<int>(blockIdx.x - r * splits);
    if (splits > 1) cluster_arrive();  // shared memory of the others is there once all have
    pdl_wait();
    const int vocab = static_cast<int>(a.vocab);
    job.blocks = (vocab + kBlock - 1) / kBlock;
    job.b0 = static_cast<int>(static_cast<int64_t>(job.blocks) * job.part / splits);
    job.b1 = static_cast<int>(static_cast<int64_t>(job.blocks) * (job.part + 1) / splits);
    const Row<F32> row(static_cast<const char *>(a.logits) + r * a.row_stride * (F32 ? 4 : 2), vocab);
    const float temperature = a.temperature ? a.temperature[r] : 1.0f;
    const float top_p = a.top_p ? a.top_p[r] : 1.0f, min_p = a.min_p ? a.min_p[r] : 0.0f;
    int top_k = a.top_k ? a.top_k[r] : 0;
    if (top_k <= 0 || top_k > vocab) top_k = vocab;
    const bool greedy = temperature == 0.0f;
    bool bad = !(greedy || (temperature >= 1e-30f && temperature <= 1e30f)) || top_p != top_p || min_p != min_p;
    job.c = div(Two{0x1.715476p+0f, 0x1.4ae0cp-26f}, Two{greedy || bad ? 1.0f : temperature, 0.0f});
    job.floor = -124.0f / job.c.h;
    if (min_p > 0.0f && tid == TH - 1) sh.log_min_p = log(static_cast<double>(fminf(min_p, 1.0f)));

    // ---- the blocks' largest logits and their masses relative to those
    for (int b = job.b0 + warp; b < job.b1; b += kWarps) {
        uint4 w[NV];
        row.load(b, w);
        const uint32_t key = __reduce_max_sync(0xffffffffu, order_key(Row<F32>::most(w)));
        const float m = key_value(key);
        float s = 0.0f;
        if (key > kKeyNegInf && key < kKeyInf) s = block_sum<F32>(w, m, job.floor, job.c, [](float) { return true; });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) {
            sh.block_key[b] = key;
            sh.block_mass[b] = Two{s, 0.0f};
        }
    }
    __syncthreads();
    uint32_t key = 0;
    for (int b = job.b0 + tid; b < job.b1; b += TH) key = max(key, sh.block_key[b]);
    key = __reduce_max_sync(0xffffffffu, key);
    if (lane == 0) sh.warp_key[warp] = key;
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) key = max(key, sh.warp_key[i]);
    if (splits > 1) {
        cluster_wait();
        if (tid < splits) dsmem_put(&sh.part_key[job.part], tid, key);
        cluster_sync_all();
        for (int i = 0; i < splits; ++i) key = max(key, sh.part_key[i]);
    }
    job.m_key = key;
    job.m = key_value(key);
    bad = bad || key >= kKeyInf;
    if (bad || key == kKeyNegInf) {  // the same in all of the row's CTAs
        if (job.part == 0 && tid == 0) {
            a.tokens[r] = -1;
            if (a.logprobs) a.logprobs[r] = 0.0f;
            if (bad) atomicOr(&g_sample_err, ERRBIT_INDEX);
        }
        return;
    }
    // ---- the blocks' masses relative to the row's largest
    Two mine{0.0f, 0.0f};
    for (int b = job.b0 + tid; b < job.b1; b += TH) {
        const uint32_t bk = sh.block_key[b];
        const Two v = bk == kKeyNegInf ? Two{0.0f, 0.0f} : mul(weight(key_value(bk), job.m, job.c), sh.block_mass[b]);
        sh.block_mass[b] = v;
        sh.block_equals[b] = 0;
        mine = add(mine, v);
    }
    // ---- the cut
    uint32_t cut = kKeyNegInf;  // tokens above it are kept, and `ties` equal to it
    int ties = 0;
    if (greedy || top_k == 1) {
        cut = job.m_key;
        ties = 1;
    } else {
        int log_v = 0;
        while ((1 << log_v) < vocab) ++log_v;
        const float q_max = static_cast<float>(1u << (31 - log_v > 24 ? 24 : 31 - log_v));
        job.q_scale = q_max / kResidual;
        job.inv_q = kResidual / q_max;
        const bool by_p = top_p < 1.0f, by_k = top_k < vocab;
        const float window = job.m - kWindow / job.c.h;
        const uint32_t lowest = max(order_key(window), kKeyNegInf + 1);
        if (by_p || by_k) {
            if (tid < 64) sh.fine[tid] = two_exp2(Two{-static_cast<float>(tid) / kPerUnit, 0.0f});
            else if (tid < 96) sh.coarse[tid - 64] = Two{exp2f(-2.0f * static_cast<float>(tid - 64)), 0.0f};
            __syncthreads();
        }
        Two whole{0.0f, 0.0f};  // the mass that top_p is a share of
        if (by_k) {
            const Found f = search<F32, TH>(row, job, sh, by_p, false, top_k, Two{0.0f, 0.0f}, lowest);
            if (f.state == 1) {
                cut = f.lo;
                ties = top_k - f.count;
                whole = add(f.mass, mul(weight(key_value(f.lo), job.m, job.c), Two{static_cast<float>(ties), 0.0f}));
            }
        }
        if (by_p) {
            if (cut == kKeyNegInf) {
                Two all;
                cta_exclusive(mine, sh, all);
                whole = all;
                if (splits > 1) {
                    if (tid < splits) dsmem_put(&sh.part_mass[job.part], tid, all);
                    cluster_sync_all();
                    whole = sh.part_mass[0];
                    for (int i = 1; i < splits; ++i) whole = add(whole, sh.part_mass[i]);
                }
            }
            const Two target = mul(whole, Two{fmaxf(top_p, 0.0f), 0.0f});
            const Found f = search<F32, TH>(row, job, sh, true, true, 0, target, lowest);
            if (f.state == 1) {
                // the fewest equals that reach the target
                const Two w = weight(key_value(f.lo), job.m, job.c);
                const Two need = div(add(target, neg(f.mass)), w);
                const float whole_need = ceilf(need.h) + (need.h == ceilf(need.h) && need.l > 0.0f ? 1.0f : 0.0f);
                const int n = whole_need < 1.0f ? 1 : min(f.equals, static_cast<int>(whole_need));
                if (f.lo > cut || (f.lo == cut && n < ties)) cut = f.lo, ties = n;
            }
        }
        if (min_p > 0.0f) {
            // the least value whose weight is min_p or more
            const uint32_t k = order_key(__double2float_ru(job.m + temperature * sh.log_min_p));
            if (k > cut) cut = k, ties = 0x7FFFFFFF;
        }
    }
    const bool filtered = cut > kKeyNegInf;
    const float cut_value = key_value(cut);
    // ---- the masses of the kept tokens above the cut's value, and its equals
    if (filtered) {
        __syncthreads();
        for (int b = job.b0 + warp; b < job.b1; b += kWarps) {
            const uint32_t bk = sh.block_key[b];
            float s = 0.0f;
            int n = 0;
            if (bk >= cut) {
                uint4 w[NV];
                row.load(b, w);
                s = block_sum<F32>(w, key_value(bk), job.floor, job.c, [&](float x) { return x > cut_value; });
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    float x[Row<F32>::VE];
                    Row<F32>::unpack(w[i], x);
#pragma unroll
                    for (int j = 0; j < Row<F32>::VE; ++j) n += x[j] == cut_value ? 1 : 0;
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                n = __reduce_add_sync(0xffffffffu, n);
            }
            if (lane == 0) {
                sh.block_mass[b] = s > 0.0f ? mul(weight(key_value(bk), job.m, job.c), Two{s, 0.0f}) : Two{0.0f, 0.0f};
                sh.block_equals[b] = n;
            }
        }
    }
    __syncthreads();
    if (splits > 1) {
        if (job.part != 0)
            for (int b = job.b0 + tid; b < job.b1; b += TH) {
                dsmem_put(&sh.block_mass[b], 0, sh.block_mass[b]);
                dsmem_put(&sh.block_equals[b], 0, sh.block_equals[b]);
            }
        cluster_sync_all();
        if (job.part != 0) return;
    }
    // ---- the block
    const float u0 = fminf(fmaxf(a.u[2 * r], 0.0f), 1.0f), u1 = fminf(fmaxf(a.u[2 * r + 1], 0.0f), 1.0f);
    const Two cut_weight = filtered ? weight(cut_value, job.m, job.c) : Two{0.0f, 0.0f};
    if (warp == 0) {
        const int per = (job.blocks + 31) / 32, first = lane * per, end = min(first + per, job.blocks);
        int n = 0;
        for (int b = first; b < end; ++b) n += sh.block_equals[b];
        const int before = warp_inclusive(n) - n;
        Two sum{0.0f, 0.0f};
        int seen = before;
        for (int b = first; b < end; ++b) {
            const int e = sh.block_equals[b], keep = min(max(ties - seen, 0), e);
            seen += e;
            Two v = sh.block_mass[b];
            if (keep > 0) v = add(v, mul(cut_weight, Two{static_cast<float>(keep), 0.0f}));
            sh.block_mass[b] = v;
            sh.block_equals[b] = keep;
            sum = add(sum, v);
        }
        const Two upto = warp_inclusive(sum), all = shfl(upto, 31);
        const Two target = mul(all, Two{u0, 0.0f});
        Two at = shfl_up(upto, 1);
        if (lane == 0) at = Two{0.0f, 0.0f};
        int hit = -1, last = -1;
        for (int b = first; b < end; ++b) {
            const Two v = sh.block_mass[b];
            if (v.h > 0.0f) {
                at = add(at, v);
                last = b;
                if (hit < 0 && above(at, target)) hit = b;
            }
        }
        const uint32_t have = __ballot_sync(0xffffffffu, hit >= 0);
        last = __reduce_max_sync(0xffffffffu, last);
        hit = have ? __shfl_sync(0xffffffffu, hit, __ffs(have) - 1) : last;
        if (lane == 0) {
            sh.result_block = hit;
            sh.allowed = sh.block_equals[hit];
            sh.total = all;
            sh.drawn = 0x7FFFFFFF;
            sh.last = -1;
        }
    }
    __syncthreads();
    // ---- the token
    constexpr int kPer = kBlock / TH;
    const int e0 = sh.result_block * kBlock + tid * kPer;
    float x[kPer];
    int eq = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        x[j] = e0 + j < vocab ? row.at(e0 + j) : -INFINITY;
        eq += filtered && x[j] == cut_value ? 1 : 0;
    }
    int all_eq, rank = 0;
    if (filtered) rank = cta_exclusive(eq, sh, all_eq);
    Two w[kPer], sum{0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        bool keep = !filtered || x[j] > cut_value;
        if (filtered && x[j] == cut_value) keep = rank++ < sh.allowed;
        w[j] = keep ? weight(x[j], job.m, job.c) : Two{0.0f, 0.0f};
        sum = add(sum, w[j]);
    }
    Two all;
    Two at = cta_exclusive(sum, sh, all);
    const Two target = mul(all, Two{u1, 0.0f});
    int hit = 0x7FFFFFFF, last = -1;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        if (w[j].h > 0.0f) {
            at = add(at, w[j]);
            last = e0 + j;
            if (hit == 0x7FFFFFFF && above(at, target)) hit = e0 + j;
        }
    }
    hit = static_cast<int>(__reduce_min_sync(0xffffffffu, hit));
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 0) {
        atomicMin(&sh.drawn, hit);
        atomicMax(&sh.last, last);
    }
    __syncthreads();
    const int token = sh.drawn != 0x7FFFFFFF ? sh.drawn : sh.last;
    if (tid == 0) {
        a.tokens[r] = token;
        if (a.logprobs) {
            // (x - m) / T - log W, with W = h (1 + l / h)
            const Two t = mul(mul(two_sum(row.at(token), -job.m), job.c), Two{kLn2, -0x1.05c61p-29f});
            a.logprobs[r] = (t.h - logf(sh.total.h)) + (t.l - sh.total.l / sh.total.h);
        }
    }
}

template <bool F32, int TH>
cudaError_t launch_rows(const SampleArgs &a, int splits, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows * splits), 1, 1);
    cfg.blockDim = dim3(TH, 1, 1);
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
    return cudaLaunchKernelEx(&cfg, sample_kernel<F32, TH>, a, splits);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, cudaStream_t stream) {
    const int64_t blocks = (a.vocab + kBlock - 1) / kBlock, sms = device_sm_count();
    int splits = 1;
    while (splits < kMaxSplit && 2 * splits * a.rows <= 2 * sms && blocks / (2 * splits) >= 8) splits *= 2;
    return a.f32 ? launch_rows<true, 512>(a, splits, stream) : launch_rows<false, 512>(a, splits, stream);
}

uint32_t take_sample_error() {
    uint32_t v = 0;
    if (cudaMemcpyFromSymbol(&v, g_sample_err, sizeof v) != cudaSuccess) return 0xFFFFFFFFu;
    const uint32_t zero = 0;
    cudaMemcpyToSymbol(g_sample_err, &zero, sizeof zero);
    return v;
}

}  // namespace fp8bs
