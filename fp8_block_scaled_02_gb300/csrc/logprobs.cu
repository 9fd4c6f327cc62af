// logprobs.cu -- log probabilities of given tokens over a row of logits, the
// row's entropy, and its top alternatives.
//
// With m = max x, l = sum e^(x - m), t = sum (x - m) e^(x - m) over the row:
//   lse = m + log l,  logprob(i) = x_i - lse,  entropy = log l - t / l.
// The top alternatives are the first k of the row ordered by value, highest
// first, and by index, lowest first, among equals.
//
// The row is read once, 16 bytes a load, by the CTAs of one cluster (one CTA
// when there are many rows); every thread keeps a running (m, l, t) of its
// elements.  The top comes out of the same maxima: the k-th largest of the
// maxima of disjoint groups of threads is a lower bound of the row part's
// k-th largest element.  The pieces (an eighth or so of a thread's elements)
// whose maximum reaches it are read again, from L2, and what reaches the
// bound is ranked in shared memory.  Rows of equals, such as masked ones,
// whose equals at the bound do not fit there take an ordered scan that stops
// when it has enough.
//
// In bytes 92 us for 2048 rows of 152064 bf16 at the measured copy rate: 100 us
// without the top, 121 us with the top 20 (5.2 TB/s).  The difference is the
// choice of the top, in which a CTA reads little.  No unit is at its limit (issue
// slots 68%, ALU 38%, FMA 32%, XU 29%): 64 registers leave 32 warps an SM, 29 at
// work, and loads that are awaited are by far the first stall.
#include "serving.cuh"
#include "internal.h"

namespace fp8bs {

namespace {

__device__ uint32_t g_lp_err;

constexpr int kLpMaxSplit = 8;   // CTAs per row
constexpr int kLpCandidates = 1024;
static_assert(kLogprobsMaxTop <= 32, "the bound comes from 32 maxima");
constexpr int kLpPieces = 8;     // of a thread's vectors
constexpr int kFlight = 6;       // 16-byte loads in flight per thread: 132 us at 2048 x 152064 bf16, 138 with four
constexpr float kLog2e = 1.4426950408889634f;
// (x - m) below this has weight 0 in fp32; it keeps -inf out of t
constexpr float kLowest = -200.0f;

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

template <bool F32>
__device__ __forceinline__ const void *row_start(const LogprobArgs &a, int64_t r) {
    return static_cast<const char *>(a.logits) + r * a.row_stride * (F32 ? 4 : 2);
}

// Order of the values as unsigned integers: -0 is +0, NaN below everything.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    return x != x ? 0u : u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct Sums {
    float m, l, t;
};

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Over groups of `width` lanes: brought to the largest maximum once, then added.
__device__ __forceinline__ Sums warp_merge(Sums s, int width = 32) {
    float m = s.m;
#pragma unroll
    for (int o = width / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float d = s.m == -INFINITY ? kLowest : fmaxf(s.m - m, kLowest), c = ex2(d * kLog2e);
    float l = c * s.l, t = c * (s.t + d * s.l);
#pragma unroll
    for (int o = width / 2; o > 0; o >>= 1) {
        l += __shfl_xor_sync(0xffffffffu, l, o);
        t += __shfl_xor_sync(0xffffffffu, t, o);
    }
    return Sums{m, l, t};
}

// One row as vectors of 16 aligned bytes; the first and the last may reach
// beyond the row, where `pre` elements stand before it.
template <bool F32>
struct Row {
    static constexpr int VE = F32 ? 4 : 8;
    const char *base;  // of vector 0
    int64_t vocab;
    int pre, vecs;

    __device__ __forceinline__ Row(const void *row, int64_t v) : vocab(v) {
        const uintptr_t p = reinterpret_cast<uintptr_t>(row);
        pre = static_cast<int>(p & 15) / (F32 ? 4 : 2);
        base = reinterpret_cast<const char *>(p & ~static_cast<uintptr_t>(15));
        vecs = static_cast<int>((v + pre + VE - 1) / VE);
    }
    __device__ __forceinline__ int64_t element(int vec, int j) const { return static_cast<int64_t>(vec) * VE - pre + j; }
    __device__ __forceinline__ bool whole(int vec) const {
        return static_cast<int64_t>(vec) * VE >= pre && static_cast<int64_t>(vec + 1) * VE - pre <= vocab;
    }
    __device__ __forceinline__ float at(int64_t e) const {
        if constexpr (F32) return reinterpret_cast<const float *>(base)[pre + e];
        else return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(base)[pre + e]);
    }
    // The vector's values; -inf for what is not in the row.
    __device__ __forceinline__ void load(int vec, float (&x)[VE]) const {
        const char *p = base + static_cast<int64_t>(vec) * 16;
        if (whole(vec)) {
            unpack(ld_v4(p), x);
            return;
        }
#pragma unroll
        for (int j = 0; j < VE; ++j) {
            const int64_t e = element(vec, j);
            x[j] = -INFINITY;
            if (e >= 0 && e < vocab) {
                if constexpr (F32) x[j] = reinterpret_cast<const float *>(p)[j];
                else x[j] = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[j]);
            }
        }
    }
    // The vector's values raised to FastSums' floor; returns the largest before that.
    __device__ __forceinline__ float load_fast(int vec, float (&x)[VE]) const {
        load(vec, x);
        float vm = -INFINITY;
#pragma unroll
        for (int j = 0; j < VE; ++j) {
            vm = fmaxf(vm, x[j]);
            x[j] = fmaxf(x[j], -1e38f);
        }
        return vm;
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[VE]) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (F32) w[j] = __float_as_uint(x[j]);
            else w[j] = f32x2_to_bf16x2(x[2 * j], x[2 * j + 1]);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // The largest value of a whole vector.
    static __device__ __forceinline__ float most(const uint4 v) {
        if constexpr (F32) {
            return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
        } else {
            const uint32_t m2 = max_bf16x2(max_bf16x2(v.x, v.y), max_bf16x2(v.z, v.w));
            return fmaxf(bf16lo_to_f32(m2), bf16hi_to_f32(m2));
        }
    }
    // The values of a whole vector raised to FastSums' floor; returns the largest before that.
    static __device__ __forceinline__ float unpack_fast(const uint4 v, float (&x)[VE]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        if constexpr (F32) {
            unpack(v, x);
#pragma unroll
            for (int j = 0; j < VE; ++j) x[j] = fmaxf(x[j], -1e38f);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t u = max_bf16x2(w[j], 0xFE96FE96u);  // -1e38 in bf16
                x[2 * j] = bf16lo_to_f32(u);
                x[2 * j + 1] = bf16hi_to_f32(u);
            }
        }
        return most(v);
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
};

// Adds a vector to sums of any values.
template <int VE>
__device__ __forceinline__ void add_any(Sums &s, const float (&x)[VE]) {
    float vm = x[0];
#pragma unroll
    for (int j = 1; j < VE; ++j) vm = fmaxf(vm, x[j]);
    if (vm > s.m) {
        const float d = fmaxf(s.m - vm, kLowest), c = ex2(d * kLog2e);
        s.t = c * (s.t + d * s.l);
        s.l *= c;
        s.m = vm;
    }
#pragma unroll
    for (int j = 0; j < VE; ++j) {
        const float d = fmaxf(x[j] - s.m, kLowest), e = ex2(d * kLog2e);
        s.l += e;
        s.t = fmaf(d, e, s.t);
    }
}

// The same in four instructions an element for ordinary values, |m| < 2^19:
// with L = fl(log2 e) and a reference r near m L, d = x L - r (one rounding),
// l = sum 2^d, t = sum d 2^d.  The reference only has to keep 2^d in range: it
// moves when a value passes it by 2^kSlack, so that the lanes of a warp hardly
// ever do (with the maximum itself as the reference some lane of 32 does at
// four of five vectors).  sums() brings it to m.  -inf counts as -1e38, and
// neither it nor any masked value below -2^19 becomes the reference; their
// weights are 0 unless the row has nothing else, which add_any then sums.
struct FastSums {
    static constexpr float kSlack = 5.0f;
    static constexpr float kHuge = 524288.0f;
    float m = -INFINITY, limit = -kHuge, r = 0.0f, l = 0.0f, t = 0.0f;  // below -kHuge nothing is a reference

    // x: values of at least kFloor (-inf raised to it); vm: the largest before that.
    template <int VE>
    __device__ __forceinline__ void add(const float (&x)[VE], float vm) {
        if (vm > limit) {
            const float rn = vm * kLog2e;
            const float d = limit == -kHuge ? kLowest : fmaxf(r - rn, kLowest), c = ex2(d);
            t = c * (t + d * l);
            l *= c;
            r = rn;
            limit = vm + kSlack / kLog2e;
        }
        m = fmaxf(m, vm);
#pragma unroll
        for (int j = 0; j < VE; ++j) {
            const float d = fmaf(x[j], kLog2e, -r), e = ex2(d);
            l += e;
            t = fmaf(d, e, t);
        }
    }
    __device__ __forceinline__ bool ordinary() const { return m == -INFINITY || fabsf(m) < kHuge; }
    __device__ __forceinline__ Sums sums() const {
        if (m == -INFINITY) return Sums{m, 0.0f, 0.0f};
        const float d0 = fmaf(m, kLog2e, -r), c = ex2(-d0);
        return Sums{m, c * l, c * (t - d0 * l) * (1.0f / kLog2e)};
    }
};

template <int TH>
struct LpShared {
    static constexpr int kWarps = TH / 32;
    float vals[kLpCandidates + kLogprobsMaxTop];
    int32_t ids[kLpCandidates + kLogprobsMaxTop];
    float piece_max[kLpPieces][TH];
    int32_t flagged[kLpPieces * TH];  // piece << 16 | thread
    Sums warp[kWarps];
    uint32_t best_keys[32];
    float best[kWarps];
    int32_t counts[kWarps];
    int32_t n_flagged, n;
    // what the CTAs of the cluster hand to the first
    Sums part[kLpMaxSplit];
    float part_vals[kLpMaxSplit * kLogprobsMaxTop];
    int32_t part_ids[kLpMaxSplit * kLogprobsMaxTop];
};

__device__ __forceinline__ bool better(float x, int32_t i, float y, int32_t j) { return x > y || (x == y && i < j); }

// The first `top` of the n candidates (value, id >= 0) in order: emit(rank, i);
// those below `least` are known not to be among them.
template <int TH, class Emit>
__device__ __forceinline__ void rank_candidates(const float *vals, const int32_t *ids, int n, int top, float least,
                                                Emit emit) {
    const int lane = threadIdx.x & 31;
    for (int i = threadIdx.x >> 5; i < n; i += TH / 32) {  // a warp per candidate
        const float x = vals[i];
        const int32_t id = ids[i];
        if (id < 0 || x < least) continue;
        int before = 0;
        for (int j = lane; j < n; j += 32) before += ids[j] >= 0 && better(vals[j], ids[j], x, id) ? 1 : 0;
        const int rank = __reduce_add_sync(0xffffffffu, before);
        if (lane == 0 && rank < top) emit(rank, i);
    }
}

// A thread's vectors in pieces, whose maxima are kept: `per` of them, the
// first `size` in piece 0, and so on.
template <int TH>
struct Pieces {
    int per, size;
    __device__ __forceinline__ explicit Pieces(int vecs) {
        per = (vecs + TH - 1) / TH;
        size = max(1, ((per + kLpPieces - 1) / kLpPieces + kFlight - 1) / kFlight * kFlight);  // whole rounds of loads
    }
};

// The candidates of vectors [v0, v1) for its first `top` elements, in sh.vals
// and sh.ids; returns how many.  m: the maximum of this thread's vectors;
// sh.piece_max has its pieces'.
template <bool F32, int TH>
__device__ int find_candidates(const Row<F32> &row, int v0, int v1, int top, float m, LpShared<TH> &sh) {
    constexpr int kBest = 1024 / TH;  // of each warp's maxima: 32 in all
    constexpr int VE = Row<F32>::VE;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // ---- a bound at or below the top-th largest of the threads' maxima, by the upper half of its key (bf16 has no
    // more): the top-th largest of the kBest largest of each warp, which every warp finds for itself
    uint32_t left = order_key(m);
#pragma unroll
    for (int i = 0; i < kBest; ++i) {
        const uint32_t best = __reduce_max_sync(0xffffffffu, left);
        const uint32_t holders = __ballot_sync(0xffffffffu, left == best);
        if (lane == __ffs(holders) - 1) {
            sh.best_keys[warp * kBest + i] = best;
            left = 0;
        }
    }
    __syncthreads();
    uint32_t bound;
    {
        const uint32_t mine = sh.best_keys[lane];
        int above = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const uint32_t other = __shfl_sync(0xffffffffu, mine, i);
            above += other > mine || (other == mine && i < lane) ? 1 : 0;
        }
        bound = __shfl_sync(0xffffffffu, mine, __ffs(__ballot_sync(0xffffffffu, above == top - 1)) - 1) & 0xFFFF0000u;
    }
    const Pieces<TH> pieces(v1 - v0);
    // ---- what the pieces that reach it hold; strict: above it only
    uint32_t unit = 0x10000u;  // what the bound resolves
    for (int strict = 0; strict < 2; ++strict) {
        if (tid == 0) sh.n_flagged = sh.n = 0;
        __syncthreads();
        const uint32_t least = strict ? bound + unit : bound;
        if (order_key(m) >= least)
            for (int i = 0; i * pieces.size < pieces.per; ++i)
                if (order_key(sh.piece_max[i][tid]) >= least) sh.flagged[atomicAdd(&sh.n_flagged, 1)] = tid | i << 16;
        __syncthreads();
        const int todo = sh.n_flagged * pieces.size;
        for (int p = tid; p < todo; p += TH) {
            const uint32_t f = p / static_cast<uint32_t>(pieces.size), at = p - f * pieces.size;
            const int owner = sh.flagged[f] & 0xFFFF, i = (sh.flagged[f] >> 16) * pieces.size + static_cast<int>(at);
            const int v = v0 + owner + i * TH;
            if (i >= pieces.per || v >= v1) continue;
            float x[VE];
            row.load(v, x);
            float vm = x[0];
#pragma unroll
            for (int j = 1; j < VE; ++j) vm = fmaxf(vm, x[j]);
            if (order_key(vm) < least) continue;
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                const int64_t e = row.element(v, j);
                if (order_key(x[j]) >= least && e >= 0 && e < row.vocab) {
                    const int n = atomicAdd(&sh.n, 1);
                    if (n < kLpCandidates) {
                        sh.vals[n] = x[j];
                        sh.ids[n] = static_cast<int32_t>(e);
                    }
                }
            }
        }
        __syncthreads();
        if (sh.n <= kLpCandidates) {
            const int n = sh.n;
            if (!strict || n >= top) return n;
            // ---- and of the many equals at the bound the lowest indices
            int have = n;
            for (int v = v0; v < v1 && have < top; v += TH) {
                float x[VE];
                uint32_t eq = 0;
                if (v + tid < v1) {
                    row.load(v + tid, x);
#pragma unroll
                    for (int j = 0; j < VE; ++j) {
                        const int64_t e = row.element(v + tid, j);
                        // equal in what the bound resolves of the key
                        if (order_key(x[j]) - bound < unit && e >= 0 && e < row.vocab) eq |= 1u << j;
                    }
                }
                const int mine = __popc(eq);
                int upto = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += y;
                }
                if (lane == 31) sh.counts[warp] = upto;
                __syncthreads();
                int at = have + upto - mine, all = 0;
                for (int w = 0; w < TH / 32; ++w) {
                    if (w < warp) at += sh.counts[w];
                    all += sh.counts[w];
                }
#pragma unroll
                for (int j = 0; j < VE; ++j)
                    if ((eq >> j) & 1) {
                        if (at < top) {
                            sh.vals[at] = x[j];
                            sh.ids[at] = static_cast<int32_t>(row.element(v + tid, j));
                        }
                        ++at;
                    }
                have += all;
                __syncthreads();
            }
            return min(have, top);
        }
        __syncthreads();
        if (F32 && !strict) {  // values of one upper half are not equals: the rest of the bound, by counting
            const uint32_t key = order_key(m);
            for (int bit = 15; bit >= 0; --bit) {
                const uint32_t cand = bound | (1u << bit);
                if (__syncthreads_count(key >= cand) >= top) bound = cand;
            }
            unit = 1;
        }
    }
    // ---- more values above the bound than fit: take the best one after the last, `top` times
    float last_x = INFINITY;
    int32_t last_i = -1;
    int n = 0;
    for (; n < top; ++n) {
        float bx = -INFINITY;
        int32_t bi = 0x7fffffff;
        for (int v = v0 + tid; v < v1; v += TH) {
            float x[VE];
            row.load(v, x);
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                const int64_t e = row.element(v, j);
                if (e < 0 || e >= row.vocab) continue;
                const int32_t i = static_cast<int32_t>(e);
                if (better(last_x, last_i, x[j], i) && better(x[j], i, bx, bi)) bx = x[j], bi = i;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float y = __shfl_xor_sync(0xffffffffu, bx, o);
            const int32_t i = __shfl_xor_sync(0xffffffffu, bi, o);
            if (better(y, i, bx, bi)) bx = y, bi = i;
        }
        __syncthreads();
        if (lane == 0) sh.best[warp] = bx, sh.counts[warp] = bi;
        __syncthreads();
        for (int w = 0; w < TH / 32; ++w)
            if (better(sh.best[w], sh.counts[w], bx, bi)) bx = sh.best[w], bi = sh.counts[w];
        if (bi == 0x7fffffff) break;  // none left (NaN among the values)
        if (tid == 0) sh.vals[n] = bx, sh.ids[n] = bi;
        last_x = bx, last_i = bi;
    }
    __syncthreads();
    return n;
}

// The sums of this thread's vectors v0 + tid, + TH, ... below v1, and
// with `pieces` the maxima of its pieces.
template <bool F32, int TH>
__device__ __forceinline__ Sums read_row(const Row<F32> &row, int v0, int v1, int tid, const Pieces<TH> &pieces,
                                         bool keep, LpShared<TH> &sh) {
    constexpr int VE = Row<F32>::VE;
    FastSums fast;
    float max_all = -INFINITY;
    int piece = 0, end = pieces.size;  // of the piece, in vectors of this thread
    auto close = [&]() {
        if (keep) sh.piece_max[piece][tid] = fast.m;
        ++piece;
        end += pieces.size;
        max_all = fmaxf(max_all, fast.m);
        fast.m = -INFINITY;
    };
    int v = v0 + tid, i = 0;
    const int v_whole = v1 > v0 && !row.whole(v1 - 1) ? v1 - 1 : v1;
    // whole rounds of loads, but for a ragged start
    for (; v + (kFlight - 1) * TH < v_whole; v += kFlight * TH, i += kFlight) {
        if (i == end) close();
        uint4 w[kFlight];
        const bool ragged = !row.whole(v);
#pragma unroll
        for (int j = 0; j < kFlight; ++j)
            if (j > 0 || !ragged) w[j] = ld_v4(row.base + static_cast<int64_t>(v + j * TH) * 16);
        if (ragged) {
            float x[VE];
            row.load(v, x);
            w[0] = Row<F32>::pack(x);
        }
#pragma unroll
        for (int j = 0; j < kFlight; ++j) {
            float x[VE];
            const float vm = Row<F32>::unpack_fast(w[j], x);
            fast.add<VE>(x, vm);
        }
    }
    for (; v < v1; v += TH, ++i) {
        if (i == end) close();
        float x[VE];
        const float vm = row.load_fast(v, x);
        fast.add<VE>(x, vm);
    }
    close();
    if (keep)  // pieces this thread has nothing of
        for (; piece * pieces.size < pieces.per; ++piece) sh.piece_max[piece][tid] = -INFINITY;
    fast.m = max_all;
    if (fast.ordinary()) return fast.sums();
    Sums s{-INFINITY, 0.0f, 0.0f};  // a maximum that the fast sums cannot hold
    for (v = v0 + tid; v < v1; v += TH) {
        float x[VE];
        row.load(v, x);
        add_any<VE>(s, x);
    }
    return s;
}

// What a row gives besides its top.  `x`: the target's logit.
__device__ __forceinline__ void store_row(const LogprobArgs &a, int64_t r, const Sums &all, int64_t target, float x) {
    const bool any = all.m != -INFINITY;
    const float lz = any ? logf(all.l) : 0.0f;
    if (target >= a.vocab) atomicOr(&g_lp_err, ERRBIT_INDEX);
    a.logprobs[r] = target < 0 || target >= a.vocab ? 0.0f : any ? (x - all.m) - lz : -INFINITY;
    a.entropy[r] = any ? lz - all.t / all.l : 0.0f;
}

template <bool F32, int TH>
__global__ void __launch_bounds__(TH, 1024 / TH) logprobs_kernel(const LogprobArgs a, int splits) {
    __shared__ LpShared<TH> sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t r = blockIdx.x / splits;
    const int part = static_cast<int>(blockIdx.x - r * splits);  // rank in the cluster
    const int top = static_cast<int>(a.top);
    if (splits > 1) cluster_arrive();  // the first CTA's shared memory is there once all have
    pdl_wait();
    const Row<F32> row(row_start<F32>(a, r), a.vocab);
    const int v0 = static_cast<int>(static_cast<int64_t>(row.vecs) * part / splits);
    const int v1 = static_cast<int>(static_cast<int64_t>(row.vecs) * (part + 1) / splits);

    int64_t target = -1;
    float x_target = 0.0f;
    if (part == 0 && tid == 0) {
        target = a.targets[r];
        if (target >= 0 && target < a.vocab) x_target = row.at(target);
    }
    const Sums s = read_row<F32, TH>(row, v0, v1, tid, Pieces<TH>(v1 - v0), top > 0, sh);
    const Sums w = warp_merge(s);
    if (lane == 0) sh.warp[warp] = w;
    int n = 0;
    if (top > 0) n = find_candidates<F32, TH>(row, v0, v1, top, s.m, sh);
    else __syncthreads();
    Sums all = warp_merge(sh.warp[lane % (TH / 32)], TH / 32);

    const float *vals = sh.vals;
    const int32_t *ids = sh.ids;
    float least = -INFINITY;
    if (splits > 1) {
        // the part's sums and first `top` go to the first CTA's shared memory
        const uint32_t to = 0;
        cluster_wait();
        if (tid == 0) {
            const uint32_t p = dsmem_map(smem_u32(&sh.part[part]), to);
            dsmem_st_f32(p, all.m);
            dsmem_st_f32(p + 4, all.l);
            dsmem_st_f32(p + 8, all.t);
        }
        if (top > 0) {
            const uint32_t pv = dsmem_map(smem_u32(&sh.part_vals[part * top]), to);
            const uint32_t pi = dsmem_map(smem_u32(&sh.part_ids[part * top]), to);
            for (int i = tid; i < top; i += TH)
                if (i >= n) dsmem_st_f32(pi + 4 * i, __int_as_float(-1));
            rank_candidates<TH>(sh.vals, sh.ids, n, top, least, [&](int rank, int i) {
                dsmem_st_f32(pv + 4 * rank, sh.vals[i]);
                dsmem_st_f32(pi + 4 * rank, __int_as_float(sh.ids[i]));
            });
        }
        __syncwarp();
        cluster_sync_all();
        if (part != 0) return;
        const Sums none{-INFINITY, 0.0f, 0.0f};
        all = warp_merge(lane < splits ? sh.part[lane] : none);
        vals = sh.part_vals;
        ids = sh.part_ids;
        n = splits * top;
        // a part with `top` candidates has them all at or above its last
        if (lane < splits && top > 0 && ids[lane * top + top - 1] >= 0) least = vals[lane * top + top - 1];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) least = fmaxf(least, __shfl_xor_sync(0xffffffffu, least, o));
    }

    const bool any = all.m != -INFINITY;
    const float lz = any ? logf(all.l) : 0.0f;
    if (tid == 0) store_row(a, r, all, target, x_target);
    if (top > 0) {
        int32_t *out_ids = a.top_ids + r * top;
        float *out = a.top_logprobs + r * top;
        int live = 0;  // candidates there are; fewer than top only where NaN took the others' places
        for (int i = lane; i < n; i += 32) live += ids[i] >= 0 ? 1 : 0;
        live = __reduce_add_sync(0xffffffffu, live);
        for (int i = live + tid; i < top; i += TH) {
            out_ids[i] = -1;
            out[i] = -INFINITY;
        }
        rank_candidates<TH>(vals, ids, n, top, least, [&](int rank, int i) {
            out_ids[rank] = ids[i];
            out[rank] = any ? (vals[i] - all.m) - lz : -INFINITY;
        });
    }
}

// CTAs per row: as many as keep the GPU's two CTAs of 512 threads per SM busy
// in one wave, while each still has a vector per thread.
int pick_row_split(const LogprobArgs &a) {
    const int64_t vecs = a.vocab / (a.f32 ? 4 : 8);
    int s = 1;
    while (s < kLpMaxSplit && 2 * s * a.rows <= 2 * static_cast<int64_t>(device_sm_count()) && vecs / (2 * s) >= 512)
        s *= 2;
    return s;
}

template <bool F32, int TH>
cudaError_t launch_rows(const LogprobArgs &a, int splits, cudaStream_t stream) {
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
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<F32, TH>, a, splits);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs &a, cudaStream_t stream) {
    // Threads a CTA.  Few rows: 512, more of a row in flight (one row of 152064 bf16, top 20: 11.2 us, 13.8 with 256;
    // 300 rows: 23 us and 26, but of 32003 9.8 us and 9.3).  Many: 256, so that four CTAs of an SM read while one
    // looks for its top (2048 rows: 123 us, 136 with 512, 129 with 128).  Many short ones, whose tops weigh more:
    // 128 and eight CTAs (4096 rows of 32003, top 20: 75 us, 90 with 256; of 65536 120 and 121; 3000 of 100003 127
    // and 123); also where those take all the rows at once and four do not (1000 rows of 152064: 63 us, 69 with 256).
    // All of bf16; fp32 rows, of twice the vectors, go by the same numbers of vectors (1024 rows of 152064: 107 us for
    // 92 of bytes).
    const int splits = pick_row_split(a);
    const int64_t sms = device_sm_count(), vecs = a.vocab / (a.f32 ? 4 : 8);
    if (splits > 1 || (a.rows <= 2 * sms && vecs >= 2 * kFlight * 512))
        return a.f32 ? launch_rows<true, 512>(a, splits, stream) : launch_rows<false, 512>(a, splits, stream);
    if (a.rows > 4 * sms && (vecs <= 8192 || a.rows <= 8 * sms))
        return a.f32 ? launch_rows<true, 128>(a, 1, stream) : launch_rows<false, 128>(a, 1, stream);
    return a.f32 ? launch_rows<true, 256>(a, 1, stream) : launch_rows<false, 256>(a, 1, stream);
}

uint32_t take_logprobs_error() {
    uint32_t v = 0;
    if (cudaMemcpyFromSymbol(&v, g_lp_err, sizeof v) != cudaSuccess) return 0xFFFFFFFFu;
    const uint32_t zero = 0;
    cudaMemcpyToSymbol(g_lp_err, &zero, sizeof zero);
    return v;
}

}  // namespace fp8bs
