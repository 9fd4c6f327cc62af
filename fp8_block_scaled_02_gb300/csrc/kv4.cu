// kv4.cu -- a paged KV cache held in 4 bits: append, gather, attention.
//
// The value of an element is code * scale * s: an e2m1 code, an e4m3 scale
// per 16 consecutive elements of a head vector, one fp32 s per layer (for K
// and for V).  A head vector of D elements takes D / 2 + D / 16 bytes, 0.28
// of bf16 and 0.56 of the FP8 cache.
//
//   append: sc = e4m3(amax / (6 s)), code = e2m1(x / (s sc)), every quotient
//           and product one fp32 rounding, both conversions to nearest even
//           and saturating; sc = 0 stores zero codes.
//   gather: bf16(code * sc * s); code * sc has 6 significant bits and is
//           exact in f16, so the value is rounded by the product with s and
//           by bf16 only.
//
// A tile is 16 tokens of one kv head: codes, then scales, contiguous, so a
// whole tile is one aligned copy of 9 D bytes.
#include "serving.cuh"
#include "fp8bs.h"
#include "internal.h"

#include <cuda_fp16.h>

#include <mutex>
#include <utility>

namespace fp8bs {

namespace {

__device__ uint32_t g_kv4_err;


// ------------------------------------------------------- append and gather
// A thread has 32 consecutive elements of a head vector (two groups): 64 bytes
// of bf16, 16 of codes and 2 of scales; a warp's accesses are contiguous.  An
// element is 2 B read and 9/16 B written, or the reverse.  K and V of 8 heads of
// 128: 65536 tokens are read in 60 us (5.7 TB/s, bound by HBM; 65 with half the
// bytes a thread and a division for its place).  8191 tokens, 43 MB, stay in L2
// when the same buffers are used again: written in 8.3 us (11.6 with IEEE
// divisions), read back in 7.1.  With the caches flushed, under a profiler, 12.7
// and 10.8 us for 6.3 us of bytes: one wave, a third of it launch and first loads.
constexpr int kCopyThreads = 256;

__device__ __forceinline__ void st_v8(void *p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// The thread's pair of groups: token, and pair within the token's row.
struct CopyItem {
    int64_t token;
    uint32_t pair;
};

// The thread's item: a block's items are contiguous.  `inverse` = ceil(2^64 / per_row)
// divides every item number below 2^47 exactly by a multiplication.
__device__ __forceinline__ CopyItem copy_item(uint64_t inverse, uint32_t per_row) {
    const uint64_t i = static_cast<uint64_t>(blockIdx.x) * kCopyThreads + threadIdx.x, t = __umul64hi(i, inverse);
    return CopyItem{static_cast<int64_t>(t), static_cast<uint32_t>(i - t * per_row)};
}

// Where the codes and the scales of a pair of groups of a slot are.
template <int D>
__device__ __forceinline__ uint8_t *slot_codes(uint8_t *cache, uint32_t slot, uint32_t h, uint32_t pair, uint32_t kv_heads,
                                               uint32_t tiles_per_page, uint8_t **scales) {
    const uint32_t tile = slot / kKv4Tile, row = slot % kKv4Tile, blk = tile / tiles_per_page;
    uint8_t *t = cache + ((static_cast<int64_t>(blk) * kv_heads + h) * tiles_per_page + (tile - blk * tiles_per_page)) *
                             kv4_tile_bytes(D);
    *scales = t + 8 * D + row * (D / 16) + 2 * pair;
    return t + row * (D / 2) + 16 * pair;
}

// (lo / d, hi / d) by Markstein's correction (P. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", IBM J. Res.
// Dev. 34(1), 1990): q0 = RN(x y), r = x - d q0 exactly, q = RN(q0 + r y) with
// y = RN(1/d), two values a packed fma; the sign is x's also where q is 0.
// With d in [2^-92, 2^92] and |x| y < 1e30 no step leaves the normal range
// where it matters, and the e2m1 code of q is that of the IEEE quotient for
// every divisor mantissa (tests/csrc/quotient_e2m1.c).
__device__ __forceinline__ void quotient2(float lo, float hi, uint64_t nd2, uint64_t y2, float &qlo, float &qhi) {
    const uint64_t negzero2 = 0x8000000080000000ull;
    uint64_t x2, q0, r, q;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x2) : "f"(lo), "f"(hi));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q0) : "l"(x2), "l"(y2), "l"(negzero2));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(nd2), "l"(q0), "l"(x2));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q) : "l"(r), "l"(y2), "l"(q0));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(qlo), "=f"(qhi) : "l"(q));
    qlo = copysignf(qlo, lo);
    qhi = copysignf(qhi, hi);
}

// 16 bf16 values (8 words) -> their group's scale code and e2m1 codes.
__device__ __forceinline__ uint32_t encode_group(const uint32_t *u, float s, float six_s, uint2 &codes) {
    uint32_t mx = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) mx = max_u16x2(mx, u[j] & 0x7FFF7FFFu);
    const float amax = __uint_as_float(max(mx & 0xFFFFu, mx >> 16) << 16);
    const uint32_t sc = f32x2_to_e4m3x2(amax / six_s, 0.0f) & 0xFFu;
    const float den = f16x2_to_f32x2(e4m3x2_to_f16x2(sc)).x * s;
    codes = make_uint2(0, 0);
    float q[2][8];
    if (den >= 0x1p-92f && den <= 0x1p92f && amax < 1e30f * den) {
        const float y = __frcp_rn(den);
        uint64_t nd2, y2;
        asm("mov.b64 %0, {%1, %1};" : "=l"(nd2) : "f"(-den));
        asm("mov.b64 %0, {%1, %1};" : "=l"(y2) : "f"(y));
#pragma unroll
        for (int j = 0; j < 8; ++j)
            quotient2(bf16lo_to_f32(u[j]), bf16hi_to_f32(u[j]), nd2, y2, q[j >> 2][2 * (j & 3)], q[j >> 2][2 * (j & 3) + 1]);
    } else if (den > 0.0f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            q[j >> 2][2 * (j & 3)] = bf16lo_to_f32(u[j]) / den;
            q[j >> 2][2 * (j & 3) + 1] = bf16hi_to_f32(u[j]) / den;
        }
    } else {
        return sc;
    }
    codes = make_uint2(f32x8_to_e2m1x8(q[0]), f32x8_to_e2m1x8(q[1]));
    return sc;
}

// blockIdx.y selects K or V; 64-byte pieces of x are 32-byte aligned if `wide`.
template <int D>
__global__ void __launch_bounds__(kCopyThreads) kv4_append_kernel(Kv4CopyArgs a, uint64_t inverse, bool wide) {
    const bool is_v = blockIdx.y != 0;
    const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(is_v ? a.v : a.k);
    const int64_t stride = is_v ? a.v_stride : a.k_stride;
    uint8_t *cache = is_v ? a.v_cache : a.k_cache;
    const uint32_t kv_heads = static_cast<uint32_t>(a.kv_heads), per_row = kv_heads * (D / 32);
    const uint32_t tpp = static_cast<uint32_t>(a.page_size / kKv4Tile);
    const CopyItem it = copy_item(inverse, per_row);
    pdl_launch_dependents();
    pdl_wait();
    if (it.token >= a.tokens) return;
    const int64_t slot = a.slots[it.token];
    if (slot < 0 || slot >= a.num_slots) {
        if (slot != -1 && it.pair == 0 && !is_v) atomicOr(&g_kv4_err, ERRBIT_INDEX);
        return;
    }
    const __nv_bfloat16 *src = x + it.token * stride + it.pair * 32;
    uint32_t u[2][8];
    if (wide) {
        ld_v8(src, u[0]);
        ld_v8(src + 16, u[1]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 w = ld_v4(src + 8 * i);
            uint32_t *d = u[i / 2] + 4 * (i & 1);
            d[0] = w.x, d[1] = w.y, d[2] = w.z, d[3] = w.w;
        }
    }
    const float s = *(is_v ? a.v_scale : a.k_scale), six_s = 6.0f * s;
    uint2 c0, c1;
    const uint32_t s0 = encode_group(u[0], s, six_s, c0), s1 = encode_group(u[1], s, six_s, c1);
    uint8_t *scales;
    uint8_t *codes = slot_codes<D>(cache, static_cast<uint32_t>(slot), it.pair / (D / 32), it.pair % (D / 32), kv_heads,
                                   tpp, &scales);
    *reinterpret_cast<uint4 *>(codes) = make_uint4(c0.x, c0.y, c1.x, c1.y);
    *reinterpret_cast<uint16_t *>(scales) = static_cast<uint16_t>(s0 | (s1 << 8));
}

template <int D>
__global__ void __launch_bounds__(kCopyThreads) kv4_gather_kernel(Kv4CopyArgs a, uint64_t inverse, bool wide) {
    const bool is_v = blockIdx.y != 0;
    uint8_t *cache = is_v ? a.v_cache : a.k_cache;
    const uint32_t kv_heads = static_cast<uint32_t>(a.kv_heads), per_row = kv_heads * (D / 32);
    const uint32_t tpp = static_cast<uint32_t>(a.page_size / kKv4Tile);
    const CopyItem it = copy_item(inverse, per_row);
    pdl_launch_dependents();
    pdl_wait();
    if (it.token >= a.tokens) return;
    const int64_t slot = a.slots[it.token];
    uint32_t r[2][8] = {};
    if (slot < 0 || slot >= a.num_slots) {
        if (slot != -1 && it.pair == 0 && !is_v) atomicOr(&g_kv4_err, ERRBIT_INDEX);
    } else {
        uint8_t *scales;
        const uint8_t *codes = slot_codes<D>(cache, static_cast<uint32_t>(slot), it.pair / (D / 32), it.pair % (D / 32),
                                             kv_heads, tpp, &scales);
        const uint4 c = ld_v4(codes);
        const uint32_t sc = *reinterpret_cast<const uint16_t *>(scales);
        const float s = *(is_v ? a.v_scale : a.k_scale);
        const uint32_t s2 = e4m3x2_to_f16x2(sc), w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t h[4];
            e2m1x8_to_f16x2x4(w[i], h);
            const uint32_t scale2 = __byte_perm(s2, s2, i < 2 ? 0x1010 : 0x3232);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 v = f16x2_to_f32x2(mul_f16x2(h[j], scale2));
                r[i / 2][4 * (i & 1) + j] = f32x2_to_bf16x2(v.x * s, v.y * s);
            }
        }
    }
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(is_v ? a.v_out : a.k_out) +
                         (it.token * per_row + it.pair) * 32;
    if (wide) {
        st_v8(out, r[0]);
        st_v8(out + 16, r[1]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t *d = r[i / 2] + 4 * (i & 1);
            *reinterpret_cast<uint4 *>(out + 8 * i) = make_uint4(d[0], d[1], d[2], d[3]);
        }
    }
}

// --------------------------------------------------------------- attention
// Query token i of the n_q tokens of a sequence of len keys stands at
// position len - n_q + i and sees the keys up to its own (of those, the
// newest `window`, if there is one).  With the log2-domain scores
// s = sm_scale log2(e) q.k, a running maximum m and p = 2^(s - m + 14):
//   l = sum p,  o = sum p v,  out = o / l,  lse = ln 2 (m - 14 + log2 l);
// the 2^14 keeps weights down to 2^-39 of the largest out of f16's zero.
//
// Work: a segment is one (sequence, kv head, tile of R = 8 NT query rows); a
// row is a (query token, head of the group) pair, so a K/V byte is read once
// for R rows.  A unit is 32 keys of a segment.  The CTAs cut the line of all
// units of all segments into equal shares (every CTA finds its own from a
// prefix sum of the lengths), so a ragged batch fills the GPU evenly and a
// single long sequence is spread over all of it.  A segment that crosses a
// share's end leaves partial (m, l, o) records in the workspace; the CTA that
// leaves the last one joins them, in the order of the CTAs.
//
// A CTA is a producer warp and W consumer warps around a ring of S units.  The
// producer walks the share and copies units in pairs, by one gather of four
// tiles for K and one for V wherever they lie (a tile is a row of the cache's
// map); a warp issues a bulk copy in some 235 clocks, and with copies of one or
// two tiles, as pages of 16 allow, it did not keep up (16 x 32768 keys of 8
// heads: 143 us, 134 with the gather; 121 with the steps after it).
// It is pieces ahead of the consumers, so table lookups and copies cost no
// time between them.  The consumers of a piece take its units in turn and join
// their (m, l, o) in shared memory; a segment of one unit is one warp's alone,
// beside others.  Per unit:
//   S^T[32 keys, R rows] = K q^T with f16 mma.sync m16n8k16.  The order of
//   the contraction is free: lane t of a quad takes elements 32 t .. 32 t + 31
//   of a key (D = 128), so its codes are one 16-byte load; codes convert to
//   f16 exactly and are multiplied with their f16 scale exactly.
//   O^T[D, R] += V^T P^T: row group g of the product is 16 consecutive
//   elements, column pair t the keys kv4_row(t, j), so a lane's codes are 8
//   bytes of each of four keys; pair_f16 interleaves two keys' values and
//   multiplies with their scales.  P^T comes from the S^T fragments by
//   movmatrix, because key m of S^T is key m of the product.
// Bytes would take 89 us at 16 x 32768 keys of 8 heads (groups of 4) at the
// measured copy rate; it takes 120 us, 5.0 TB/s.  Neither HBM (a cache that fits
// L2 saved 3% when tried) nor a pipe is at its limit: on a ragged batch ALU 44%,
// FMA 25%, tensor 21%, issue slots 60%.  A unit is a chain of dependent steps
// (copy, conversions, product, maximum, exponentials, transpose, product) and 18
// warps an SM do not cover its latency (stalled warps per issue: long scoreboard
// 1.25, fixed latency 1.13, not selected 1.05), so every instruction of the chain
// counts: without the conversions it took 107 us of 131 then.  An eighth of the
// SMs' time is idle, at the start and where the shares end.
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kPShift = 14.0f;
constexpr int kMaxSms = 160;  // CTAs the workspace has records for: two per SM of 16 rows, or one of 32
constexpr int kMinShare = 8;  // a CTA's share at least, in steps of the line

// A producer warp, W consumer warps and a ring of S units per CTA, kRes CTAs
// per SM: measured at D = 128.  D = 64, with stages and accumulators half as
// large, takes the same (16 x 32768: 92 us for 44 us of bytes).
template <int D, int NT>
struct AttnCfg {
    static constexpr int kRes = NT <= 2 ? 2 : 1;
    static constexpr int W = NT == 1 ? 8 : NT == 2 ? 5 : 7;
    static constexpr int UT = 2;                    // tiles per unit
    static constexpr int kKeys = UT * kKv4Tile;     // keys per unit
    // A stage belongs to one consumer warp: unit i of a CTA is warp i % W's and
    // in stage i % S, with W a divisor of S.  Copies land in any order, and a
    // warp that waited for the next phase of a stage before the last one is
    // complete would take the phase before that for it.  Units are copied in
    // pairs, so S is even.
    static constexpr int S = 2 * W;
    static_assert(S % W == 0 && S % 2 == 0, "a stage's units are one warp's");
    static constexpr int kThreads = (W + 1) * 32;
    static constexpr int R = 8 * NT;
    static constexpr int T = 9 * D;                 // bytes of a tile
    static constexpr int kStageBytes = 2 * UT * T;
    // What a segment costs besides its units (its q, the merge of the warps, its
    // output), in units, which cost more with more rows; shares are equal in
    // units + kSegCost a segment (48 ragged sequences: 83 us with 6, 72 with 12, 70 with 20).
    static constexpr int kSegCost = NT == 1 ? 20 : 12;
    static constexpr int kRecFloats = R * (D + 2);  // m[R], l[R], o[R][D]
    static constexpr int kSmemBytes = S * kStageBytes + W * kRecFloats * 4 + S * (4 + 4 + 4);
    static_assert(kSmemBytes * kRes <= 226 * 1024, "shared memory per SM");
};

// One sequence's share of the line of units.
struct SeqWork {
    int32_t len, q0, n_q;
    int32_t tile0, tiles;  // first tile any row sees, end of the last
    int32_t units, row_tiles;
    uint32_t err;
    __device__ __forceinline__ int64_t cost(int seg_cost, int hkv) const {
        return (static_cast<int64_t>(units) + seg_cost) * hkv * row_tiles;
    }
};

template <int R, int UT>
__device__ __forceinline__ SeqWork seq_work(const Kv4AttnArgs &a, int b, int group) {
    SeqWork w;
    w.err = 0;
    w.q0 = b;
    w.n_q = 1;
    if (a.cu_q) {
        const int64_t q0 = a.cu_q[b], n = static_cast<int64_t>(a.cu_q[b + 1]) - q0;
        if (q0 < 0 || n < 0 || n > a.max_q || q0 + n > a.tokens) {
            w.err = ERRBIT_INDEX;
            w.n_q = 0;
        } else {
            w.n_q = static_cast<int32_t>(n);
        }
        w.q0 = static_cast<int32_t>(q0);
    }
    const int32_t len = a.seq_lens[b], cap = static_cast<int32_t>(a.max_seq_len);
    if (len < 0 || len > cap) w.err = ERRBIT_INDEX;
    w.len = min(max(len, 0), cap);
    const int64_t lo = a.window > 0 ? static_cast<int64_t>(w.len) - w.n_q - a.window + 1 : 0;
    w.tiles = (w.len + kKv4Tile - 1) / kKv4Tile;
    w.tile0 = lo > 0 ? static_cast<int32_t>(lo / kKv4Tile) : 0;
    w.units = max(1, (w.tiles - w.tile0 + UT - 1) / UT);
    w.row_tiles = (w.n_q * group + R - 1) / R;
    return w;
}

// a / b of non-negative numbers, by the 32-bit division where they fit.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// A CTA's walk along its share: pieces of segments, in order.  On the line a
// segment is kSegCost steps and then its units.
template <int R, int UT, int kSegCost>
struct Walk {
    SeqWork w;
    int64_t left;  // steps left in the share
    int b, at;     // next step of the segment
    int kvh, row_tile;
    int u0, u1;    // the piece's units

    // Starts at step `p` of sequence `first`.
    __device__ __forceinline__ void start(const Kv4AttnArgs &a, int first, int64_t p, int64_t steps, int group) {
        b = first;
        left = steps;
        w = seq_work<R, UT>(a, b, group);
        const int seg_cost = w.units + kSegCost;
        const int64_t seg = quotient(p, seg_cost);
        at = static_cast<int>(p - seg * seg_cost);
        kvh = static_cast<int>(quotient(seg, w.row_tiles));
        row_tile = static_cast<int>(seg - static_cast<int64_t>(kvh) * w.row_tiles);
    }
    __device__ __forceinline__ bool next(const Kv4AttnArgs &a, int hkv, int group) {
        while (left > 0) {
            const int seg_cost = w.units + kSegCost;
            if (at >= seg_cost) {
                at = 0;
                if (++row_tile < w.row_tiles) continue;
                row_tile = 0;
                if (++kvh < hkv) continue;
                kvh = 0;
                do {  // sequences without rows have no steps
                    if (++b >= a.batch) return false;
                    w = seq_work<R, UT>(a, b, group);
                } while (w.row_tiles == 0);
                continue;
            }
            const int end = static_cast<int>(min(static_cast<int64_t>(seg_cost), at + left));
            u0 = max(0, at - kSegCost);
            u1 = end - kSegCost;
            left -= end - at;
            at = end;
            if (u1 > u0) return true;  // else the share ends before the segment's first unit
        }
        return false;
    }
};

constexpr uint32_t kNoTile = 0xffffffffu;  // a tile that is not there or left out: row -1 of the maps

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ void bar_consumers(int threads) {
    asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
}

// (a.h sa, b.h sb) for half h of a and b, from (sa, 0) and (0, sb): two
// instructions of the FMA pipe instead of a byte permute and one; the ALU pipe
// has the conversions already (128 us instead of 130 at 16 x 32768 keys of 8 heads when it came).
__device__ __forceinline__ uint32_t pair_f16(uint32_t a, uint32_t b, uint32_t sa, uint32_t sb, int h) {
    const __half2 va = *reinterpret_cast<const __half2 *>(&a), vb = *reinterpret_cast<const __half2 *>(&b);
    const __half2 x = h ? __high2half2(va) : __low2half2(va), y = h ? __high2half2(vb) : __low2half2(vb);
    const __half2 r =
        __hfma2(x, *reinterpret_cast<const __half2 *>(&sa), __hmul2(y, *reinterpret_cast<const __half2 *>(&sb)));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Over groups of `width` lanes.
template <int width>
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = width / 2; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

template <int width>
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = width / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <int E>
__device__ __forceinline__ void load_floats(const float *p, float (&v)[E]) {
    if constexpr (E == 4) {
        const float4 x = *reinterpret_cast<const float4 *>(p);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
        const float2 x = *reinterpret_cast<const float2 *>(p);
        v[0] = x.x, v[1] = x.y;
    }
}

template <int E>
__device__ __forceinline__ void load_floats_cg(const float *p, float (&v)[E]) {
    if constexpr (E == 4) {
        const float4 x = __ldcg(reinterpret_cast<const float4 *>(p));
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
        const float2 x = __ldcg(reinterpret_cast<const float2 *>(p));
        v[0] = x.x, v[1] = x.y;
    }
}

template <int E>
__device__ __forceinline__ void store_floats(float *p, const float (&v)[E]) {
    if constexpr (E == 4) *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
}

template <int E>
__device__ __forceinline__ void fma_floats(float (&o)[E], float f, const float (&v)[E]) {
#pragma unroll
    for (int d = 0; d < E; ++d) o[d] += f * v[d];
}

// Releases this CTA's earlier writes and acquires the others' to the GPU.
__device__ __forceinline__ uint32_t atomic_inc_acq_rel(uint32_t *p, uint32_t limit) {
    uint32_t before;
    asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;" : "=r"(before) : "l"(p), "r"(limit) : "memory");
    return before;
}

// Where 16 bytes of a row of a warp's o are in shared memory: the eight lanes of
// a store (two values of g, four rows two apart) and of a load meet no bank twice.
template <int D>
__device__ __forceinline__ int merge_chunk(int r, int chunk) {
    return chunk ^ (D == 128 ? (r >> 1) & 3 : ((r >> 1) & 1) | (r & 4));
}

// Key of a tile that is row m (and m + 8) of the score product, and column
// pair t, half j of the value product: neighbouring m differ in parity, so
// the 16-byte loads of eight lanes (two keys of 64 bytes) meet no bank twice.
__device__ __forceinline__ int kv4_row(int m) { return (m & 1) ? 4 + ((m >> 1) ^ 1) : m >> 1; }

template <int D, int NT>
__global__ void __launch_bounds__(AttnCfg<D, NT>::kThreads, AttnCfg<D, NT>::kRes) kv4_attn_kernel(
    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const Kv4AttnArgs a) {
    using C = AttnCfg<D, NT>;
    constexpr int W = C::W, R = C::R, T = C::T, UT = C::UT, S = C::S;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *ring = smem;                                                 // [S / 2][K tiles | V tiles of two units]
    float *merge = reinterpret_cast<float *>(ring + S * C::kStageBytes);  // [W] records
    uint64_t *full = reinterpret_cast<uint64_t *>(merge + W * C::kRecFloats);
    uint64_t *empty = full + S / 2;
    int32_t *holds = reinterpret_cast<int32_t *>(empty + S / 2);              // which tiles a stage holds, a bit each
    __shared__ int64_t s_sums[W + 1], s_p;
    __shared__ int s_b, s_first, s_parts;
    __shared__ Walk<R, UT, C::kSegCost> s_walk[W];
    __shared__ struct {
        int64_t total, ctas, lo, hi;  // of the line: its steps, the shares, this one
    } s_line;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hkv = static_cast<int>(a.kv_heads), group = static_cast<int>(a.q_heads / a.kv_heads);
    const int batch = static_cast<int>(a.batch), cta = blockIdx.x;
    uint32_t *arrived = static_cast<uint32_t *>(a.workspace);  // [2 kMaxSms], 0 between calls
    float *records = reinterpret_cast<float *>(arrived + 2 * kMaxSms);
    if (tid == 0) {
        for (int i = 0; i < S / 2; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 2);
        }
        fence_mbarrier_init();
    }
    if (tid == 32) {
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
    }
    pdl_wait();  // q, the cache and the lengths may come from the previous kernel

    // ---- this CTA's share
    const int per = (batch + C::kThreads - 1) / C::kThreads;
    const int b0 = min(batch, tid * per), b1 = min(batch, b0 + per);
    int64_t mine = 0;
    uint32_t err = 0;
    for (int b = b0; b < b1; ++b) {
        const SeqWork w = seq_work<R, UT>(a, b, group);
        err |= w.err;
        mine += w.cost(C::kSegCost, hkv);
    }
    if (err && cta == 0) atomicOr(&g_kv4_err, err);
    int64_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_sums[warp] = x;
    __syncthreads();
    int64_t total = 0, before = x - mine;
#pragma unroll
    for (int w = 0; w <= W; ++w) {
        if (w < warp) before += s_sums[w];
        total += s_sums[w];
    }
    const int64_t ctas = min(static_cast<int64_t>(gridDim.x), (total + kMinShare - 1) / kMinShare);
    if (cta >= ctas) return;
    const int64_t lo = quotient(total * cta, ctas), hi = quotient(total * (cta + 1), ctas);
    if (tid == 0) s_line.total = total, s_line.ctas = ctas, s_line.lo = lo, s_line.hi = hi;
    if (lo >= before && lo < before + mine) {
        int64_t at = before;
        for (int b = b0; b < b1; ++b) {
            const int64_t cost = seq_work<R, UT>(a, b, group).cost(C::kSegCost, hkv);
            if (lo < at + cost) {
                s_b = b;
                s_p = lo - at;
                break;
            }
            at += cost;
        }
    }
    __syncthreads();
    Walk<R, UT, C::kSegCost> walk;
    walk.start(a, s_b, s_p, hi - lo, group);

    if (warp == W) {
        // ================================================== producer
        const int tpp = static_cast<int>(a.page_size) / kKv4Tile;
        constexpr int kWindow = 32 / UT;  // units looked up together, a lane per tile
        constexpr int kPairs = S / 2;     // pairs of units in the ring
        uint32_t pairs = 0;               // pairs put into the ring before the window
        bool inside = walk.next(a, hkv, group);
        int ub = walk.u0;
        // the next window of units, over piece ends: how many, and lane j's place of its tile j
        auto look_up = [&](uint32_t &place) -> int {
            place = kNoTile;
            int n = 0;
            while (inside && n < kWindow) {
                const int take = min(kWindow - n, walk.u1 - ub);
                const int tile = walk.w.tile0 + ub * UT + lane - n * UT;
                if (lane >= n * UT && lane < (n + take) * UT && tile < walk.w.tiles) {
                    const int pg = tile / tpp;
                    const int32_t blk = a.block_table[static_cast<int64_t>(walk.b) * a.max_blocks + pg];
                    if (blk >= 0 && blk < a.num_blocks)
                        place =
                            static_cast<uint32_t>((static_cast<int64_t>(blk) * hkv + walk.kvh) * tpp + (tile - pg * tpp));
                    else
                        atomicOr(&g_kv4_err, ERRBIT_INDEX);  // left out
                }
                n += take;
                ub += take;
                if (ub == walk.u1) {
                    inside = walk.next(a, hkv, group);
                    ub = walk.u0;
                }
            }
            return n;
        };
        bool ok = true;
        uint32_t place, place_next;
        int n = look_up(place);
        while (n > 0 && ok) {
            int n_next = -1;  // not looked up yet
            place_next = kNoTile;
            // lanes 2 j and 2 j + 1 copy K and V of pair j: four tiles each, rows of the caches' maps
            int32_t row[2 * UT];
#pragma unroll
            for (int i = 0; i < 2 * UT; ++i)
                row[i] = static_cast<int32_t>(__shfl_sync(0xffffffffu, place, ((lane / 2) * 2 * UT + i) & 31));
            const uint32_t have = __ballot_sync(0xffffffffu, place != kNoTile);
            const int window_pairs = (n + 1) / 2;
            const uint32_t pair = pairs + lane / 2, st = pair % kPairs, parity = (pair / kPairs - 1) & 1;
            uint8_t *dst = ring + st * (2 * C::kStageBytes) + lane % 2 * C::kStageBytes;
            for (int first = 0; first < window_pairs; first += 2) {
                const bool live = lane / 4 == first / 2 && lane / 2 < window_pairs;
                bool free_now = true;
                if (live && pair >= kPairs) free_now = mbar_wait_bounded(&empty[st], parity);
                ok = __all_sync(0xffffffffu, free_now);
                if (!ok) {
                    pairs += static_cast<uint32_t>(first);
                    break;
                }
                if (live) holds[2 * st + lane % 2] = static_cast<int32_t>((have >> (lane * UT)) & ((1u << UT) - 1));
                __syncwarp();
                if (live) {
                    if (lane % 2 == 0) mbar_arrive_expect_tx(&full[st], 2 * C::kStageBytes);
                    // a row out of range reads zeros
                    tma_gather4_2d(dst, lane % 2 ? &tm_v : &tm_k, &full[st], 0, row);
                }
                __syncwarp();
                // with copies under way, what comes after this window
                if (n_next < 0 && (first == 2 || first + 2 >= window_pairs)) n_next = look_up(place_next);
            }
            if (ok) pairs += static_cast<uint32_t>(window_pairs);
            n = n_next;
            place = place_next;
        }
        if (!ok) {  // a consumer gave up: never leave with copies in flight
            if (lane == 0) atomicOr(&g_kv4_err, ERRBIT_EMPTY_WAIT);
            for (uint32_t i = pairs > kPairs ? pairs - kPairs : 0; i < pairs; ++i)
                (void)mbar_wait_bounded(&full[i % kPairs], (i / kPairs) & 1);
        }
        return;
    }

    // ==================================================== consumers
    const int g = lane >> 2, t = lane & 3;
    const float base = a.sm_scale * *a.k_scale * kLog2e;
    const float v_scale = *a.v_scale;
    constexpr int kLaneCodes = D / 4;  // codes of a key a lane holds for S^T
    constexpr int E = D / 32;          // of a row, when a warp joins its parts
    constexpr int kSteps = D / 16;
    static_assert(NT * kSteps * 32 * 8 <= C::kRecFloats * 4, "a record holds q");
    uint32_t count = 0;  // units of the pieces before this one
    int turn = 0;        // count % W
    bool failed = false;

    // The walk stays in shared memory: what the unit loop does not need would
    // cost it a dozen registers.
    Walk<R, UT, C::kSegCost> &kept = s_walk[warp];
    if (lane == 0) kept = walk;
    __syncwarp();
    while (true) {
        Walk<R, UT, C::kSegCost> walk = kept;
        __syncwarp();
        const bool more = walk.next(a, hkv, group);
        if (lane == 0) kept = walk;
        __syncwarp();
        if (!more) break;
        const int n_units = walk.u1 - walk.u0;
        const bool alone = n_units == 1 && walk.w.units == 1;
        int first = warp - turn;  // this warp's first unit of the piece
        if (first < 0) first += W;
        const uint32_t piece = count;
        count += static_cast<uint32_t>(n_units);
        turn = (turn + n_units) % W;
        if (alone && first != 0) continue;
        const int tile_row0 = walk.row_tile * R;
        const int tile_rows = walk.w.n_q * group - tile_row0;  // rows left of the sequence (some may be other tiles')
        const int first_pos = walk.w.len - walk.w.n_q;  // position of query token 0

        // ---- q as f16 B fragments, an exact power-of-two rescale per row
        // in the warp's record, which is free until the piece ends: in registers they would
        // take a thread past the 96 that let eight consumer warps run beside the producer
        // (16 x 32768 keys of 8 heads: 129 us instead of 123)
        uint2 *sq = reinterpret_cast<uint2 *>(merge + warp * C::kRecFloats) + lane;  // [NT][kSteps][32]
        float sc[NT][2];   // score scale of this lane's columns 2t, 2t + 1
        int pos[NT][2];    // their positions
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = n * 8 + g;
            const bool live = r < tile_rows;
            const int tok = live && walk.w.n_q > 1 ? (tile_row0 + r) / group : 0, h = live ? tile_row0 + r - tok * group : 0;
            const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.q) +
                                       static_cast<int64_t>(walk.w.q0 + tok) * a.q_stride +
                                       (walk.kvh * group + h) * D + t * kLaneCodes;
            uint4 v[kLaneCodes / 8];
            uint32_t mx = 0;
#pragma unroll
            for (int i = 0; i < kLaneCodes / 8; ++i) {
                v[i] = live ? *reinterpret_cast<const uint4 *>(src + 8 * i) : make_uint4(0, 0, 0, 0);
                mx = max_u16x2(max_u16x2(max_u16x2(mx, v[i].x & 0x7FFF7FFFu), v[i].y & 0x7FFF7FFFu),
                               max_u16x2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu));
            }
            uint32_t m16 = max(mx & 0xFFFFu, mx >> 16);
            m16 = max(m16, __shfl_xor_sync(0xffffffffu, m16, 1));
            m16 = max(m16, __shfl_xor_sync(0xffffffffu, m16, 2));
            const int e = f16_rescale_exp(m16);
            const float up = pow2_int(e), down = pow2_int(-e);
#pragma unroll
            for (int i = 0; i < kLaneCodes / 8; ++i) {
                const uint2 b0 = make_uint2(f32x2_to_f16x2(bf16lo_to_f32(v[i].x) * up, bf16hi_to_f32(v[i].x) * up),
                                            f32x2_to_f16x2(bf16lo_to_f32(v[i].y) * up, bf16hi_to_f32(v[i].y) * up));
                const uint2 b1 = make_uint2(f32x2_to_f16x2(bf16lo_to_f32(v[i].z) * up, bf16hi_to_f32(v[i].z) * up),
                                            f32x2_to_f16x2(bf16lo_to_f32(v[i].w) * up, bf16hi_to_f32(v[i].w) * up));
                sq[(n * kSteps + 2 * i) * 32] = b0;
                sq[(n * kSteps + 2 * i + 1) * 32] = b1;
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                sc[n][c] = base * __shfl_sync(0xffffffffu, down, 8 * t + 4 * c);
                pos[n][c] = first_pos + __shfl_sync(0xffffffffu, tok, 8 * t + 4 * c);
            }
        }
        // keys below `clear_hi` and from `clear_lo` on are seen by every row of the tile
        const int last_tok = walk.w.n_q > 1 ? min(tile_row0 + R - 1, walk.w.n_q * group - 1) / group : 0;
        const int clear_hi = first_pos + (walk.w.n_q > 1 ? tile_row0 / group : 0) + 1;
        const int clear_lo =
            a.window > 0 ? static_cast<int>(max(int64_t{0}, static_cast<int64_t>(first_pos) + last_tok - a.window + 1)) : 0;
        const int len = walk.w.len, piece_key = (walk.w.tile0 + walk.u0 * UT) * kKv4Tile;

        float m_run[NT][2], l_run[NT][2], o[NT][kSteps][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int c = 0; c < 2; ++c) m_run[n][c] = -INFINITY, l_run[n][c] = 0.0f;
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[n][i][j] = 0.0f;
        }

        for (int u = first; u < n_units && !failed; u += W) {
            const uint32_t idx = piece + static_cast<uint32_t>(u), st = idx % S;
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(&full[st / 2], (idx / S) & 1))) {
                if (lane == 0) atomicOr(&g_kv4_err, ERRBIT_FULL_WAIT);
                failed = true;
                break;
            }
            const uint32_t have = static_cast<uint32_t>(holds[st]);
            const uint8_t *kt = ring + st / 2 * (2 * C::kStageBytes) + st % 2 * (UT * T), *vt = kt + C::kStageBytes;
            const int key0 = piece_key + u * C::kKeys;
            // some row does not see some key, or a key is not there
            const bool partial = have != (1u << UT) - 1 || key0 + C::kKeys > min(len, clear_hi) || key0 < clear_lo;

            // ---- S^T: lane holds keys kv4_row(g), + 8 of each tile, rows 2t, 2t + 1 of each n
            float s[UT][NT][4];
#pragma unroll
            for (int h = 0; h < UT; ++h) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[h][n][j] = 0.0f;
                uint32_t f[2][kSteps * 2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int row = kv4_row(g) + 8 * q;
                    const uint8_t *src = kt + h * T + row * (D / 2) + t * (kLaneCodes / 2);
                    if constexpr (D == 128) {
                        const uint4 w = *reinterpret_cast<const uint4 *>(src);
                        const uint32_t sb = *reinterpret_cast<const uint16_t *>(kt + h * T + 8 * D + row * 8 + 2 * t);
                        const uint32_t s2 = e4m3x2_to_f16x2(sb);
                        const uint32_t sl = __byte_perm(s2, s2, 0x1010), sh = __byte_perm(s2, s2, 0x3232);
                        uint32_t c[4];
                        e2m1x8_to_f16x2x4(w.x, c);
#pragma unroll
                        for (int i = 0; i < 4; ++i) f[q][i] = mul_f16x2(c[i], sl);
                        e2m1x8_to_f16x2x4(w.y, c);
#pragma unroll
                        for (int i = 0; i < 4; ++i) f[q][4 + i] = mul_f16x2(c[i], sl);
                        e2m1x8_to_f16x2x4(w.z, c);
#pragma unroll
                        for (int i = 0; i < 4; ++i) f[q][8 + i] = mul_f16x2(c[i], sh);
                        e2m1x8_to_f16x2x4(w.w, c);
#pragma unroll
                        for (int i = 0; i < 4; ++i) f[q][12 + i] = mul_f16x2(c[i], sh);
                    } else {
                        const uint2 w = *reinterpret_cast<const uint2 *>(src);
                        const uint32_t sb = kt[h * T + 8 * D + row * 4 + t];
                        const uint32_t sl = e4m3x2_to_f16x2(sb | (sb << 8));
                        uint32_t c[4];
                        e2m1x8_to_f16x2x4(w.x, c);
#pragma unroll
                        for (int i = 0; i < 4; ++i) f[q][i] = mul_f16x2(c[i], sl);
                        e2m1x8_to_f16x2x4(w.y, c);
#pragma unroll
                        for (int i = 0; i < 4; ++i) f[q][4 + i] = mul_f16x2(c[i], sl);
                    }
                }
#pragma unroll
                for (int i = 0; i < kSteps; ++i)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint2 b = sq[(n * kSteps + i) * 32];
                        mma_f16_16816(s[h][n], f[0][2 * i], f[1][2 * i], f[0][2 * i + 1], f[1][2 * i + 1], b.x, b.y);
                    }
            }
#pragma unroll
            for (int h = 0; h < UT; ++h)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[h][n][j] *= sc[n][j & 1];
            if (partial) {
#pragma unroll
                for (int h = 0; h < UT; ++h)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int key = key0 + h * kKv4Tile + kv4_row(g) + 8 * (j >> 1);
                            const int p = pos[n][j & 1];
                            const bool seen = ((have >> h) & 1) && key <= p && (a.window == 0 || key > p - a.window);
                            if (!seen) s[h][n][j] = -INFINITY;
                        }
            }

            // ---- online softmax per row over the unit's keys
            float mt[NT][2];
            bool grows = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float v = fmaxf(s[0][n][c], s[0][n][c + 2]);
#pragma unroll
                    for (int h = 1; h < UT; ++h) v = fmaxf(v, fmaxf(s[h][n][c], s[h][n][c + 2]));
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
                    mt[n][c] = v;
                    grows |= v > m_run[n][c];
                }
            if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float al[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float mn = fmaxf(m_run[n][c], mt[n][c]);
                        al[c] = mn == -INFINITY ? 1.0f : ex2(m_run[n][c] - mn);
                        m_run[n][c] = mn;
                        l_run[n][c] *= al[c];
                    }
#pragma unroll
                    for (int i = 0; i < kSteps; ++i) {
                        o[n][i][0] *= al[0];
                        o[n][i][1] *= al[1];
                        o[n][i][2] *= al[0];
                        o[n][i][3] *= al[1];
                    }
                }
            }
            uint32_t pb[UT][NT][2];  // P^T as B fragments: keys 2t, 2t + 1 (+ 8) of the tile, row g
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float ref[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) ref[c] = m_run[n][c] == -INFINITY ? 0.0f : m_run[n][c] - kPShift;
#pragma unroll
                for (int h = 0; h < UT; ++h) {
                    float p[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) p[j] = ex2(s[h][n][j] - ref[j & 1]);
                    l_run[n][0] += p[0] + p[2];
                    l_run[n][1] += p[1] + p[3];
                    pb[h][n][0] = transpose8x8(f32x2_to_f16x2(p[0], p[1]));
                    pb[h][n][1] = transpose8x8(f32x2_to_f16x2(p[2], p[3]));
                }
            }

            // ---- O^T += V^T P^T
#pragma unroll
            for (int h = 0; h < UT; ++h) {
                uint32_t sb[4], w[4][D / 64];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int row = kv4_row(2 * t + (j & 1)) + 8 * (j >> 1);
                    const uint8_t *src = vt + h * T + row * (D / 2) + g * (D / 16);
                    if constexpr (D == 128) {
                        const uint2 v = *reinterpret_cast<const uint2 *>(src);
                        w[j][0] = v.x;
                        w[j][1] = v.y;
                    } else {
                        w[j][0] = *reinterpret_cast<const uint32_t *>(src);
                    }
                    sb[j] = vt[h * T + 8 * D + row * (D / 16) + g * D / 128];
                }
                if (partial) {
                    // What a row does not see has weight 0, which does not hide NaN: not the old bytes past the end and
                    // in tiles left out, nor a stored NaN scale, which goes to the rows that see its key by hand.
                    uint32_t nan = 0;  // the tile's keys with NaN in this lane's elements
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int row = kv4_row(2 * t + (j & 1)) + 8 * (j >> 1);
                        if (!((have >> h) & 1) || key0 + h * kKv4Tile + row >= len) sb[j] = 0;
                        if ((sb[j] & 0x7Fu) == 0x7Fu) sb[j] = 0, nan |= 1u << row;
                    }
                    if (__any_sync(0xffffffffu, nan != 0)) {
                        nan |= __shfl_xor_sync(0xffffffffu, nan, 1);
                        nan |= __shfl_xor_sync(0xffffffffu, nan, 2);
                        for (; nan != 0; nan &= nan - 1) {
                            const int key = key0 + h * kKv4Tile + __ffs(nan) - 1;
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int c = 0; c < 2; ++c) {
                                    if (key > pos[n][c] || (a.window > 0 && key <= pos[n][c] - a.window)) continue;
#pragma unroll
                                    for (int i = 0; i < kSteps; ++i) o[n][i][c] = o[n][i][c + 2] = NAN;
                                }
                        }
                    }
                }
                const uint32_t s01 = e4m3x2_to_f16x2(sb[0] | (sb[1] << 8)), s23 = e4m3x2_to_f16x2(sb[2] | (sb[3] << 8));
                const uint32_t s0 = s01 & 0xFFFFu, s1 = s01 & 0xFFFF0000u, s2 = s23 & 0xFFFFu, s3 = s23 & 0xFFFF0000u;
#pragma unroll
                for (int q = 0; q < D / 64; ++q) {
                    uint32_t f0[4], f1[4], f2[4], f3[4];
                    e2m1x8_to_f16x2x4(w[0][q], f0);
                    e2m1x8_to_f16x2x4(w[1][q], f1);
                    e2m1x8_to_f16x2x4(w[2][q], f2);
                    e2m1x8_to_f16x2x4(w[3][q], f3);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t a0 = pair_f16(f0[i], f1[i], s0, s1, 0);
                        const uint32_t a1 = pair_f16(f0[i], f1[i], s0, s1, 1);
                        const uint32_t a2 = pair_f16(f2[i], f3[i], s2, s3, 0);
                        const uint32_t a3 = pair_f16(f2[i], f3[i], s2, s3, 1);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma_f16_16816(o[n][q * 4 + i], a0, a1, a2, a3, pb[h][n][0], pb[h][n][1]);
                    }
                }
            }
            __syncwarp();  // the stage has been read
            if (lane == 0) mbar_arrive(&empty[st / 2]);
        }

#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    l_run[n][c] += __shfl_xor_sync(0xffffffffu, l_run[n][c], off);
        const int q0 = kept.w.q0, n_q = kept.w.n_q, head0 = kept.kvh * group, row0 = kept.row_tile * R;
        const int rows = n_q * group - row0;
        const bool starts = kept.u0 == 0, ends = kept.u1 == kept.w.units;
        if (alone) {  // lane: elements g D / 8 .. of rows 2t, 2t + 1 of each n
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int r = n * 8 + 2 * t + c;
                    if (r >= rows) continue;
                    const int tok = n_q > 1 ? (row0 + r) / group : 0, h = row0 + r - tok * group;
                    const int64_t row = static_cast<int64_t>(q0 + tok) * a.q_heads + head0 + h;
                    const float L = l_run[n][c], inv = L == 0.0f ? 0.0f : v_scale / L;  // 0: no key; may be NaN
                    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + row * D + g * (D / 8));
#pragma unroll
                    for (int i = 0; i < kSteps; i += 4)
                        dst[i / 4] = make_uint4(f32x2_to_bf16x2(o[n][i][c] * inv, o[n][i][c + 2] * inv),
                                                f32x2_to_bf16x2(o[n][i + 1][c] * inv, o[n][i + 1][c + 2] * inv),
                                                f32x2_to_bf16x2(o[n][i + 2][c] * inv, o[n][i + 2][c + 2] * inv),
                                                f32x2_to_bf16x2(o[n][i + 3][c] * inv, o[n][i + 3][c + 2] * inv));
                    if (a.lse && g == 0)
                        a.lse[row] = L == 0.0f ? -INFINITY : (m_run[n][c] - kPShift + log2f(L)) * kLn2;
                }
            continue;
        }
        // ---- the warps' parts of the piece: m[R], l[R], o[R][D] each
        float *rec = merge + warp * C::kRecFloats;
        __syncwarp();  // q has been read
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = n * 8 + 2 * t + c;
                if (g == 0) {
                    rec[r] = m_run[n][c];
                    rec[R + r] = l_run[n][c];
                }
#pragma unroll
                for (int i = 0; i < kSteps; i += 2)
                    *reinterpret_cast<float4 *>(rec + 2 * R + r * D + 4 * merge_chunk<D>(r, g * (D / 32) + i / 2)) =
                        make_float4(o[n][i][c], o[n][i][c + 2], o[n][i + 1][c], o[n][i + 1][c + 2]);
            }
        bar_consumers(W * 32);
        // ---- joined, a warp per row; a lane has D / 32 elements of it
        float *out_rec = records + static_cast<int64_t>(2 * cta + (starts ? 1 : 0)) * C::kRecFloats;
        const int live = min(rows, R);
        auto finish_row = [&](int r, float M, float L, const float (&O)[E]) {
            const int tok = n_q > 1 ? (row0 + r) / group : 0, h = row0 + r - tok * group;
            const int64_t row = static_cast<int64_t>(q0 + tok) * a.q_heads + head0 + h;
            const float inv = L == 0.0f ? 0.0f : v_scale / L;
            uint32_t *dst =
                reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(a.out) + row * D + lane * E);
            if constexpr (E == 4)
                *reinterpret_cast<uint2 *>(dst) =
                    make_uint2(f32x2_to_bf16x2(O[0] * inv, O[1] * inv), f32x2_to_bf16x2(O[2] * inv, O[3] * inv));
            else
                *dst = f32x2_to_bf16x2(O[0] * inv, O[1] * inv);
            if (a.lse && lane == 0) a.lse[row] = L == 0.0f ? -INFINITY : (M - kPShift + log2f(L)) * kLn2;
        };
        // eight lanes find the weights of the warps' parts of one of four rows
        for (int r0 = warp; r0 < live; r0 += 4 * W) {
            const int mine = r0 + (lane >> 3) * W, w_mine = lane & 7;
            const bool there = w_mine < W && mine < live;
            const float m = there ? merge[w_mine * C::kRecFloats + mine] : -INFINITY;
            const float l = there ? merge[w_mine * C::kRecFloats + R + mine] : 0.0f;
            // a part without keys has weight -1 and is left out; its l is 0, or NaN where its scores are
            const float M = warp_max<8>(m), f = m == -INFINITY ? -1.0f : ex2(m - M);
            const float L = warp_sum<8>(f < 0.0f ? l : f * l);
#pragma unroll
            for (int k = 0; k < 4 && k * W < R; ++k) {
                const int r = r0 + k * W;
                if (r >= live) break;
                float O[E] = {};
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const float fw = __shfl_sync(0xffffffffu, f, 8 * k + w);
                    float v[E];
                    load_floats(merge + w * C::kRecFloats + 2 * R + r * D + 4 * merge_chunk<D>(r, lane * E / 4) +
                                    lane * E % 4, v);
                    if (fw >= 0.0f) fma_floats(O, fw, v);
                }
                const float Mr = __shfl_sync(0xffffffffu, M, 8 * k), Lr = __shfl_sync(0xffffffffu, L, 8 * k);
                if (starts && ends) {
                    finish_row(r, Mr, Lr, O);
                } else {
                    if (lane == 0) out_rec[r] = Mr, out_rec[R + r] = Lr;
                    store_floats(out_rec + 2 * R + r * D + lane * E, O);
                }
            }
        }
        bar_consumers(W * 32);  // the warps' records are free again
        if (starts && ends) continue;
        // ---- a part of a split segment: the last of its CTAs to come here joins them, in their order
        if (tid == 0) {
            // the line's step of the segment's first unit, and whose share a step is in
            const int64_t at = starts ? s_line.hi - kept.u1 : s_line.lo - kept.u0;
            auto owner = [&](int64_t step) {
                return static_cast<int>(quotient((step + 1) * s_line.ctas + s_line.total - 1, s_line.total) - 1);
            };
            const int c0 = owner(at), parts = owner(at + kept.w.units - 1) - c0 + 1;
            // releases what the barrier has ordered before it, the whole CTA's record; wraps to 0
            const uint32_t before = atomic_inc_acq_rel(arrived + c0, static_cast<uint32_t>(parts - 1));
            s_first = c0;
            s_parts = before == static_cast<uint32_t>(parts - 1) ? parts : 0;
        }
        bar_consumers(W * 32);
        const int parts = s_parts;
        if (parts == 0) continue;  // s_first and s_parts are written after the next piece's barriers only
        const int first_cta = s_first;
        auto part = [&](int j) {
            return records + static_cast<int64_t>(2 * (first_cta + j) + (j == 0)) * C::kRecFloats;
        };
#pragma unroll 1
        for (int r = warp; r < live; r += W) {
            float M = -INFINITY, L = 0.0f;
            float O[E] = {};
            for (int j0 = 0; j0 < parts; j0 += 32) {  // lane j: part j0 + j's m and l
                constexpr int kAhead = 8;
                const int count = min(32, parts - j0);
                float m = -INFINITY, l = 0.0f;
                if (lane < count) m = __ldcg(part(j0 + lane) + r), l = __ldcg(part(j0 + lane) + R + r);
                float v[kAhead][E];
                auto load = [&](int i) {
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) {
#pragma unroll
                        for (int d = 0; d < E; ++d) v[u][d] = 0.0f;
                        if (i + u < count) load_floats_cg(part(j0 + i + u) + 2 * R + r * D + lane * E, v[u]);
                    }
                };
                load(0);  // on their way beside m and l
                const float M_new = fmaxf(M, warp_max<32>(m));
                const float f = m == -INFINITY ? 0.0f : ex2(m - M_new), keep = M == -INFINITY ? 0.0f : ex2(M - M_new);
                L = L * keep + warp_sum<32>(f * l);
#pragma unroll
                for (int d = 0; d < E; ++d) O[d] *= keep;
                const uint32_t some = __ballot_sync(0xffffffffu, m != -INFINITY);
                for (int i = 0; i < count; i += kAhead) {
                    if (i > 0) load(i);
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) {
                        const float fu = __shfl_sync(0xffffffffu, f, (i + u) & 31);
                        if (i + u < count && ((some >> (i + u)) & 1)) fma_floats(O, fu, v[u]);
                    }
                }
                M = M_new;
            }
            finish_row(r, M, L, O);
        }
    }
}

template <int D, int NT>
cudaError_t launch_attn(const Kv4AttnArgs &a, cudaStream_t stream) {
    using C = AttnCfg<D, NT>;
    auto kern = kv4_attn_kernel<D, NT>;
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!done[dev]) {
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
            if (e != cudaSuccess) return e;
            done[dev] = true;
        }
    }
    const int sms = device_sm_count() < kMaxSms ? device_sm_count() : kMaxSms;
    const unsigned ctas = static_cast<unsigned>(sms * C::kRes);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, 1, 1);
    cfg.blockDim = dim3(C::kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    CUtensorMap tm_k, tm_v;
    const uint64_t tiles = static_cast<uint64_t>(a.num_blocks * (a.page_size / kKv4Tile) * a.kv_heads);
    for (const auto &m : {std::make_pair(&tm_k, a.k_cache), std::make_pair(&tm_v, a.v_cache)})
        if (!encode_tensor_map_2d(m.first, CU_TENSOR_MAP_DATA_TYPE_INT64, m.second, C::T / 8, tiles, C::T, C::T / 8, 1,
                                  CU_TENSOR_MAP_SWIZZLE_NONE))
            return cudaErrorInvalidValue;
    return cudaLaunchKernelEx(&cfg, kern, tm_k, tm_v, a);
}

template <int D>
cudaError_t launch_attn_rows(const Kv4AttnArgs &a, cudaStream_t stream) {
    const int64_t rows = a.max_q * (a.q_heads / a.kv_heads);
    if (rows <= 8) return launch_attn<D, 1>(a, stream);
    if (rows <= 16) return launch_attn<D, 2>(a, stream);
    if (rows <= 24) return launch_attn<D, 3>(a, stream);
    return launch_attn<D, 4>(a, stream);
}

cudaError_t launch_copy(void (*kern)(Kv4CopyArgs, uint64_t, bool), const Kv4CopyArgs &a, bool wide, cudaStream_t stream) {
    const uint64_t per_row = static_cast<uint64_t>(a.kv_heads * (a.head_dim / 32));  // >= 2
    const uint64_t inverse = ~uint64_t{0} / per_row + 1;
    const int64_t items = a.tokens * static_cast<int64_t>(per_row);
    const int64_t blocks = (items + kCopyThreads - 1) / kCopyThreads;
    if (blocks >= int64_t{1} << 31) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 2, 1);
    cfg.blockDim = dim3(kCopyThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a, inverse, wide);
}

bool aligned32(const void *p) { return reinterpret_cast<uintptr_t>(p) % 32 == 0; }

}  // namespace

cudaError_t launch_kv4_append(const Kv4CopyArgs &a, cudaStream_t stream) {
    const bool wide = aligned32(a.k) && aligned32(a.v) && a.k_stride % 16 == 0 && a.v_stride % 16 == 0;
    return launch_copy(a.head_dim == 128 ? kv4_append_kernel<128> : kv4_append_kernel<64>, a, wide, stream);
}

cudaError_t launch_kv4_gather(const Kv4CopyArgs &a, cudaStream_t stream) {
    const bool wide = aligned32(a.k_out) && aligned32(a.v_out);
    return launch_copy(a.head_dim == 128 ? kv4_gather_kernel<128> : kv4_gather_kernel<64>, a, wide, stream);
}

int64_t kv4_attention_ws_bytes(int64_t head_dim) {
    static_assert(2 * kMaxSms * 4 == FP4KV_WORKSPACE_COUNTER_BYTES, "the counters are first");
    return 2 * kMaxSms * 4 + int64_t{2} * kMaxSms * 32 * (head_dim + 2) * 4;
}

cudaError_t launch_kv4_attention(const Kv4AttnArgs &a, cudaStream_t stream) {
    return a.head_dim == 128 ? launch_attn_rows<128>(a, stream) : launch_attn_rows<64>(a, stream);
}

uint32_t take_kv4_error() {
    uint32_t v = 0;
    if (cudaMemcpyFromSymbol(&v, g_kv4_err, sizeof v) != cudaSuccess) return 0xFFFFFFFFu;
    const uint32_t zero = 0;
    cudaMemcpyToSymbol(g_kv4_err, &zero, sizeof zero);
    return v;
}

}  // namespace fp8bs
