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
#include "common.cuh"
#include "internal.h"

namespace fp8bs {

namespace {

__device__ uint32_t g_kv4_err;


__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The tile that holds slot `slot` of kv head `h`.
__device__ __forceinline__ int64_t tile_index(int64_t slot, int h, int kv_heads, int page_size) {
    const int64_t blk = slot / page_size;
    const int off = static_cast<int>(slot - blk * page_size);
    return (blk * kv_heads + h) * (page_size / kKv4Tile) + off / kKv4Tile;
}

// ------------------------------------------------------- append and gather
constexpr int kCopyThreads = 256;

// One thread per group of 16 elements; blockIdx.y selects K or V.
__global__ void __launch_bounds__(kCopyThreads) kv4_append_kernel(Kv4CopyArgs a) {
    const bool is_v = blockIdx.y != 0;
    const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(is_v ? a.v : a.k);
    const int64_t stride = is_v ? a.v_stride : a.k_stride;
    uint8_t *cache = is_v ? a.v_cache : a.k_cache;
    const int d = static_cast<int>(a.head_dim), groups = d / 16;
    const int per_row = static_cast<int>(a.kv_heads) * groups;
    pdl_wait();
    const float s = __ldg(is_v ? a.v_scale : a.k_scale);
    const float six_s = 6.0f * s;
    const int64_t total = a.tokens * per_row;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * kCopyThreads) {
        const int64_t t = i / per_row;
        const int e = static_cast<int>(i - t * per_row), h = e / groups, g = e - h * groups;
        const int64_t slot = __ldg(a.slots + t);
        if (slot < 0 || slot >= a.num_slots) {
            if (slot != -1 && e == 0 && !is_v) atomicOr(&g_kv4_err, ERRBIT_INDEX);
            continue;
        }
        const __nv_bfloat16 *src = x + t * stride + static_cast<int64_t>(e) * 16;
        const uint4 w[2] = {ld_nc_v4(src), ld_nc_v4(src + 8)};
        const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
        uint32_t mx = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) mx = max_u16x2(mx, u[j] & 0x7FFF7FFFu);
        const float amax = __uint_as_float(max(mx & 0xFFFFu, mx >> 16) << 16);
        const uint32_t sc = f32x2_to_e4m3x2(amax / six_s, 0.0f) & 0xFFu;
        const float den = f16x2_to_f32x2(e4m3x2_to_f16x2(sc)).x * s;
        uint2 codes = make_uint2(0, 0);
        if (den > 0.0f) {
            float q[2][8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                q[j >> 2][2 * (j & 3)] = bf16lo_to_f32(u[j]) / den;
                q[j >> 2][2 * (j & 3) + 1] = bf16hi_to_f32(u[j]) / den;
            }
            codes = make_uint2(f32x8_to_e2m1x8(q[0]), f32x8_to_e2m1x8(q[1]));
        }
        uint8_t *tile = cache + tile_index(slot, h, static_cast<int>(a.kv_heads), static_cast<int>(a.page_size)) *
                                    kv4_tile_bytes(d);
        const int row = static_cast<int>(slot & (kKv4Tile - 1));
        *reinterpret_cast<uint2 *>(tile + row * (d / 2) + g * 8) = codes;
        tile[8 * d + row * groups + g] = static_cast<uint8_t>(sc);
    }
}

__global__ void __launch_bounds__(kCopyThreads) kv4_gather_kernel(Kv4CopyArgs a) {
    const bool is_v = blockIdx.y != 0;
    const uint8_t *cache = is_v ? a.v_cache : a.k_cache;
    uint4 *out = static_cast<uint4 *>(is_v ? a.v_out : a.k_out);
    const int d = static_cast<int>(a.head_dim), groups = d / 16;
    const int per_row = static_cast<int>(a.kv_heads) * groups;
    pdl_wait();
    const float s = __ldg(is_v ? a.v_scale : a.k_scale);
    const int64_t total = a.tokens * per_row;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * kCopyThreads) {
        const int64_t t = i / per_row;
        const int e = static_cast<int>(i - t * per_row), h = e / groups, g = e - h * groups;
        const int64_t slot = __ldg(a.slots + t);
        uint32_t r[8] = {};
        if (slot < 0 || slot >= a.num_slots) {
            if (slot != -1 && e == 0 && !is_v) atomicOr(&g_kv4_err, ERRBIT_INDEX);
        } else {
            const uint8_t *tile = cache + tile_index(slot, h, static_cast<int>(a.kv_heads),
                                                     static_cast<int>(a.page_size)) * kv4_tile_bytes(d);
            const int row = static_cast<int>(slot & (kKv4Tile - 1));
            const uint2 codes = *reinterpret_cast<const uint2 *>(tile + row * (d / 2) + g * 8);
            const uint32_t sc = tile[8 * d + row * groups + g];
            const uint32_t sc2 = e4m3x2_to_f16x2(sc | (sc << 8));
            uint32_t h0[4], h1[4];
            e2m1x8_to_f16x2x4(codes.x, h0);
            e2m1x8_to_f16x2x4(codes.y, h1);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 lo = f16x2_to_f32x2(mul_f16x2(h0[j], sc2)), hi = f16x2_to_f32x2(mul_f16x2(h1[j], sc2));
                r[j] = f32x2_to_bf16x2(lo.x * s, lo.y * s);
                r[4 + j] = f32x2_to_bf16x2(hi.x * s, hi.y * s);
            }
        }
        out[2 * i] = make_uint4(r[0], r[1], r[2], r[3]);
        out[2 * i + 1] = make_uint4(r[4], r[5], r[6], r[7]);
    }
}

// --------------------------------------------------------------- attention
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// One warp per (query token, query head): a key at a time, the head's D
// elements over the lanes, an online softmax.  Query token i of the n_q
// tokens of a sequence of len keys stands at position len - n_q + i and sees
// the keys up to its own (of those, the newest `window`, if there is one).
__global__ void __launch_bounds__(32) kv4_attn_kernel(Kv4AttnArgs a) {
    const int lane = threadIdx.x;
    const int b = blockIdx.z, h = blockIdx.y, i = blockIdx.x;
    const int d = static_cast<int>(a.head_dim), per = d / 32;
    const int hkv = static_cast<int>(a.kv_heads), kvh = h / static_cast<int>(a.q_heads / a.kv_heads);
    pdl_wait();
    int64_t first = b, n_q = 1;
    if (a.cu_q) {
        first = a.cu_q[b];
        n_q = static_cast<int64_t>(a.cu_q[b + 1]) - first;
    }
    if (n_q < 0 || n_q > a.max_q || first < 0 || first + n_q > a.tokens) {
        if (lane == 0) atomicOr(&g_kv4_err, ERRBIT_INDEX);
        return;
    }
    if (i >= n_q) return;
    const int64_t cap = a.max_seq_len;
    int64_t len = a.seq_lens[b];
    if (len < 0 || len > cap) {
        if (lane == 0) atomicOr(&g_kv4_err, ERRBIT_INDEX);
        len = len < 0 ? 0 : cap;
    }
    const int64_t row = first + i;
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + row * a.q_stride + static_cast<int64_t>(h) * d;
    const float ks = *a.k_scale, vs = *a.v_scale;
    float qv[4], o[4] = {};
    for (int e = 0; e < per; ++e) qv[e] = __bfloat162float(q[lane * per + e]);
    float m = -INFINITY, l = 0.0f;
    const int64_t last = len - n_q + i;
    const int64_t from = a.window > 0 && last - a.window + 1 > 0 ? last - a.window + 1 : 0;
    for (int64_t j = from; j <= last; ++j) {
        const int32_t blk = a.block_table[b * a.max_blocks + j / a.page_size];
        if (blk < 0 || blk >= a.num_blocks) {
            if (lane == 0) atomicOr(&g_kv4_err, ERRBIT_INDEX);
            continue;
        }
        const int64_t slot = static_cast<int64_t>(blk) * a.page_size + j % a.page_size;
        const int64_t off = tile_index(slot, kvh, hkv, static_cast<int>(a.page_size)) * kv4_tile_bytes(d);
        const int r = static_cast<int>(slot & (kKv4Tile - 1));
        const uint8_t *kt = a.k_cache + off, *vt = a.v_cache + off;
        const int cb = r * (d / 2) + lane * per / 2, sb = 8 * d + r * (d / 16) + lane * per / 16;
        uint32_t kw = 0, vw = 0;
        for (int e = 0; e < per / 2; ++e) {
            kw |= static_cast<uint32_t>(kt[cb + e]) << (8 * e);
            vw |= static_cast<uint32_t>(vt[cb + e]) << (8 * e);
        }
        uint32_t kh[4], vh[4];
        e2m1x8_to_f16x2x4(kw, kh);
        e2m1x8_to_f16x2x4(vw, vh);
        const float ksc = f16x2_to_f32x2(e4m3x2_to_f16x2(kt[sb])).x * ks;
        const float vsc = f16x2_to_f32x2(e4m3x2_to_f16x2(vt[sb])).x * vs;
        float dot = 0.0f;
        for (int e = 0; e < per; ++e) {
            const float2 p = f16x2_to_f32x2(kh[e / 2]);
            dot += qv[e] * ((e & 1 ? p.y : p.x) * ksc);
        }
        const float s = warp_sum(dot) * a.sm_scale * kLog2e;
        const float mn = fmaxf(m, s);
        const float al = exp2f(m - mn), p = exp2f(s - mn);
        m = mn;
        l = l * al + p;
        for (int e = 0; e < per; ++e) {
            const float2 v = f16x2_to_f32x2(vh[e / 2]);
            o[e] = o[e] * al + p * ((e & 1 ? v.y : v.x) * vsc);
        }
    }
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + (row * a.q_heads + h) * d;
    for (int e = 0; e < per; ++e) out[lane * per + e] = __float2bfloat16_rn(l > 0.0f ? o[e] / l : 0.0f);
    if (a.lse && lane == 0) a.lse[row * a.q_heads + h] = l > 0.0f ? m * kLn2 + logf(l) : -INFINITY;
}

int copy_blocks(const Kv4CopyArgs &a) {
    const int64_t total = a.tokens * a.kv_heads * (a.head_dim / 16);
    int64_t blocks = (total + kCopyThreads - 1) / kCopyThreads;
    const int64_t cap = static_cast<int64_t>(device_sm_count()) * 8;
    return static_cast<int>(blocks > cap ? cap : blocks);
}

cudaError_t launch_pdl(void (*kern)(Kv4CopyArgs), dim3 grid, const Kv4CopyArgs &a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kCopyThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4CopyArgs &a, cudaStream_t stream) {
    return launch_pdl(kv4_append_kernel, dim3(copy_blocks(a), 2, 1), a, stream);
}

cudaError_t launch_kv4_gather(const Kv4CopyArgs &a, cudaStream_t stream) {
    return launch_pdl(kv4_gather_kernel, dim3(copy_blocks(a), 2, 1), a, stream);
}

int64_t kv4_attention_ws_bytes(int64_t head_dim) {
    return 160 * 32 * 2 * (head_dim + 2) * 4 + 16384;
}

cudaError_t launch_kv4_attention(const Kv4AttnArgs &a, cudaStream_t stream) {
    if (a.tokens == 0) return cudaSuccess;
    kv4_attn_kernel<<<dim3(static_cast<unsigned>(a.max_q), static_cast<unsigned>(a.q_heads),
                           static_cast<unsigned>(a.batch)),
                      32, 0, stream>>>(a);
    return cudaGetLastError();
}

uint32_t take_kv4_error() {
    uint32_t v = 0;
    if (cudaMemcpyFromSymbol(&v, g_kv4_err, sizeof v) != cudaSuccess) return 0xFFFFFFFFu;
    const uint32_t zero = 0;
    cudaMemcpyToSymbol(g_kv4_err, &zero, sizeof zero);
    return v;
}

}  // namespace fp8bs
