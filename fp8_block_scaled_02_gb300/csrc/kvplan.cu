// kvplan.cu -- the paging plan of one serving step, built on the device from
// request lengths: new cache blocks from a free list, slot map, positions.
//
// For request b with c = ctx_lens[b] cached and n = new_lens[b] new tokens,
// page size P:
//   cu_new[b + 1] = cu_new[b] + n                  (the step's token axis)
//   have = ceil(c / P), need = ceil((c + n) / P) - have
//   block p of b: block_table[b][p] for p < have, else
//                 free_blocks[free_head + (need of requests before b) + p - have]
//   token i of b at position c + i: slot = block((c + i) / P) * P + (c + i) % P
// All of it is prefix sums over the requests plus one lookup per token, a few
// hundred KB at most: bound by launch and dependent-load latency, not bytes.
//
// One thread-block cluster: every CTA scans all the requests into its own
// shared memory (no exchange between CTAs), then the CTAs share the tokens.
// The cluster barrier between the scan and the first store lets seq_lens and
// free_head_out be the arrays they were read from.
#include "serving.cuh"
#include "internal.h"

#include <mutex>

namespace fp8bs {

namespace {

__device__ uint32_t g_plan_err;

constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;

// Exclusive sum of `v` over the CTA's threads; `total` gets the whole sum.
__device__ __forceinline__ int64_t block_exclusive(int64_t v, int64_t *warp_sums, int64_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) {
        const int64_t s = warp_sums[w];
        if (w < warp) before += s;
        all += s;
    }
    __syncthreads();
    total = all;
    return before + x - v;
}

__device__ __forceinline__ int32_t clamp_i32(int64_t v) {
    return static_cast<int32_t>(v > 0x7fffffffll ? 0x7fffffffll : v);
}

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(KvPlanArgs a) {
    extern __shared__ int32_t plan_smem[];
    int32_t *cu = plan_smem;               // [batch + 1] first token of each request
    int32_t *ctx = cu + a.batch + 1;       // [batch] cached tokens
    int32_t *base = ctx + a.batch;         // [batch] free-list index of the first new block; -1: refused
    __shared__ int64_t sums[kPlanWarps];
    __shared__ int64_t s_taken;

    const int tid = threadIdx.x;
    const int rank = static_cast<int>(cluster_ctarank()), ctas = static_cast<int>(gridDim.x);
    const int batch = static_cast<int>(a.batch);
    const int64_t page = a.page_size, cap = a.max_blocks * page;
    const int per = (batch + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(batch, tid * per), b1 = min(batch, b0 + per);
    uint32_t err = 0;
    if (tid == 0) s_taken = 0;
    pdl_wait();  // the lengths and the tables may come from the previous kernel

    const int64_t head = *a.free_head;
    const bool head_ok = head >= 0 && head <= a.num_free;
    if (!head_ok) err |= ERRBIT_INDEX;

    // ---- the token axis
    int64_t tokens = 0;
    for (int b = b0; b < b1; ++b) tokens += max(0, a.new_lens[b]);
    int64_t total_tokens, at = block_exclusive(tokens, sums, total_tokens);

    // ---- blocks asked for, in request order
    int64_t asked = 0;
    for (int b = b0; b < b1; ++b) {
        const int64_t c = a.ctx_lens[b], n = a.new_lens[b];
        cu[b] = clamp_i32(at);
        ctx[b] = static_cast<int32_t>(c);
        at += n > 0 ? n : 0;
        const bool ok = c >= 0 && n >= 0 && c + n <= cap && at <= a.num_tokens;
        if (!ok) err |= ERRBIT_INDEX;
        const int64_t need = ok ? (c + n + page - 1) / page - (c + page - 1) / page : 0;
        base[b] = ok ? static_cast<int32_t>(need) : -1;  // the need, until the scan is known
        asked += need;
    }
    if (tid == 0) cu[batch] = clamp_i32(total_tokens);
    int64_t total_asked, before = block_exclusive(asked, sums, total_asked);
    int64_t taken = 0;
    for (int b = b0; b < b1; ++b) {
        const int64_t need = base[b];
        if (need < 0) continue;
        const int64_t upto = before + need;
        if (need > 0 && (!head_ok || head + upto > a.num_free)) {
            base[b] = -1;  // the list has run out: refused whole, as is every later request that needs a block
            err |= ERRBIT_CAPACITY;
        } else {
            base[b] = need > 0 ? clamp_i32(head + before) : 0;
            if (need > 0) taken = upto;
        }
        before = upto;
    }
    if (taken > 0) atomicMax(reinterpret_cast<unsigned long long *>(&s_taken), static_cast<unsigned long long>(taken));
    __syncthreads();
    cluster_sync_all();  // every CTA has read the lengths and the head

    // ---- per request
    for (int b = rank * kPlanThreads + tid; b <= batch; b += ctas * kPlanThreads) {
        a.cu_new[b] = cu[b];
        if (b < batch) {
            const int64_t c = ctx[b];
            a.seq_lens[b] = static_cast<int32_t>(base[b] >= 0 ? c + (cu[b + 1] - cu[b]) : min(max(c, int64_t{0}), cap));
        }
    }
    if (rank == 0 && tid == 0) *a.free_head_out = static_cast<int32_t>(head + s_taken);

    // ---- per token
    for (int64_t j = static_cast<int64_t>(rank) * kPlanThreads + tid; j < a.num_tokens;
         j += static_cast<int64_t>(ctas) * kPlanThreads) {
        int lo = 0, hi = batch;  // the request whose [cu[b], cu[b + 1]) holds j; batch: none
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid + 1] > j) hi = mid;
            else lo = mid + 1;
        }
        int32_t req = -1, pos = -1, slot = -1;
        if (lo < batch) {
            req = lo;
            if (base[lo] >= 0) {
                const int64_t c = ctx[lo], p = c + (j - cu[lo]);
                const int64_t pg = p / page, have = (c + page - 1) / page;
                pos = static_cast<int32_t>(p);
                int32_t *entry = a.block_table + lo * a.max_blocks + pg;
                int32_t blk;
                if (pg < have) {
                    blk = *entry;
                } else {
                    blk = a.free_blocks[base[lo] + (pg - have)];
                    if (blk < 0 || blk >= a.num_blocks) blk = -1;
                    if (p == pg * page) *entry = blk;  // the block's first token opens it
                }
                if (blk < 0 || blk >= a.num_blocks) err |= ERRBIT_INDEX;
                else slot = static_cast<int32_t>(blk * page + (p - pg * page));
            }
        }
        a.requests[j] = req;
        a.positions[j] = pos;
        a.slots[j] = slot;
    }
    if (err) atomicOr(&g_plan_err, err);
    pdl_launch_dependents();
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlanArgs &a, cudaStream_t stream) {
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!done[dev]) {
            const cudaError_t e = cudaFuncSetAttribute(kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       static_cast<int>(12 * kPlanMaxBatch + 4));
            if (e != cudaSuccess) return e;
            done[dev] = true;
        }
    }
    int ctas = 1;
    while (ctas < 8 && static_cast<int64_t>(ctas) * kPlanThreads * 4 < a.num_tokens) ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, 1, 1);
    cfg.blockDim = dim3(kPlanThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(12 * a.batch + 4);
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = ctas;
    attrs[1].val.clusterDim.y = 1;
    attrs[1].val.clusterDim.z = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kv_plan_kernel, a);
}

uint32_t take_plan_error() {
    uint32_t v = 0;
    if (cudaMemcpyFromSymbol(&v, g_plan_err, sizeof v) != cudaSuccess) return 0xFFFFFFFFu;
    const uint32_t zero = 0;
    cudaMemcpyToSymbol(g_plan_err, &zero, sizeof zero);
    return v;
}

}  // namespace fp8bs
