// logprobs.cu -- log probabilities of given tokens over a row of logits, the
// row's entropy, and its top alternatives.
//
// With m = max x, l = sum e^(x - m), t = sum (x - m) e^(x - m) over the row:
//   lse = m + log l,  logprob(i) = x_i - lse,  entropy = log l - t / l.
// The top alternatives are the first k of the row ordered by value, highest
// first, and by index, lowest first, among equals.
#include "common.cuh"
#include "internal.h"

namespace fp8bs {

namespace {

__device__ uint32_t g_lp_err;

constexpr int kLpThreads = 256;

template <bool F32>
__device__ __forceinline__ float logit(const void *row, int64_t i) {
    return F32 ? static_cast<const float *>(row)[i] : __bfloat162float(static_cast<const __nv_bfloat16 *>(row)[i]);
}

// Two partial sums over parts of a row: the second is brought to the larger maximum.
__device__ __forceinline__ void merge(float &m, float &l, float &t, float m2, float l2, float t2) {
    const float mn = fmaxf(m, m2);
    if (mn == -INFINITY) return;
    const float a = m == -INFINITY ? 0.0f : expf(m - mn), b = m2 == -INFINITY ? 0.0f : expf(m2 - mn);
    const float da = fmaxf(m - mn, -200.0f), db = fmaxf(m2 - mn, -200.0f);  // their weights are 0 there
    t = a * (t + da * l) + b * (t2 + db * l2);
    l = a * l + b * l2;
    m = mn;
}

template <bool F32>
__global__ void __launch_bounds__(kLpThreads) logprobs_kernel(LogprobArgs a) {
    __shared__ float sm[kLpThreads], sl[kLpThreads], st[kLpThreads];
    __shared__ int32_t si[kLpThreads];
    const int tid = threadIdx.x;
    const int64_t r = blockIdx.x, v = a.vocab;
    pdl_wait();
    const void *row = static_cast<const char *>(a.logits) + r * a.row_stride * (F32 ? 4 : 2);
    float m = -INFINITY, l = 0.0f, t = 0.0f;
    for (int64_t i = tid; i < v; i += kLpThreads) {
        const float x = logit<F32>(row, i);
        if (x == -INFINITY) continue;
        merge(m, l, t, x, 1.0f, 0.0f);
    }
    sm[tid] = m, sl[tid] = l, st[tid] = t;
    __syncthreads();
    for (int s = kLpThreads / 2; s > 0; s >>= 1) {
        if (tid < s) {
            merge(m, l, t, sm[tid + s], sl[tid + s], st[tid + s]);
            sm[tid] = m, sl[tid] = l, st[tid] = t;
        }
        __syncthreads();
    }
    m = sm[0], l = sl[0], t = st[0];
    const bool any = m != -INFINITY;
    const float lz = any ? logf(l) : 0.0f;
    if (tid == 0) {
        const int64_t tgt = a.targets[r];
        if (tgt >= v) atomicOr(&g_lp_err, ERRBIT_INDEX);
        float lp = 0.0f;
        if (tgt >= 0 && tgt < v) lp = any ? (logit<F32>(row, tgt) - m) - lz : -INFINITY;
        a.logprobs[r] = lp;
        a.entropy[r] = any ? lz - t / l : 0.0f;
    }
    // top alternatives: k times the best one after the last in the order
    float px = INFINITY;
    int32_t pi = -1;
    for (int64_t n = 0; n < a.top; ++n) {
        __syncthreads();
        float bx = -INFINITY;
        int32_t bi = 0x7fffffff;
        for (int64_t i = tid; i < v; i += kLpThreads) {
            const float x = logit<F32>(row, i);
            const bool after = x < px || (x == px && i > pi);
            if (after && (x > bx || (x == bx && i < bi))) bx = x, bi = static_cast<int32_t>(i);
        }
        sm[tid] = bx, si[tid] = bi;
        __syncthreads();
        for (int s = kLpThreads / 2; s > 0; s >>= 1) {
            if (tid < s) {
                if (sm[tid + s] > sm[tid] || (sm[tid + s] == sm[tid] && si[tid + s] < si[tid]))
                    sm[tid] = sm[tid + s], si[tid] = si[tid + s];
            }
            __syncthreads();
        }
        px = sm[0], pi = si[0];
        if (tid == 0) {
            a.top_ids[r * a.top + n] = pi;
            a.top_logprobs[r * a.top + n] = any ? (px - m) - lz : -INFINITY;
        }
    }
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs &a, cudaStream_t stream) {
    if (a.f32) logprobs_kernel<true><<<static_cast<unsigned>(a.rows), kLpThreads, 0, stream>>>(a);
    else logprobs_kernel<false><<<static_cast<unsigned>(a.rows), kLpThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

uint32_t take_logprobs_error() {
    uint32_t v = 0;
    if (cudaMemcpyFromSymbol(&v, g_lp_err, sizeof v) != cudaSuccess) return 0xFFFFFFFFu;
    const uint32_t zero = 0;
    cudaMemcpyToSymbol(g_lp_err, &zero, sizeof zero);
    return v;
}

}  // namespace fp8bs
