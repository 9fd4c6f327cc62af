// serving.cuh -- helpers of the serving step's kernels (kvplan.cu, kv4.cu,
// logprobs.cu) beside those of common.cuh, which stays with the linears: the
// DRAM traffic reported for a linear's kernel is the captured one only while
// its sources, common.cuh among them, are those that were captured.
#pragma once

#include "common.cuh"

namespace fp8bs {

// Beside common.cuh's bits of a kernel's error word.
constexpr uint32_t ERRBIT_CAPACITY = 1u << 5;  // a request found no free cache blocks

// Loads of what the kernels before this one wrote.  A kernel here may be on
// the GPU while they still write (programmatic dependent launch), so it does
// not promise, as ld.global.nc and __ldg do, that nothing changes while it
// lives: griddepcontrol.wait orders ordinary loads.  Not kept in L1.
__device__ __forceinline__ uint4 ld_v4(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ void ld_v8(const void *p, uint32_t (&v)[8]) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "l"(p));
}

// Four rows of a 2-D map whose box is one row, from column x: row[0 .. 3] one
// after the other in shared memory (128-byte aligned).  A row out of range
// reads zeros.
__device__ __forceinline__ void tma_gather4_2d(void *smem_dst, const CUtensorMap *map, uint64_t *bar, int32_t x,
                                               const int32_t (&row)[4]) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(row[0]), "r"(row[1]), "r"(row[2]),
        "r"(row[3])
        : "memory");
}

// The two halves of a cluster barrier apart.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Eight e2m1 codes (one 32-bit word, code i in bits 4i .. 4i + 3) -> four
// exact f16 pairs (codes 2i, 2i + 1; the lower code in the lower half).
__device__ __forceinline__ void e2m1x8_to_f16x2x4(uint32_t word, uint32_t (&out)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3])
        : "r"(word));
}

// Eight fp32 values -> eight e2m1 codes (round to nearest even, saturating
// to +-6), value i in bits 4i .. 4i + 3.
__device__ __forceinline__ uint32_t f32x8_to_e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Two e4m3 codes (the low 16 bits) -> one exact f16 pair, lower code first.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
    uint32_t r;
    asm("{\n\t.reg .b16 l;\n\tcvt.u16.u32 l, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(codes));
    return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t v) {
    float lo, hi;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(v));
    return make_float2(lo, hi);
}

// Two fp32 values -> one bf16 pair (round to nearest even), `lo` in the lower half.
__device__ __forceinline__ uint32_t f32x2_to_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace fp8bs
