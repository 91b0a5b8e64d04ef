// Device helpers shared by the tensor-core attention kernels: exponentials,
// NaN-keeping maxima, packed fp32 pairs, bf16 packing and the shared-memory
// descriptors of 64-column bf16 tiles; and the host side of their TMA maps.
#pragma once

#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "fma_exp2.cuh"
#include "tc_prims.cuh"

namespace ttt {
namespace attn {

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// max that returns NaN if an operand is NaN (fmaxf would drop it); two- and three-input forms
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Pairs of fp32 values in one 64-bit register pair, for the packed f32x2 arithmetic of sm_100
// (one instruction for two elements).
__device__ __forceinline__ uint64_t f2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void f2_split(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t f2_sub(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Where the exponentials on the FMA pipe hold x: there the polynomial is just above 1 and the exponent field reaches
// zero, so what comes out is below 2^-139 and becomes +0 as bf16.  A weight has to: at the clamp of -125 a masked
// score (-infinity) got 2^-125, which is nothing beside a row's sum but 8 times a value of 3e38.  Between -126 and
// here the result falls to that without a jump, off by less than 2^-126.
// A NaN comes out as 2^128 - 2^104 (the bits 0x7fffffff that the arithmetic makes of any NaN, plus themselves shifted
// left by 23), an infinity once it is bf16: the callers look for NaN in their rows' maxima, statistics or inputs.
constexpr float kLowest = -126.99985f;

// 2^x0, 2^x1 on the FMA pipe: a cubic of fma_exp2.cuh's kind (coefficients c0 .. c3) on a pair, with the packed f32x2
// arithmetic.  x <= 8 here; +0 as bf16 from kLowest on.
__device__ __forceinline__ void ex2_cubic2(uint64_t x, float c0, float c1, float c2, float c3, float& p0, float& p1) {
    float x0, x1;
    f2_split(x, x0, x1);
    x = f2(max_nan(x0, kLowest), max_nan(x1, kLowest));
    using namespace fexp;
    const uint64_t shift = f2(kShift, kShift);
    const uint64_t t = f2_add(x, shift);
    const uint64_t f = f2_sub(x, f2_sub(t, shift));
    uint64_t p = f2_fma(f2(c3, c3), f, f2(c2, c2));
    p = f2_fma(p, f, f2(c1, c1));
    p = f2_fma(p, f, f2(c0, c0));
    float t0, t1, q0, q1;
    f2_split(t, t0, t1);
    f2_split(p, q0, q1);
    p0 = scale_by_rint(q0, t0);
    p1 = scale_by_rint(q1, t1);
}

// The same with fma_exp2.cuh's quartic (relative error 2.7e-6), for sums that are kept in fp32; +0 as bf16 from kLowest on.
__device__ __forceinline__ void ex2_poly2_fine(uint64_t x, float& p0, float& p1) {
    float x0, x1;
    f2_split(x, x0, x1);
    x = f2(max_nan(x0, kLowest), max_nan(x1, kLowest));
    using namespace fexp;
    const uint64_t shift = f2(kShift, kShift);
    const uint64_t t = f2_add(x, shift);
    const uint64_t f = f2_sub(x, f2_sub(t, shift));
    uint64_t p = f2_fma(f2(kC4_4, kC4_4), f, f2(kC4_3, kC4_3));
    p = f2_fma(p, f, f2(kC4_2, kC4_2));
    p = f2_fma(p, f, f2(kC4_1, kC4_1));
    p = f2_fma(p, f, f2(kC4_0, kC4_0));
    float t0, t1, q0, q1;
    f2_split(t, t0, t1);
    f2_split(p, q0, q1);
    p0 = scale_by_rint(q0, t0);
    p1 = scale_by_rint(q1, t1);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint64_t kmajor_desc(const uint8_t* p) { return tc::smem_desc(tc::smem_u32(p), 16, 1024); }
// MN-major (V): one 64-wide block, 8-row groups 1 KB apart; K step of 16 keys = 2048 bytes.
__device__ __forceinline__ uint64_t mnmajor_desc(const uint8_t* p) { return tc::smem_desc(tc::smem_u32(p), 16384, 1024); }

// ------------------------------------------------------------------ host
inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// bf16 [T rows x cols columns], row stride ld elements; boxes of 64 columns x 128 rows, 128-byte swizzle
// (rows past T read as zero).
inline bool make_map(CUtensorMap* m, const void* base, int T, int cols, long long ld) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)T};
    cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
    cuuint32_t box[2] = {64, 128};
    cuuint32_t es[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace attn
}  // namespace ttt
