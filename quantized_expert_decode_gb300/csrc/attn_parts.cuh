// attn_parts.cuh — what the streaming attention kernels share: asynchronous copies, the conversion of cached and
// query elements to the matrix types. Internal to libcolimoe.
#pragma once

#include "act.cuh"
#include "colilayer.h"

namespace colimoe {

namespace attn {

// `bytes` of 16 are copied, the rest are zeros (of 0, src is not read)
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// two e4m3 values to two f16 values (exact; NaN stays NaN)
__device__ __forceinline__ uint32_t widen(uint32_t two_bytes) {
    uint32_t y;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(y) : "r"(two_bytes));
    return y;
}
__device__ __forceinline__ uint32_t widen_hi(uint32_t four_bytes) {
    uint32_t y;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(y) : "r"(four_bytes));
    return y;
}

// the leading part of (a, b) in the matrix type as two packed 16-bit values; a, b keep the rest
template <int FMT>
__device__ __forceinline__ uint32_t take_part(float &a, float &b) {
    uint32_t r;
    if (FMT == COLI_KV_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        a -= __low2float(h);
        b -= __high2float(h);
        r = *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        a -= __low2float(h);
        b -= __high2float(h);
        r = *reinterpret_cast<const uint32_t *>(&h);
    }
    return r;
}

// the same with the rest of both in one packed subtraction
template <int FMT>
__device__ __forceinline__ uint32_t take_part2(float2 &x) {
    uint32_t r;
    float2 h;
    if (FMT == COLI_KV_BF16) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x.x, x.y);
        r = *reinterpret_cast<const uint32_t *>(&b);
        h = make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
    } else {
        const __half2 b = __floats2half2_rn(x.x, x.y);
        r = *reinterpret_cast<const uint32_t *>(&b);
        h = __half22float2(b);
    }
    x = __fadd2_rn(x, make_float2(-h.x, -h.y));
    return r;
}

__device__ __forceinline__ float load_act(const void *p, int64_t i, int act) {
    return act == COLI_ACT_F32 ? ((const float *)p)[i]
           : act == COLI_ACT_BF16 ? to_f32(((const __nv_bfloat16 *)p)[i])
                                  : to_f32(((const __half *)p)[i]);
}

}  // namespace attn

}  // namespace colimoe
