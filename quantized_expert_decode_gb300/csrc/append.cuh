// append.cuh — what the kernels that append to a paged cache share: the turn of a pair by its position, and the
// rounding to the cache's type. Internal to libcolimoe.
//
// Pair i of a head turns by p * inv_freq[i]. In units of a full turn that is p * (inv_freq[i] / 2 pi), and only its
// fraction counts. fp32 has no fraction left at far positions, so inv_freq / 2 pi is taken as a 64-bit
// fixed-point fraction of a turn (the 24-bit mantissa times 64 bits of 1 / 2 pi) and the product with the integer p
// wraps modulo one turn by itself: off by p * 2^-64 turns. sincospi then takes the fraction as a float.
#pragma once

#include "act.cuh"

namespace colimoe {

// f / 2 pi as a fraction of a turn in units of 2^-64, modulo one turn
__device__ __forceinline__ unsigned long long turns_per_step(float f) {
    constexpr unsigned long long kR = 0xa2f9836e4e441529ull;  // 2^66 / 2 pi
    const unsigned bits = __float_as_uint(f), e = (bits >> 23) & 0xff;
    const unsigned long long m = e ? (bits & 0x7fffff) | 0x800000 : 0;  // f = m * 2^(e - 150); below 2^-126: 0
    const unsigned long long hi = __umul64hi(m, kR), lo = m * kR;
    const int s = 152 - (int)e;
    unsigned long long c;
    if (s >= 128) c = 0;
    else if (s >= 64) c = hi >> (s - 64);
    else if (s > 0) c = (hi << (64 - s)) | (lo >> s);
    else c = s > -64 ? lo << -s : 0;
    return (bits >> 31) ? 0ull - c : c;
}

__device__ __forceinline__ float2 turn(int p, float f) {
    const long long t = (long long)((unsigned long long)(long long)p * turns_per_step(f));
    float s, c;
    sincospif((float)t * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
    if (!isfinite(f)) s = c = __int_as_float(0x7fffffff);
    return make_float2(c, s);
}

// Division by an e4m3 scale: 1 / scale = r + rest, with r the largest float that is no larger in size, so that
// x * rest + x * r in one rounding is the quotient rounded to fp32, but for 2^-22 of its last bit. (The product with a
// rounded reciprocal puts some values next to a border between two e4m3 values on its other side.) r and rest have one
// sign and neither is 0, so infinities stay infinite. Scales far from 1, whose reciprocal would leave fp32's range, are
// brought nearer by a power of two, and x with them. Two packed instructions for two values, as many as the product
// alone took: 16,411 tokens of 64 + 2 x 8 bf16 heads 103.5 us against 105, 2048 of 32 + 2 x 32 heads 18.1 against 16.9
// (there each item's r and rest count); the plain division 105.7 and 21.8.
struct Divisor {
    float r, rest, shift;
    __device__ __forceinline__ explicit Divisor(float scale) {
        shift = fabsf(scale) < 0x1p-60f ? 0x1p100f : fabsf(scale) > 0x1p60f ? 0x1p-100f : 1.f;
        const float s = scale * shift;
        r = 1.f / s;
        float left = fmaf(-s, r, 1.f);
        if (left < 0.f) {
            r = __uint_as_float(__float_as_uint(r) - 1);
            left = fmaf(-s, r, 1.f);
        }
        rest = left > 0.f ? left * r : r * 0x1p-60f;
    }
};

// N values in the cache's type; e4m3 holds value / scale and is converted in pairs
template <typename C, int N>
__device__ __forceinline__ void to_cache(C (&to)[N], const float (&x)[N], const Divisor &by) {
#pragma unroll
    for (int j = 0; j < N; j++) to[j] = from_f32<C>(x[j]);
}
template <int N>
__device__ __forceinline__ void to_cache(__nv_fp8_e4m3 (&to)[N], const float (&v)[N], const Divisor &by) {
    float x[N];
#pragma unroll
    for (int j = 0; j < N; j++) x[j] = v[j];
    if (by.shift != 1.f) {
#pragma unroll
        for (int j = 0; j < N; j++) x[j] *= by.shift;
    }
    if constexpr (N % 2 == 0) {
        const float2 r = make_float2(by.r, by.r), rest = make_float2(by.rest, by.rest);
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const float2 a = make_float2(x[j], x[j + 1]);
            const __nv_fp8x2_storage_t p = __nv_cvt_float2_to_fp8x2(__ffma2_rn(a, r, __fmul2_rn(a, rest)), __NV_SATFINITE, __NV_E4M3);
            to[j].__x = (__nv_fp8_storage_t)p;
            to[j + 1].__x = (__nv_fp8_storage_t)(p >> 8);
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; j++) to[j] = from_f32<__nv_fp8_e4m3>(fmaf(x[j], by.r, x[j] * by.rest));
    }
}

// whether rows at p, `stride` elements apart, let runs of `run` elements be moved in their widest words
inline bool multiple(const void *p, int64_t stride, int act_bytes, int run) {
    const int64_t bytes = (int64_t)run * act_bytes;
    const int64_t a = bytes % 16 == 0 ? 16 : bytes;
    return reinterpret_cast<uintptr_t>(p) % a == 0 && (stride * act_bytes) % a == 0;
}

}  // namespace colimoe
