// act.cuh — activation and cache element types of the layer operators: runs of elements loaded from
// and stored to memory as fp32 values. Internal to libcolimoe.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace colimoe {

// bytes of the widest access that takes N elements of S bytes: 16, 8, 4, 2 or 1
template <int S, int N>
struct RunBytes {
    static constexpr int total = S * N;
    static constexpr int value = total % 16 == 0 ? 16 : total % 8 == 0 ? 8 : total % 4 == 0 ? 4 : total % 2 == 0 ? 2 : 1;
};

template <int B> struct Word;
template <> struct Word<16> { using type = uint4; };
template <> struct Word<8> { using type = uint2; };
template <> struct Word<4> { using type = uint32_t; };
template <> struct Word<2> { using type = uint16_t; };
template <> struct Word<1> { using type = uint8_t; };

// N elements of T in registers, moved in the widest words that divide them (p aligned to that)
template <typename T, int N>
struct alignas(RunBytes<sizeof(T), N>::value) Run {
    T e[N];
    using W = typename Word<RunBytes<sizeof(T), N>::value>::type;
    static constexpr int kWords = sizeof(T) * N / sizeof(W);
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < kWords; i++) reinterpret_cast<W *>(e)[i] = reinterpret_cast<const W *>(p)[i];
    }
    __device__ __forceinline__ void store(T *p) const {
#pragma unroll
        for (int i = 0; i < kWords; i++) reinterpret_cast<W *>(p)[i] = reinterpret_cast<const W *>(e)[i];
    }
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_fp8_e4m3 x) { return (float)x; }

// one rounding, to nearest even
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
// saturated to +-448, NaN stays NaN
template <> __device__ __forceinline__ __nv_fp8_e4m3 from_f32<__nv_fp8_e4m3>(float x) {
    __nv_fp8_e4m3 r;
    r.__x = __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
    return r;
}

}  // namespace colimoe
