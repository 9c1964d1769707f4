// Pairs of floats (two elements are worked on in one instruction) and 16-byte vectors of them.
#pragma once

#include "m3_common.cuh"

namespace m3 {

// 16 bytes of T as pairs of floats (two elements are worked on in one instruction)
template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 2;
    static __device__ __forceinline__ void unpack(const uint4& v, float2* f) {
        f[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
        f[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    static __device__ __forceinline__ void store(float* p, const float2* f) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(const uint4& v, float2* f) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float2* f) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(f[i].x, f[i].y);
            w[i] = *reinterpret_cast<const uint32_t*>(&v);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 mul2(const float2& a, const float2& b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(const float2& a, const float2& b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(const float2& a, const float2& b, const float2& c) { return __ffma2_rn(a, b, c); }

// 1 / (1 + e^-v) of two elements, with the hardware's 2^x and 1 / x (1 + 2^x lies in [1, inf], so that
// denormals need no care).
__device__ __forceinline__ float2 sigmoid2(const float2& v) {
    float2 e = mul2(v, both(-1.4426950408889634f));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.x));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.y));
    e = add2(e, both(1.f));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.x));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.y));
    return e;
}

}  // namespace m3
