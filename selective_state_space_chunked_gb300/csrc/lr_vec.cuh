// lr_vec.cuh -- neighbouring values as one load, and the activation that the
// memory-bound kernels share.
#pragma once

#include "lr_device.cuh"

namespace lr {
namespace {

// silu in fp32: x / (1 + e^-x).  The fast division gives 0 for divisors past
// 2^126, where the quotient is below 1.2e-36.
__device__ __forceinline__ float silu_f(float x) { return __fdividef(x, 1.0f + ex2_approx(-x * kLog2e)); }
__device__ __forceinline__ float2 pair(const float *v) { return make_float2(v[0], v[1]); }

// N neighbouring values as one load
template <typename IO, int N_> struct Vec;
template <> struct Vec<float, 4> {
    static constexpr int N = 4;
    using Raw = float4;
    __device__ __forceinline__ static void widen(const Raw &u, float *v) { v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w; }
    __device__ __forceinline__ static Raw narrow(const float *v) { return make_float4(v[0], v[1], v[2], v[3]); }
};
__device__ __forceinline__ void widen2(uint32_t w, float *v) {
    v[0] = __uint_as_float(w << 16), v[1] = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ uint32_t narrow2(const float *v) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(v[0], v[1]);
    return *reinterpret_cast<const uint32_t *>(&t);
}
template <> struct Vec<__nv_bfloat16, 8> {
    static constexpr int N = 8;
    using Raw = uint4;
    __device__ __forceinline__ static void widen(const Raw &u, float *v) {
        widen2(u.x, v), widen2(u.y, v + 2), widen2(u.z, v + 4), widen2(u.w, v + 6);
    }
    __device__ __forceinline__ static Raw narrow(const float *v) {
        return make_uint4(narrow2(v), narrow2(v + 2), narrow2(v + 4), narrow2(v + 6));
    }
};
template <> struct Vec<__nv_bfloat16, 4> {
    static constexpr int N = 4;
    using Raw = uint2;
    __device__ __forceinline__ static void widen(const Raw &u, float *v) { widen2(u.x, v), widen2(u.y, v + 2); }
    __device__ __forceinline__ static Raw narrow(const float *v) { return make_uint2(narrow2(v), narrow2(v + 2)); }
};
// silu of a pair
__device__ __forceinline__ float2 silu2_f(float2 x) {
    const float2 e = __fmul2_rn(x, make_float2(-kLog2e, -kLog2e));
    const float2 d = __fadd2_rn(make_float2(ex2_approx(e.x), ex2_approx(e.y)), make_float2(1.0f, 1.0f));
    return __fmul2_rn(x, make_float2(rcp_approx(d.x), rcp_approx(d.y)));
}

// a value at a time
template <> struct Vec<float, 1> {
    static constexpr int N = 1;
    using Raw = float;
    __device__ __forceinline__ static void widen(Raw u, float *v) { v[0] = u; }
    __device__ __forceinline__ static Raw narrow(const float *v) { return v[0]; }
};
template <> struct Vec<__nv_bfloat16, 1> {
    static constexpr int N = 1;
    using Raw = uint16_t;
    __device__ __forceinline__ static void widen(Raw u, float *v) { v[0] = __uint_as_float(uint32_t(u) << 16); }
    __device__ __forceinline__ static Raw narrow(const float *v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v[0])); }
};

}  // namespace
}  // namespace lr
