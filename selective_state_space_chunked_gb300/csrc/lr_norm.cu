// lr_norm.cu -- group normalisation with an activation, channels last:
//   per row and group of d = C / G channels
//     m = mean(x), s2 = mean((x - m)^2), n = gamma (x - m) / sqrt(s2 + eps) + beta
//     y = act(n) silu(z)          act = identity or silu; no z: no gate
//
// Every value is read once and written once, so memory bandwidth bounds the
// kernel.  A group stays in the registers of the lanes that share it: the
// mean, then the centred squares (no cancellation), then the output.
#include "lr_decay.cuh"

namespace lr {
namespace {

__device__ __forceinline__ float silu_f(float x) { return x / (1.0f + expf(-x)); }

template <typename IO> struct Vec16;
template <> struct Vec16<float> {
    static constexpr int N = 4;
    __device__ __forceinline__ static void load(const float *p, float *v) {
        const float4 u = __ldcs(reinterpret_cast<const float4 *>(p));
        v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
    }
    __device__ __forceinline__ static void store(float *p, const float *v) {
        __stcs(reinterpret_cast<float4 *>(p), make_float4(v[0], v[1], v[2], v[3]));
    }
};
template <> struct Vec16<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ __forceinline__ static void load(const __nv_bfloat16 *p, float *v) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(p));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ static void store(__nv_bfloat16 *p, const float *v) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&t);
        }
        __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
    }
};

// any sizes: one block per (row, group), three passes over the group
template <typename IO>
__global__ void __launch_bounds__(128)
    group_norm_any_kernel(const IO *__restrict__ x, const IO *__restrict__ z, const float *__restrict__ gamma,
                          const float *__restrict__ beta, IO *__restrict__ y, int64_t NG, int64_t C, int64_t G,
                          int64_t d, float eps, int act) {
    __shared__ float red[4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto total = [&](float v) -> float {
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
        __syncthreads();
        if (lane == 0) red[warp] = v;
        __syncthreads();
        return (red[0] + red[1]) + (red[2] + red[3]);
    };
    for (int64_t r = blockIdx.x; r < NG; r += gridDim.x) {
        const int64_t row = r / G, gi = r - row * G;
        const int64_t at = row * C + gi * d;
        float s = 0.0f;
        for (int64_t i = threadIdx.x; i < d; i += 128) s += Io<IO>::to_f(x[at + i]);
        const float mean = total(s) / float(d);
        s = 0.0f;
        for (int64_t i = threadIdx.x; i < d; i += 128) {
            const float t = Io<IO>::to_f(x[at + i]) - mean;
            s = fmaf(t, t, s);
        }
        const float rs = 1.0f / sqrtf(total(s) / float(d) + eps);
        for (int64_t i = threadIdx.x; i < d; i += 128) {
            const int64_t c = gi * d + i;
            float n = (Io<IO>::to_f(x[at + i]) - mean) * rs;
            if (gamma != nullptr) n *= gamma[c];
            if (beta != nullptr) n += beta[c];
            if (act == LR_ACT_SILU) n = silu_f(n);
            if (z != nullptr) n *= silu_f(Io<IO>::to_f(z[at + i]));
            y[at + i] = Io<IO>::from_f(n);
        }
    }
}

template <typename IO>
int norm_io(const IO *x, const IO *z, const float *gamma, const float *beta, IO *y, int64_t N, int64_t C,
            int64_t G, float eps, int act, cudaStream_t s) {
    const int64_t NG = N * G;
    const unsigned grid = unsigned(NG < (1 << 20) ? NG : (1 << 20));
    group_norm_any_kernel<IO><<<grid, 128, 0, s>>>(x, z, gamma, beta, y, NG, C, G, C / G, eps, act);
    return cudaGetLastError() == cudaSuccess ? LR_OK : LR_ERR_CUDA;
}

}  // namespace

int group_norm_act_launch(const void *x, const void *z, const float *gamma, const float *beta, void *y,
                          int64_t N, int64_t C, int64_t G, float eps, int act, int io_bf16, cudaStream_t stream) {
    if (N == 0 || C == 0) return LR_OK;
    using bf = __nv_bfloat16;
    return io_bf16 ? norm_io<bf>(static_cast<const bf *>(x), static_cast<const bf *>(z), gamma, beta,
                                 static_cast<bf *>(y), N, C, G, eps, act, stream)
                   : norm_io<float>(static_cast<const float *>(x), static_cast<const float *>(z), gamma, beta,
                                    static_cast<float *>(y), N, C, G, eps, act, stream);
}

}  // namespace lr
