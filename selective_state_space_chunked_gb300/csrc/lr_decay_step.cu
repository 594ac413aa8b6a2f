// lr_decay_step.cu -- one token of the decayed linear attention:
//   S = a S + v k^T,  o = scale S q,  a = exp(a_log[h] + g[b, h]).
//
// The state is read and written once: 8 dk dv bytes per (batch row, head)
// against 4 dk dv operations, so the kernel is bound by memory bandwidth (by
// the launch and one trip to memory at one sequence).  TL lanes share a state
// row, each holding groups of four consecutive keys; a warp has its R rows'
// loads in flight before the first is used.
#include "lr_decay.cuh"

namespace lr {
namespace {

template <typename IO>
__device__ __forceinline__ float4 step_ld4(const IO *p);
template <>
__device__ __forceinline__ float4 step_ld4<float>(const float *p) {
    return *reinterpret_cast<const float4 *>(p);
}
template <>
__device__ __forceinline__ float4 step_ld4<__nv_bfloat16>(const __nv_bfloat16 *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                       __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}

constexpr int kStepT = 128;

__device__ __forceinline__ float decay_of(float l) { return expf(l); }

// VEC rows: dk % 4 == 0 and dk <= 4 TL (one group of four keys per lane).
// A warp takes 32 / TL rows at a time, R times.
template <typename IO, int TL, int R>
__global__ void __launch_bounds__(kStepT)
    decay_step_kernel(const IO *__restrict__ q, const IO *__restrict__ k, const IO *__restrict__ v,
                      const float *__restrict__ a_log, const IO *__restrict__ g, float scale,
                      const float *S_in, float *S_out, IO *__restrict__ o, int64_t BH, int H, int Hk, int dk,
                      int dv, int tiles) {
    constexpr int RPW = 32 / TL;          // rows a warp holds at once
    constexpr int ROWS = RPW * R;         // rows per warp
    const int lane = threadIdx.x & 31, sub = lane / TL, j = 4 * (lane % TL);
    const int64_t w = int64_t(blockIdx.x) * (kStepT / 32) + (threadIdx.x >> 5);
    if (w >= BH * tiles) return;   // warp-uniform
    const int64_t bh = w / tiles;
    const int row0 = int(w - bh * tiles) * ROWS;
    const int64_t b = bh / H;
    const int h = int(bh - b * H), hk = h / (H / Hk);
    const bool col = j < dk;
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int64_t base = bh * dv;
    float4 s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = row0 + r * RPW + sub;
        s[r] = S_in != nullptr && col && i < dv ? __ldcs(reinterpret_cast<const float4 *>(S_in + (base + i) * dk + j))
                                                : zero;
    }
    const int64_t kat = (b * Hk + hk) * dk + j;
    const float4 k4 = col ? step_ld4(k + kat) : zero, q4 = col ? step_ld4(q + kat) : zero;
    float l = a_log != nullptr ? a_log[h] : 0.0f;
    if (g != nullptr) l += Io<IO>::to_f(g[bh]);
    const float a = decay_of(l);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = row0 + r * RPW + sub;
        const bool in = i < dv;
        const float vi = in ? Io<IO>::to_f(v[base + i]) : 0.0f;
        s[r] = make_float4(fmaf(a, s[r].x, vi * k4.x), fmaf(a, s[r].y, vi * k4.y), fmaf(a, s[r].z, vi * k4.z),
                           fmaf(a, s[r].w, vi * k4.w));
        if (in && col) __stcs(reinterpret_cast<float4 *>(S_out + (base + i) * dk + j), s[r]);
        float acc = fmaf(s[r].x, q4.x, fmaf(s[r].y, q4.y, fmaf(s[r].z, q4.z, s[r].w * q4.w)));
#pragma unroll
        for (int m = TL / 2; m >= 1; m >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, m);
        if (in && lane % TL == 0) o[base + i] = Io<IO>::from_f(scale * acc);
    }
}

// any dk: one warp per row
template <typename IO>
__global__ void __launch_bounds__(kStepT)
    decay_step_any_kernel(const IO *__restrict__ q, const IO *__restrict__ k, const IO *__restrict__ v,
                          const float *__restrict__ a_log, const IO *__restrict__ g, float scale,
                          const float *S_in, float *S_out, IO *__restrict__ o, int64_t BH, int H, int Hk,
                          int dk, int dv) {
    const int64_t row = int64_t(blockIdx.x) * (kStepT / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= BH * dv) return;   // warp-uniform
    const int64_t bh = row / dv, b = bh / H;
    const int h = int(bh - b * H), hk = h / (H / Hk);
    float l = a_log != nullptr ? a_log[h] : 0.0f;
    if (g != nullptr) l += Io<IO>::to_f(g[bh]);
    const float a = decay_of(l), vi = Io<IO>::to_f(v[row]);
    const IO *kb = k + (b * Hk + hk) * dk, *qb = q + (b * Hk + hk) * dk;
    float acc = 0.0f;
#pragma unroll 4
    for (int j = lane; j < dk; j += 32) {
        const float s0 = S_in != nullptr ? S_in[row * dk + j] : 0.0f;
        const float s = fmaf(a, s0, vi * Io<IO>::to_f(kb[j]));
        S_out[row * dk + j] = s;
        acc = fmaf(s, Io<IO>::to_f(qb[j]), acc);
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, m);
    if (lane == 0) o[row] = Io<IO>::from_f(scale * acc);
}

template <typename IO>
int step_io(const IO *q, const IO *k, const IO *v, const float *a_log, const IO *g, float scale,
            const float *S_in, float *S_out, IO *o, int64_t B, int64_t H, int64_t Hk, int64_t dk, int64_t dv,
            cudaStream_t s) {
    const int64_t BH = B * H;
    int sms = 0;
    if (device_sm_count(&sms) != LR_OK) return LR_ERR_CUDA;
    auto go = [&](auto kern, int rows) -> int {
        const int64_t tiles = (dv + rows - 1) / rows;
        const int64_t grid = (BH * tiles + kStepT / 32 - 1) / (kStepT / 32);
        if (grid > INT32_MAX) return LR_ERR_UNSUPPORTED;
        kern<<<unsigned(grid), kStepT, 0, s>>>(q, k, v, a_log, g, scale, S_in, S_out, o, BH, int(H), int(Hk),
                                               int(dk), int(dv), int(tiles));
        return cudaGetLastError() == cudaSuccess ? LR_OK : LR_ERR_CUDA;
    };
    if (dk % 4 == 0 && dk <= 128) {
        // four rows in flight per lane once that still fills the SMs
        const bool deep = BH * dv * dk >= int64_t(sms) * 64 * 512;
        if (dk <= 32) return deep ? go(decay_step_kernel<IO, 8, 4>, 16) : go(decay_step_kernel<IO, 8, 1>, 4);
        if (dk <= 64) return deep ? go(decay_step_kernel<IO, 16, 4>, 8) : go(decay_step_kernel<IO, 16, 1>, 2);
        return deep ? go(decay_step_kernel<IO, 32, 4>, 4) : go(decay_step_kernel<IO, 32, 1>, 1);
    }
    const int64_t grid = (BH * dv + kStepT / 32 - 1) / (kStepT / 32);
    if (grid > INT32_MAX) return LR_ERR_UNSUPPORTED;
    decay_step_any_kernel<IO><<<unsigned(grid), kStepT, 0, s>>>(q, k, v, a_log, g, scale, S_in, S_out, o, BH, int(H),
                                                                int(Hk), int(dk), int(dv));
    return cudaGetLastError() == cudaSuccess ? LR_OK : LR_ERR_CUDA;
}

}  // namespace

int decay_step_launch(const void *q, const void *k, const void *v, const float *a_log, const void *g,
                      float scale, const float *S_in, float *S_out, void *o, int64_t B, int64_t H, int64_t Hk,
                      int64_t dk, int64_t dv, int io_bf16, cudaStream_t stream) {
    if (B == 0) return LR_OK;
    using bf = __nv_bfloat16;
    return io_bf16 ? step_io<bf>(static_cast<const bf *>(q), static_cast<const bf *>(k), static_cast<const bf *>(v),
                                 a_log, static_cast<const bf *>(g), scale, S_in, S_out, static_cast<bf *>(o), B, H,
                                 Hk, dk, dv, stream)
                   : step_io<float>(static_cast<const float *>(q), static_cast<const float *>(k),
                                    static_cast<const float *>(v), a_log, static_cast<const float *>(g), scale, S_in,
                                    S_out, static_cast<float *>(o), B, H, Hk, dk, dv, stream);
}

}  // namespace lr
