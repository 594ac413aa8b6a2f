// lr_decay_step.cu -- one token of the decayed linear attention:
//   S = a S + v k^T,  o = scale S q,  a = exp(a_log[h] + g[b, h]).
//
// The state is read and written once: 8 dk dv bytes per (batch row, head)
// against 5 dk dv operations, so the kernel is bound by memory bandwidth (by
// the launch and one trip to memory at one sequence).  TL lanes share a state
// row, each holding groups of four consecutive keys; a warp has its R rows'
// loads in flight before the first is used.  fp32 throughout; o is rounded once.
//
// Measured back to back in one graph, states in turn (bf16 H16 d128): B64 22.1 us,
// 90 % of the copy bandwidth; B32 12.5; B8 4.6; B1 2.35.  fp32 B32 H16 dk256 dv128
// 21.2 us, 93 %.
//   four rows of a warp in flight against one: B64 23 us against 35, B8 5.4
//   against 6.2; at B1, where it leaves fewer warps, 2.4 against 2.3.  Eight: B64
//   22.6 against 23.2, but B1 3.1
//   blocks of 64 threads against 128: B64 22.6 us against 23.2, B32 12.9
//   against 13.1, B1 2.6 against 2.4; of 256: 23.7
//   streaming loads and stores, the state being larger than the cache over a
//   model's layers: B64 23.2 us against 23.5
//   launched while the kernel before it drains (the kernel waits for that one's
//   results): calls one after another B64 24.6 -> 22.5 us, B8 7.8 -> 5.6; a step and
//   a gated norm at B8 H16 d128 10.3 -> 7.5
//   dk up to 512 in the same form: B32 H16 dk192 18.7 us against 36 with a row
//   read element by element, which stays for dk that is no multiple of four
#include "lr_decay.cuh"

namespace lr {
namespace {

// The inputs are plain pointers: a const __restrict__ one says that its data stays
// the same while the kernel lives, and a kernel that starts early lives while the
// one before it may still be writing them.  So all are read before the first store
// (B64 24.6 us with v read between the stores).

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

constexpr int kStepT = 64;

// dk % 4 == 0 and dk <= 4 TL V: V groups of four keys per lane.
// A warp takes 32 / TL rows at a time, R times.  20 blocks per SM leave 48 registers
// (B64 22.9 us with 52).
template <typename IO, int TL, int R, int V>
__global__ void __launch_bounds__(kStepT, V == 1 ? 20 : V == 2 ? 1 : 12)
    decay_step_kernel(const IO *q, const IO *k, const IO *v, const float *a_log, const IO *g, float scale,
                      const float *S_in, float *S_out, IO *o, int64_t BH, int H, int Hk, int dk, int dv, int tiles) {
    constexpr int RPW = 32 / TL;          // rows a warp holds at once
    constexpr int ROWS = RPW * R;         // rows per warp
    const int lane = threadIdx.x & 31, sub = lane / TL, j0 = 4 * (lane % TL);
    launch_dependents();
    grid_dependency_wait();
    const int64_t w = int64_t(blockIdx.x) * (kStepT / 32) + (threadIdx.x >> 5);
    if (w >= BH * tiles) return;   // warp-uniform
    const int64_t bh = w / tiles;
    const int row0 = int(w - bh * tiles) * ROWS;
    const int64_t b = bh / H;
    const int h = int(bh - b * H), hk = h / (H / Hk);
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int64_t base = bh * dv;
    float4 s[R][V];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = row0 + r * RPW + sub;
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int j = j0 + 4 * TL * u;
            s[r][u] = S_in != nullptr && j < dk && i < dv
                          ? __ldcs(reinterpret_cast<const float4 *>(S_in + (base + i) * dk + j))
                          : zero;
        }
    }
    float4 k4[V], q4[V];
#pragma unroll
    for (int u = 0; u < V; ++u) {
        const int j = j0 + 4 * TL * u;
        const int64_t kat = (b * Hk + hk) * dk + j;
        k4[u] = j < dk ? step_ld4(k + kat) : zero;
        q4[u] = j < dk ? step_ld4(q + kat) : zero;
    }
    float vr[R];   // before the first store, which may be to anywhere
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = row0 + r * RPW + sub;
        vr[r] = i < dv ? Io<IO>::to_f(v[base + i]) : 0.0f;
    }
    float l = a_log != nullptr ? a_log[h] : 0.0f;
    if (g != nullptr) l += Io<IO>::to_f(g[bh]);
    const float a = expf(l);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = row0 + r * RPW + sub;
        const bool in = i < dv;
        const float vi = vr[r];
        float acc = 0.0f;
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int j = j0 + 4 * TL * u;
            float4 &x = s[r][u];
            x = make_float4(fmaf(a, x.x, vi * k4[u].x), fmaf(a, x.y, vi * k4[u].y), fmaf(a, x.z, vi * k4[u].z),
                            fmaf(a, x.w, vi * k4[u].w));
            if (in && j < dk) __stcs(reinterpret_cast<float4 *>(S_out + (base + i) * dk + j), x);
            acc += fmaf(x.x, q4[u].x, fmaf(x.y, q4[u].y, fmaf(x.z, q4[u].z, x.w * q4[u].w)));
        }
#pragma unroll
        for (int m = TL / 2; m >= 1; m >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, m);
        if (in && lane % TL == 0) o[base + i] = Io<IO>::from_f(scale * acc);
    }
}

// any dk: one warp per row
template <typename IO>
__global__ void __launch_bounds__(kStepT)
    decay_step_any_kernel(const IO *q, const IO *k, const IO *v, const float *a_log, const IO *g, float scale,
                          const float *S_in, float *S_out, IO *o, int64_t BH, int H, int Hk, int dk, int dv) {
    const int64_t row = int64_t(blockIdx.x) * (kStepT / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    launch_dependents();
    grid_dependency_wait();
    if (row >= BH * dv) return;   // warp-uniform
    const int64_t bh = row / dv, b = bh / H;
    const int h = int(bh - b * H), hk = h / (H / Hk);
    float l = a_log != nullptr ? a_log[h] : 0.0f;
    if (g != nullptr) l += Io<IO>::to_f(g[bh]);
    const float a = expf(l), vi = Io<IO>::to_f(v[row]);
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
    auto go = [&](auto kern, int rows) -> int {
        const int64_t tiles = (dv + rows - 1) / rows;
        const int64_t grid = (BH * tiles + kStepT / 32 - 1) / (kStepT / 32);
        if (grid > INT32_MAX) return LR_ERR_UNSUPPORTED;
        return launch_early(kern, dim3(unsigned(grid)), kStepT, s, q, k, v, a_log, g, scale, S_in, S_out, o, BH, H,
                            Hk, dk, dv, tiles);
    };
    if (dk % 4 == 0 && dk <= 512) {
        if (dk <= 32) return go(decay_step_kernel<IO, 8, 4, 1>, 16);
        if (dk <= 64) return go(decay_step_kernel<IO, 16, 4, 1>, 8);
        if (dk <= 128) return go(decay_step_kernel<IO, 32, 4, 1>, 4);
        if (dk <= 256) return go(decay_step_kernel<IO, 32, 2, 2>, 2);
        return go(decay_step_kernel<IO, 32, 2, 4>, 2);
    }
    const int64_t grid = (BH * dv + kStepT / 32 - 1) / (kStepT / 32);
    if (grid > INT32_MAX) return LR_ERR_UNSUPPORTED;
    return launch_early(decay_step_any_kernel<IO>, dim3(unsigned(grid)), kStepT, s, q, k, v, a_log, g, scale, S_in,
                        S_out, o, BH, H, Hk, dk, dv);
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
