// lr_conv.cu -- short causal convolution of every channel by its own W taps, channels last:
//   y_t[c] = act(bias[c] + sum_j w[c][j] x_{t - W + 1 + j}[c]),   j = 0 .. W - 1
// with the inputs before a row's first step from the carried state (zero without
// one), and one step of it for decoding.
//
// Every input is read once and every output written once (2 W operations an
// element), so memory bandwidth bounds the prompt form and the launch's latency
// the step.  A thread owns one vector of four channels (one where rows do not fit
// vectors) over a range of steps: its taps and the last W - 1 inputs stay in registers,
// and the steps' loads are in flight in groups, each sent for again as soon as it is
// used.  Measured, in turn over 500 MB: bf16 B4 L4096 C2304 W4, a slice, 29.0 us (77 % of
// the copy bandwidth); B1 L32768 52.5 (85 %); fp32 B4 L4096 W2 47.0 (95 %); fp32 B8 L1017
// C1320 W3 17.6, C1321 (a value at a time) 18.7; bf16 B1 L77 3.3.  In bf16 issue is 37 %,
// the fp32 pipe 15 %, and 22 % of the warps are there (128 registers a thread hold the steps
// in flight).
//   eight channels a thread: bf16 36-40 us (217 registers without a bound: 48)
//   eight steps' loads, used before the next are sent for 31.1 us; four groups of four in
//   turn 29.0, two 31.9; fp32 two 47.0, four 50.4
//   one reciprocal for two values of silu: 29.3
#include <type_traits>

#include "lr_decay.cuh"
#include "lr_vec.cuh"

namespace lr {
namespace {

constexpr int kConvT = 128;    // threads per block

struct ConvArgs {
    const void *x;
    int64_t ldx;             // elements between the rows of x
    const float *w, *bias;
    const void *state;       // (B, W - 1, C) or NULL
    const int32_t *lens;
    void *y, *state_out;
    int64_t B, L;
    int C, steps, tiles;     // steps of a thread, ranges of a row
    int act;
};

// The inputs are plain pointers for the reason given in lr_decay_step.cu.

// Taps as [j][channel of the vector].
template <int VN, int W>
__device__ __forceinline__ void load_taps(const ConvArgs &a, int c, float (&wt)[W][VN], float (&be)[VN]) {
    float f[VN * W];
    const float *src = a.w + int64_t(c) * W;
    if constexpr (VN % 4 == 0) {
#pragma unroll
        for (int i = 0; i < VN * W; i += 4) {
            const float4 u = *reinterpret_cast<const float4 *>(src + i);
            f[i] = u.x, f[i + 1] = u.y, f[i + 2] = u.z, f[i + 3] = u.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VN * W; ++i) f[i] = src[i];
    }
#pragma unroll
    for (int i = 0; i < VN; ++i) {
        be[i] = a.bias != nullptr ? a.bias[c + i] : 0.0f;
#pragma unroll
        for (int j = 0; j < W; ++j) wt[j][i] = f[i * W + j];
    }
}

// The output of one step from the W inputs that end there; two channels at a time.
template <typename X, int W>
__device__ __forceinline__ typename X::Raw conv_one(const float (*in)[X::N], const float (&wt)[W][X::N],
                                                    const float (&be)[X::N], int act) {
    float v[X::N];
    if constexpr (X::N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < X::N; i += 2) {
            float2 y = pair(be + i);
#pragma unroll
            for (int j = 0; j < W; ++j) y = __ffma2_rn(pair(wt[j] + i), pair(in[j] + i), y);
            if (act == LR_ACT_SILU) y = silu2_f(y);
            v[i] = y.x, v[i + 1] = y.y;
        }
    } else {
        v[0] = be[0];
#pragma unroll
        for (int j = 0; j < W; ++j) v[0] = fmaf(wt[j][0], in[j][0], v[0]);
        if (act == LR_ACT_SILU) v[0] = silu_f(v[0]);
    }
    return X::narrow(v);
}

// Input t >= -(W - 1) of a row: its own, or of the state.
template <typename Raw, int W>
__device__ __forceinline__ Raw input_at(const Raw *x, int64_t ld, const Raw *state, int64_t lds, int t) {
    if (t >= 0) return x[t * ld];
    return state != nullptr ? state[(W - 1 + t) * lds] : Raw{};
}

// Range 0 of a row alone reads the row's old state and writes its new one, which
// may be the same memory: each of its threads has read all it needs by then.
template <typename X, int W>
__global__ void __launch_bounds__(kConvT, X::N == 1 ? 8 : 4) conv_kernel(const ConvArgs a) {
    using Raw = typename X::Raw;
    constexpr int VN = X::N, R = sizeof(Raw) == 16 ? 2 : 4, Q = 4;
    launch_dependents();
    grid_dependency_wait();
    const int nvec = a.C / VN;
    const int64_t idx = int64_t(blockIdx.x) * kConvT + threadIdx.x;
    const int cv = int(idx % nvec);
    const int64_t rt = idx / nvec;
    const int tile = int(rt % a.tiles);
    const int64_t b = rt / a.tiles;
    if (b >= a.B) return;
    const int n = dec::row_len(a.lens, int(b), a.L);
    const int t0 = tile * a.steps, t1 = int(min(a.L, int64_t(t0) + a.steps)), te = min(t1, n);
    const int64_t ld = a.ldx / VN;
    // (VN elements apart: ldx is a multiple of VN wherever VN > 1)
    const Raw *x = static_cast<const Raw *>(a.x) + b * a.L * ld + cv;
    const Raw *state = a.state == nullptr ? nullptr : static_cast<const Raw *>(a.state) + b * (W - 1) * nvec + cv;
    Raw *y = static_cast<Raw *>(a.y) + b * a.L * nvec + cv;
    float wt[W][VN], be[VN];
    Raw last[W - 1];   // the row's new state
    if (tile == 0 && a.state_out != nullptr) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) last[j] = input_at<Raw, W>(x, ld, state, nvec, n - (W - 1) + j);
    }
    int t = t0;
    if (t < te) {
        load_taps<VN, W>(a, cv * VN, wt, be);
        float in[W - 1 + Q][VN];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) X::widen(input_at<Raw, W>(x, ld, state, nvec, t0 - (W - 1) + j), in[j]);
        Raw r[R][Q];   // steps t ..: R groups of Q, each loaded again as soon as it is widened
        const Raw *next = x + int64_t(t) * ld;
        Raw *dst = y + int64_t(t) * nvec;
#pragma unroll
        for (int g = 0; g < R; ++g)
#pragma unroll
            for (int k = 0; k < Q; ++k) r[g][k] = t + g * Q + k < te ? next[(g * Q + k) * ld] : Raw{};
        auto round = [&](auto whole) {   // whole: the next R groups are there too
            constexpr bool ALL = decltype(whole)::value;
            next += R * Q * ld;
#pragma unroll
            for (int g = 0; g < R; ++g) {
#pragma unroll
                for (int k = 0; k < Q; ++k) X::widen(r[g][k], in[W - 1 + k]);
#pragma unroll
                for (int k = 0; k < Q; ++k)
                    if (ALL || t + (R + g) * Q + k < te) r[g][k] = next[(g * Q + k) * ld];
#pragma unroll
                for (int k = 0; k < Q; ++k)
                    if (ALL || t + g * Q + k < te) dst[int64_t(g * Q + k) * nvec] = conv_one<X, W>(in + k, wt, be, a.act);
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
#pragma unroll
                    for (int i = 0; i < VN; ++i) in[j][i] = in[Q + j][i];
            }
            t += R * Q;
            dst += int64_t(R * Q) * nvec;
        };
        while (t + 2 * R * Q <= te) round(std::true_type{});
        while (t < te) round(std::false_type{});
    }
    for (t = max(t0, te); t < t1; ++t) y[int64_t(t) * nvec] = Raw{};   // past the row's end
    if (tile == 0 && a.state_out != nullptr) {
        Raw *out = static_cast<Raw *>(a.state_out) + b * (W - 1) * nvec + cv;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) out[int64_t(j) * nvec] = last[j];
    }
}

// One step of every row: the state moves up by one input.
template <typename X, int W>
__global__ void __launch_bounds__(kConvT) conv_step_kernel(const ConvArgs a) {
    using Raw = typename X::Raw;
    constexpr int VN = X::N;
    launch_dependents();
    grid_dependency_wait();
    const int nvec = a.C / VN;
    const int64_t idx = int64_t(blockIdx.x) * kConvT + threadIdx.x, b = idx / nvec;
    if (b >= a.B) return;
    const int cv = int(idx - b * nvec);
    Raw r[W];
    r[W - 1] = static_cast<const Raw *>(a.x)[b * (a.ldx / VN) + cv];
    const int64_t at = b * (W - 1) * nvec + cv;
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
        r[j] = a.state != nullptr ? static_cast<const Raw *>(a.state)[at + int64_t(j) * nvec] : Raw{};
    float wt[W][VN], be[VN], in[W][VN];
    load_taps<VN, W>(a, cv * VN, wt, be);
#pragma unroll
    for (int j = 0; j < W; ++j) X::widen(r[j], in[j]);
    const Raw y = conv_one<X, W>(in, wt, be, a.act);
    Raw *out = static_cast<Raw *>(a.state_out) + at;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) out[int64_t(j) * nvec] = r[j + 1];
    static_cast<Raw *>(a.y)[idx] = y;
}

template <typename X, int W>
int conv_go(ConvArgs a, bool step, cudaStream_t s) {
    const int64_t nvec = a.C / X::N;
    if (step) {
        const int64_t grid = (a.B * nvec + kConvT - 1) / kConvT;
        if (grid > INT32_MAX) return LR_ERR_UNSUPPORTED;
        return launch_early(conv_step_kernel<X, W>, dim3(unsigned(grid)), kConvT, s, a);
    }
    int sms = 0;
    if (device_sm_count(&sms) != LR_OK) return LR_ERR_CUDA;
    // the longest ranges that still give every SM its threads: a range reads its
    // taps and the W - 1 inputs before it again (B4 L4096: 32 steps 31.8 us, 64 29.0, 128 29.1)
    a.steps = 64;
    while (a.steps > 16 && a.B * ((a.L + a.steps - 1) / a.steps) * nvec < int64_t(sms) * 512) a.steps /= 2;
    const int64_t tiles = (a.L + a.steps - 1) / a.steps, grid = (a.B * tiles * nvec + kConvT - 1) / kConvT;
    if (grid > INT32_MAX) return LR_ERR_UNSUPPORTED;
    a.tiles = int(tiles);
    return launch_early(conv_kernel<X, W>, dim3(unsigned(grid)), kConvT, s, a);
}

template <typename X>
int conv_taps(const ConvArgs &a, int W, bool step, cudaStream_t s) {
    switch (W) {
        case 2: return conv_go<X, 2>(a, step, s);
        case 3: return conv_go<X, 3>(a, step, s);
        case 4: return conv_go<X, 4>(a, step, s);
    }
    return LR_ERR_UNSUPPORTED;
}

template <typename IO>
int conv_io(const ConvArgs &a, int W, bool step, cudaStream_t s) {
    // whole vectors where every row of x and y starts on one
    constexpr int V = 4;
    if (a.C % V == 0 && a.ldx % V == 0) return conv_taps<Vec<IO, V>>(a, W, step, s);
    return conv_taps<Vec<IO, 1>>(a, W, step, s);
}

}  // namespace

int causal_conv_launch(const void *x, int64_t ldx, const float *w, const float *bias, const void *state,
                       const int32_t *lens, void *y, void *state_out, int64_t B, int64_t L, int64_t C, int W, int act,
                       int io_bf16, bool step, cudaStream_t stream) {
    if (B == 0 || C == 0) return LR_OK;
    const ConvArgs a{x, ldx, w, bias, state, lens, y, state_out, B, L, int(C), 0, 0, act};
    return io_bf16 ? conv_io<__nv_bfloat16>(a, W, step, stream) : conv_io<float>(a, W, step, stream);
}

}  // namespace lr
