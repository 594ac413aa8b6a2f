// lr_norm.cu -- group normalisation with an activation, channels last:
//   per row and group of d = C / G channels
//     m = mean(x), s2 = mean((x - m)^2), n = gamma (x - m) / sqrt(s2 + eps) + beta
//     y = act(n) silu(z)          act = identity or silu; no z: no gate
//
// Every value is read once and written once, so memory bandwidth bounds the
// kernel.  A group stays in the registers of the lanes that share it: the
// mean, then the centred squares (no cancellation), then the output.
//
// Measured in a graph of calls, 600 MB of inputs and outputs in turn (share of the copy
// bandwidth): bf16 16384 x 2048, G 16, gate 34.8 us (85 %; 32.4 onto one output
// tensor, half of which stays in L2); fp32 62.3 us (95 %); bf16 8192 x 4096, G 32
// 24.5 us (81 %); fp32 3001 x 1920, G 24 9.5 us (72 %; 7.5 onto one output); bf16 8192 x
// 4096, G 2, gate 36.2 us (82 %; element by element 82 us).  Sums and the affine step in
// packed fp32 pairs: the first 38.4 -> 36.7 us at the time.
//
// The figures at the variants below were taken onto one output.  Launched while the
// kernel before it drains: calls one after another 35.0 -> 33.0 us for the first, 10.5
// -> 8.4 for 3001 x 1920, so measured.
//
//   lanes   groups of up to 128 vectors (16 bytes; 8 for a bf16 group of an odd
//           number of those): TL lanes of a warp hold a group, up to four vectors
//           each, with the fewest idle slots; a thread keeps its group and walks
//           rows, several in flight
//   block   larger groups of 16-byte multiples: a block holds the group, up to
//           four vectors per thread
//   any     the rest (odd sizes, groups past a block's registers): a block per
//           group, three passes
#include "lr_decay.cuh"
#include "lr_vec.cuh"

namespace lr {
namespace {

struct NormArgs {
    const void *x, *z;
    const float *gamma, *beta;
    void *y;
    int64_t N;
    int C, G, d;
    float eps, inv_d;
    int act;
};

// y of one vector whose values are already centred
template <typename X, bool GATE>
__device__ __forceinline__ typename X::Raw finish(float *v, float rs, const float *ga, const float *be,
                                                  const typename X::Raw &zr, int act) {
    constexpr int VN = X::N;
    float z[VN];
    if (GATE) X::widen(zr, z);
    const float2 rs2 = make_float2(rs, rs);
#pragma unroll
    for (int i = 0; i < VN; i += 2) {
        const float2 n = __ffma2_rn(__fmul2_rn(pair(v + i), rs2), pair(ga + i), pair(be + i));
        v[i] = n.x, v[i + 1] = n.y;
    }
    if (act == LR_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < VN; ++i) v[i] = silu_f(v[i]);
    }
    if (GATE) {
#pragma unroll
        for (int i = 0; i < VN; ++i) v[i] *= silu_f(z[i]);
    }
    return X::narrow(v);
}

template <int VN>
__device__ __forceinline__ void load_affine(const float *gamma, const float *beta, int c, bool in, float *ga, float *be) {
#pragma unroll
    for (int i = 0; i < VN; i += 4) {
        const float4 one = make_float4(1.0f, 1.0f, 1.0f, 1.0f), zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const float4 g = gamma != nullptr && in ? *reinterpret_cast<const float4 *>(gamma + c + i) : one;
        const float4 b = beta != nullptr && in ? *reinterpret_cast<const float4 *>(beta + c + i) : zero;
        ga[i] = g.x, ga[i + 1] = g.y, ga[i + 2] = g.z, ga[i + 3] = g.w;
        be[i] = b.x, be[i + 1] = b.y, be[i + 2] = b.z, be[i + 3] = b.w;
    }
}

// TL lanes per group, V vectors per lane (vector u of lane l: l + u TL).  A
// thread keeps its group (its channels, so gamma and beta stay in registers)
// and walks rows, ROWS of them in flight: groups are dealt over grid.y and the
// lane sets of a block, rows over grid.x.
template <typename X, int TL, int V, int ROWS, bool GATE>
__global__ void __launch_bounds__(256)
    group_norm_lanes_kernel(const NormArgs a, int gper) {
    launch_dependents();
    grid_dependency_wait();
    using Raw = typename X::Raw;
    constexpr int VN = X::N, SETS = 256 / TL;   // lane sets of a block
    const int set = threadIdx.x / TL, l = threadIdx.x % TL;
    // sets of a block: consecutive groups of a row, then rows
    const int rper = SETS / gper;
    const int gi = blockIdx.y * gper + set % gper;
    const int r0 = set / gper;
    const bool live = gi < a.G && r0 < rper;
    const int nv = a.d / VN;
    float ga[V][VN], be[V][VN];
    bool in[V];
#pragma unroll
    for (int u = 0; u < V; ++u) {
        in[u] = live && l + u * TL < nv;
        load_affine<VN>(a.gamma, a.beta, gi * a.d + (l + u * TL) * VN, in[u], ga[u], be[u]);
    }
    const Raw *x = static_cast<const Raw *>(a.x);
    const Raw *z = static_cast<const Raw *>(a.z);
    Raw *y = static_cast<Raw *>(a.y);
    const int64_t row_vecs = a.C / VN, col = int64_t(gi) * nv + l;
    const int64_t step = int64_t(gridDim.x) * rper;
    for (int64_t base = int64_t(blockIdx.x) * rper; base < a.N; base += step * ROWS) {
        Raw xr[ROWS][V], zr[ROWS][V];
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const int64_t r = base + k * step + r0;
#pragma unroll
            for (int u = 0; u < V; ++u) {
                xr[k][u] = Raw{};
                zr[k][u] = Raw{};
                if (in[u] && r < a.N) {
                    xr[k][u] = __ldcs(x + r * row_vecs + col + u * TL);
                    if (GATE) zr[k][u] = __ldcs(z + r * row_vecs + col + u * TL);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const int64_t r = base + k * step + r0;
            float v[V][VN];
            float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int u = 0; u < V; ++u) {
                X::widen(xr[k][u], v[u]);
#pragma unroll
                for (int i = 0; i < VN; i += 2) s2 = __fadd2_rn(s2, pair(v[u] + i));
            }
            float s = s2.x + s2.y;
#pragma unroll
            for (int m = TL / 2; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
            const float mean = s * a.inv_d;
            s = 0.0f;
#pragma unroll
            for (int u = 0; u < V; ++u) {
                s2 = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int i = 0; i < VN; i += 2) {
                    const float2 c = __fadd2_rn(pair(v[u] + i), make_float2(-mean, -mean));
                    s2 = __ffma2_rn(c, c, s2);
                    v[u][i] = c.x, v[u][i + 1] = c.y;
                }
                if (in[u]) s += s2.x + s2.y;
            }
#pragma unroll
            for (int m = TL / 2; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
            const float rs = 1.0f / sqrtf(fmaf(s, a.inv_d, a.eps));
#pragma unroll
            for (int u = 0; u < V; ++u)
                if (in[u] && r < a.N)
                    __stcs(y + r * row_vecs + col + u * TL, finish<X, GATE>(v[u], rs, ga[u], be[u], zr[k][u], a.act));
        }
    }
}

// sum over a block of NT threads, to all of them
template <int NT>
__device__ __forceinline__ float block_sum(float s, float *red) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    __syncthreads();   // the last sum has been read
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) s += red[i];
    return s;
}

// a block per group (grid-stride over row-groups), V vectors per thread
template <typename X, int NT, int V, bool GATE>
__global__ void __launch_bounds__(NT)
    group_norm_block_kernel(const NormArgs a) {
    launch_dependents();
    grid_dependency_wait();
    using Raw = typename X::Raw;
    constexpr int VN = X::N;
    __shared__ float red[NT / 32];
    const int nv = a.d / VN;
    for (int64_t rg = blockIdx.x; rg < a.N * a.G; rg += gridDim.x) {
        const int gi = int(rg % a.G);
        const int64_t at = rg * nv;
        const Raw *x = static_cast<const Raw *>(a.x) + at;
        const Raw *z = static_cast<const Raw *>(a.z) + at;
        Raw xr[V], zr[V];
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int i = threadIdx.x + u * NT;
            xr[u] = Raw{};
            zr[u] = Raw{};
            if (i < nv) {
                xr[u] = __ldcs(x + i);
                if (GATE) zr[u] = __ldcs(z + i);
            }
        }
        float v[V][VN];
        float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int u = 0; u < V; ++u) {
            X::widen(xr[u], v[u]);
#pragma unroll
            for (int i = 0; i < VN; i += 2) s2 = __fadd2_rn(s2, pair(v[u] + i));
        }
        const float mean = block_sum<NT>(s2.x + s2.y, red) * a.inv_d;
        float s = 0.0f;
#pragma unroll
        for (int u = 0; u < V; ++u) {
            s2 = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < VN; i += 2) {
                const float2 c = __fadd2_rn(pair(v[u] + i), make_float2(-mean, -mean));
                s2 = __ffma2_rn(c, c, s2);
                v[u][i] = c.x, v[u][i + 1] = c.y;
            }
            if (threadIdx.x + u * NT < nv) s += s2.x + s2.y;
        }
        const float rs = 1.0f / sqrtf(fmaf(block_sum<NT>(s, red), a.inv_d, a.eps));
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int i = threadIdx.x + u * NT;
            if (i < nv) {
                float ga[VN], be[VN];
                load_affine<VN>(a.gamma, a.beta, gi * a.d + i * VN, true, ga, be);
                __stcs(static_cast<Raw *>(a.y) + at + i, finish<X, GATE>(v[u], rs, ga, be, zr[u], a.act));
            }
        }
    }
}

// any sizes: a block of NT threads per (row, group), three passes over the group
template <typename IO, int NT>
__global__ void __launch_bounds__(NT)
    group_norm_any_kernel(const NormArgs a) {
    launch_dependents();
    grid_dependency_wait();
    __shared__ float red[NT / 32];
    const IO *x = static_cast<const IO *>(a.x), *z = static_cast<const IO *>(a.z);
    IO *y = static_cast<IO *>(a.y);
    for (int64_t rg = blockIdx.x; rg < a.N * a.G; rg += gridDim.x) {
        const int gi = int(rg % a.G);
        const int64_t at = rg * a.d;
        float s = 0.0f;
        for (int i = threadIdx.x; i < a.d; i += NT) s += Io<IO>::to_f(x[at + i]);
        const float mean = block_sum<NT>(s, red) * a.inv_d;
        s = 0.0f;
        for (int i = threadIdx.x; i < a.d; i += NT) {
            const float t = Io<IO>::to_f(x[at + i]) - mean;
            s = fmaf(t, t, s);
        }
        const float rs = 1.0f / sqrtf(fmaf(block_sum<NT>(s, red), a.inv_d, a.eps));
        for (int i = threadIdx.x; i < a.d; i += NT) {
            const int c = gi * a.d + i;
            float n = (Io<IO>::to_f(x[at + i]) - mean) * rs;
            if (a.gamma != nullptr) n *= a.gamma[c];
            if (a.beta != nullptr) n += a.beta[c];
            if (a.act == LR_ACT_SILU) n = silu_f(n);
            if (z != nullptr) n *= silu_f(Io<IO>::to_f(z[at + i]));
            y[at + i] = Io<IO>::from_f(n);
        }
    }
}

template <typename X, int TL, int V, bool GATE>
int launch_lanes(const NormArgs &a, int sms, cudaStream_t s) {
    constexpr int SETS = 256 / TL;
    // groups of a row per block: the count that leaves the fewest sets idle, the
    // larger of two, since neighbouring groups are neighbouring bytes (16384 x 2048
    // bf16, G 32, gate: the smaller 45.5 us against 36.1; 8192 x 4096 32.3 against
    // 26.5)
    int gper = 1;
    double best = 0.0;
    for (int g = 1; g <= SETS && g <= a.G; ++g) {
        const double used = double(g * (SETS / g)) / SETS * double(a.G) / double((a.G + g - 1) / g * g);
        if (used >= best - 1e-9) best = used, gper = g;
    }
    const int rper = SETS / gper, gy = (a.G + gper - 1) / gper;
    const int64_t row_blocks = (a.N + rper - 1) / rper;
    // Rows in flight per thread once every SM has its blocks, one where there
    // are few.  bf16: 16384 x 2048, G 32, gate (one vector a lane) 1 row 41.5 us, 2
    // rows 34.7, 4 rows 36.1; without gate 2 rows 30.0, 4 rows 27.3; 8192 x 4096,
    // G 32 (two vectors) 1 row 28.8 us, 2 rows 26.5, 4 rows 32.9.  Three and four
    // vectors: 4096 x 3200, G 40, gate 1 row 18.3 us, 2 rows 26.7.
    constexpr int R = V == 1 ? (GATE ? 2 : 4) : V == 2 ? 2 : 1;
    // The blocks that fit, which then walk the rows, against six per SM: 16384 x
    // 2048 bf16, gate, G 32 31.3 us against 34.6, G 16 33.0 against 34.4; 8192 x 4096
    // 24.5 against 26.5; 591 x 8192 fp32, gate 9.8 against 11.3.  Groups of three
    // vectors a lane take twice as many: 3001 x 1920 fp32 8.45 us against 9.1.
    static DeviceSetup setup;
    static std::atomic<int> fit{1};   // (the same on every GPU that runs this code)
    if (!setup.run([] {
            int n = 0;
            if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, group_norm_lanes_kernel<X, TL, V, R, GATE>, 256, 0) !=
                    cudaSuccess || n < 1)
                return false;
            fit = n;
            return true;
        }))
        return LR_ERR_CUDA;
    const int64_t full = int64_t(sms) * fit * (V == 3 ? 2 : 1);
    const bool deep = row_blocks * gy >= full * R;
    int64_t gx = deep ? (full + gy - 1) / gy : row_blocks;
    if (gx > row_blocks) gx = row_blocks;
    const dim3 grid{unsigned(gx), unsigned(gy), 1};
    return launch_early(deep ? group_norm_lanes_kernel<X, TL, V, R, GATE> : group_norm_lanes_kernel<X, TL, V, 1, GATE>,
                        grid, 256, s, a, gper);
}

template <typename X, int NT, int V, bool GATE>
int launch_block(const NormArgs &a, int sms, cudaStream_t s) {
    const int64_t ng = a.N * a.G, most = int64_t(sms) * (2048 / NT) * 2;
    return launch_early(group_norm_block_kernel<X, NT, V, GATE>, dim3(unsigned(ng < most ? ng : most)), NT, s, a);
}

template <typename IO>
int launch_any(const NormArgs &a, int sms, cudaStream_t s) {
    const int64_t ng = a.N * a.G, most = int64_t(sms) * 128;
    const dim3 grid(unsigned(ng < most ? ng : most));
    // one warp where a block's barriers cost more than its width gives (4096 x
    // 999 fp32, G 9: 21.8 us against 36.4; 8192 x 1111, G 1: 25.6 against 20.2)
    return a.d <= 256 ? launch_early(group_norm_any_kernel<IO, 32>, grid, 32, s, a)
                      : launch_early(group_norm_any_kernel<IO, 128>, grid, 128, s, a);
}

// nv vectors per group: lanes x vectors with the fewest idle slots (4096 x 3200
// bf16, 10 vectors: 4 x 3 18.2 us, 16 x 1 23.5).  Past a warp's 128 vectors a
// block per group, up to four vectors a thread (2000 x 12000 bf16, G 8, gate, 375
// vectors of 8 bytes: 128 x 4 31.3 us, 256 x 2 38.4).
template <typename X, bool GATE>
int launch_vec(const NormArgs &a, int nv, int sms, cudaStream_t s) {
    if (nv <= 4) return launch_lanes<X, 4, 1, GATE>(a, sms, s);
    if (nv <= 8) return launch_lanes<X, 8, 1, GATE>(a, sms, s);
    if (nv <= 12) return launch_lanes<X, 4, 3, GATE>(a, sms, s);
    // two vectors a lane halve the shuffles: 16384 x 2048 bf16, G 16, gate 34.4 us
    // against 36.9 with 16 lanes; 8192 x 4096 without gate 26.5 against 30.2
    if (nv <= 16) return launch_lanes<X, 8, 2, GATE>(a, sms, s);
    if (nv <= 24) return launch_lanes<X, 8, 3, GATE>(a, sms, s);
    if (nv <= 32) return launch_lanes<X, 16, 2, GATE>(a, sms, s);
    if (nv <= 48) return launch_lanes<X, 16, 3, GATE>(a, sms, s);
    if (nv <= 64) return launch_lanes<X, 32, 2, GATE>(a, sms, s);
    if (nv <= 96) return launch_lanes<X, 32, 3, GATE>(a, sms, s);
    if (nv <= 128) return launch_lanes<X, 32, 4, GATE>(a, sms, s);
    if (nv <= 256) return launch_block<X, 128, 2, GATE>(a, sms, s);
    if (nv <= 512) return launch_block<X, 128, 4, GATE>(a, sms, s);
    if (nv <= 1024) return launch_block<X, 256, 4, GATE>(a, sms, s);
    return launch_block<X, 512, 4, GATE>(a, sms, s);
}

template <typename IO, bool GATE>
int norm_gate(const NormArgs &a, cudaStream_t s) {
    constexpr bool BF = sizeof(IO) == 2;
    int sms = 0;
    if (device_sm_count(&sms) != LR_OK) return LR_ERR_CUDA;
    // C is a multiple of d, so every group starts on a vector's boundary
    constexpr int W = BF ? 8 : 4;
    if (a.G <= 65535) {
        if (a.d % W == 0 && a.d / W <= 2048) return launch_vec<Vec<IO, W>, GATE>(a, a.d / W, sms, s);
        if constexpr (BF)
            if (a.d % 4 == 0 && a.d / 4 <= 2048) return launch_vec<Vec<IO, 4>, GATE>(a, a.d / 4, sms, s);
    }
    return launch_any<IO>(a, sms, s);
}

}  // namespace

int group_norm_act_launch(const void *x, const void *z, const float *gamma, const float *beta, void *y,
                          int64_t N, int64_t C, int64_t G, float eps, int act, int io_bf16, cudaStream_t stream) {
    if (N == 0 || C == 0) return LR_OK;
    const int d = int(C / G);
    const NormArgs a{x, z, gamma, beta, y, N, int(C), int(G), d, eps, 1.0f / float(d), act};
    if (io_bf16) return z != nullptr ? norm_gate<__nv_bfloat16, true>(a, stream) : norm_gate<__nv_bfloat16, false>(a, stream);
    return z != nullptr ? norm_gate<float, true>(a, stream) : norm_gate<float, false>(a, stream);
}

}  // namespace lr
