// lr_rope.cu -- norm of every head of the queries and the keys, and the rotation of
// its pairs by the token's position, in one pass:
//   n = gamma x / sqrt(mean(x^2) + eps)   (rms; l2: the sum of the squares; none: gamma x)
//   (a, b) = pair i of n:  (a cos - b sin, b cos + a sin),  angle pos freqs[i]
//
// Every value is read once and written once, so memory bandwidth bounds the kernel
// (the launch's latency for a few tokens).  The lanes that share a head each hold
// both partners of their pairs, so the norm is one sum over lanes and the rotation
// needs no exchange; they keep their pairs' angles for all heads of a token that
// they take.
//
// Angles.  freqs is turned into turns (1 / 2 pi) as two floats, to 2^-48 of it, and
// those into a 64-bit fraction of a turn, whose product with the position wraps by
// itself: far positions lose nothing to the size of their angle.
#include "lr_decay.cuh"
#include "lr_vec.cuh"

namespace lr {
namespace {

constexpr int kRopeT = 128;

struct RopeArgs {
    const void *q, *k;
    int64_t ldq, ldk;
    const float *gq, *gk, *freqs;
    const int32_t *pos;
    void *qo, *ko;
    int64_t N;
    int H, Hk, d, rot;
    int norm;
    float eps;
    int sets, heads;   // lane sets of a token, heads of each
};

// The part of a turn that a position adds, in units of 2^-64.
__device__ __forceinline__ long long turn_of(float f) {
    constexpr double kTurn = 0.15915494309189535;   // 1 / 2 pi
    constexpr float kHi = float(kTurn), kLo = float(kTurn - double(kHi)), k62 = 4611686018427387904.0f;
    float p = f * kHi;
    const float r = fmaf(f, kLo, fmaf(f, kHi, -p));
    p -= rintf(p);   // whole turns; exact
    return static_cast<long long>(static_cast<unsigned long long>(__float2ll_rn(p * k62) + __float2ll_rn(r * k62)) << 2);
}

// TL lanes a head; U units a lane, each of two vectors of X::N values.
//   halves      (NB = 0, pair i: values i and i + rot / 2): unit u holds vectors u
//               and u + rot / 2 / N
//   neighbours  (pair i: values 2 i and 2 i + 1): vectors 2 u and 2 u + 1, whose pairs
//               lie inside them; of single values they are the pair
// Units past the rotated ones hold two vectors that are only normalised.
template <typename X, int TL, int U, bool NB>
__global__ void __launch_bounds__(kRopeT) rope_kernel(const RopeArgs a) {
    using Raw = typename X::Raw;
    constexpr int VN = X::N;
    constexpr bool INSIDE = NB && VN > 1;   // pairs inside a vector
    launch_dependents();
    grid_dependency_wait();
    const int l = threadIdx.x % TL;
    const int64_t set = (int64_t(blockIdx.x) * kRopeT + threadIdx.x) / TL;
    const int64_t n = set / a.sets;
    const bool live = n < a.N;
    const int h0 = int(set - n * a.sets) * a.heads, h1 = live ? min(h0 + a.heads, a.H + a.Hk) : h0;
    const int nv = a.d / VN, rv = a.rot / 2 / VN, nr = a.rot / 2;
    int va[U], vb[U];          // a unit's vectors, -1: none
    int turned[U];             // its pairs that are rotated
    float co[U][VN], si[U][VN];
    const long long pos = live && nr > 0 ? a.pos[n] : 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int un = l + u * TL;
        if (NB || un >= rv) {
            va[u] = 2 * un, vb[u] = va[u] + 1;
            turned[u] = NB ? max(0, min(VN, nr - un * VN)) : 0;
        } else {
            va[u] = un, vb[u] = un + rv;
            turned[u] = VN;
        }
        if (va[u] >= nv) va[u] = -1;
        if (vb[u] >= nv) vb[u] = -1;
#pragma unroll
        for (int e = 0; e < VN; ++e)
            if (e < turned[u]) {
                const long long t = static_cast<long long>(static_cast<unsigned long long>(turn_of(a.freqs[un * VN + e])) *
                                                           static_cast<unsigned long long>(pos));
                sincospif(1.0842021724855044e-19f * __ll2float_rn(t), &si[u][e], &co[u][e]);   // half turns
            }
    }
    auto row = [&](int h) {
        return h >= a.H ? static_cast<const Raw *>(a.k) + n * (a.ldk / VN) + int64_t(h - a.H) * nv
                        : static_cast<const Raw *>(a.q) + n * (a.ldq / VN) + int64_t(h) * nv;
    };
    Raw r[U][2];
    auto load = [&](int h) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            r[u][0] = h < h1 && va[u] >= 0 ? row(h)[va[u]] : Raw{};
            r[u][1] = h < h1 && vb[u] >= 0 ? row(h)[vb[u]] : Raw{};
        }
    };
    load(h0);
    // (every lane of the warp goes through all a.heads turns: the sum needs them)
    for (int h = h0; h < h0 + a.heads; ++h) {
        float x[U][2][VN];
        float s = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            X::widen(r[u][0], x[u][0]);
            X::widen(r[u][1], x[u][1]);
#pragma unroll
            for (int e = 0; e < VN; ++e) s = fmaf(x[u][0][e], x[u][0][e], fmaf(x[u][1][e], x[u][1][e], s));
        }
        load(h + 1);   // on its way during this one's arithmetic
        float rs = 1.0f;
        if (a.norm != LR_NORM_NONE) {
#pragma unroll
            for (int m = TL / 2; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
            rs = 1.0f / sqrtf((a.norm == LR_NORM_RMS ? s / float(a.d) : s) + a.eps);
        }
        if (h >= h1) continue;
        const bool key = h >= a.H;
        const float *g = key ? a.gk : a.gq;
        Raw *dst = key ? static_cast<Raw *>(a.ko) + (n * a.Hk + (h - a.H)) * int64_t(nv)
                       : static_cast<Raw *>(a.qo) + (n * a.H + h) * int64_t(nv);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float *p = x[u][0], *q = x[u][1];
#pragma unroll
            for (int e = 0; e < VN; ++e) {
                p[e] *= g != nullptr && va[u] >= 0 ? rs * g[va[u] * VN + e] : rs;
                q[e] *= g != nullptr && vb[u] >= 0 ? rs * g[vb[u] * VN + e] : rs;
            }
#pragma unroll
            for (int e = 0; e < VN; ++e) {
                if (e >= turned[u]) continue;
                const float c = co[u][e], sn = si[u][e];
                // pair e of the unit
                float &v = INSIDE ? (2 * e < VN ? p[(2 * e) % VN] : q[(2 * e) % VN]) : p[e];
                float &w = INSIDE ? (2 * e < VN ? p[(2 * e + 1) % VN] : q[(2 * e + 1) % VN]) : q[e];
                const float v0 = v;
                v = v0 * c - w * sn;
                w = w * c + v0 * sn;
            }
            if (va[u] >= 0) dst[va[u]] = X::narrow(p);
            if (vb[u] >= 0) dst[vb[u]] = X::narrow(q);
        }
    }
}

template <typename X, int TL, int U, bool NB>
int rope_go(RopeArgs a, cudaStream_t s) {
    int sms = 0;
    if (device_sm_count(&sms) != LR_OK) return LR_ERR_CUDA;
    // as many heads for one set of lanes as still leave every SM its threads
    const int heads = a.H + a.Hk;
    a.heads = 1;
    while (a.heads < heads && a.N * ((heads + 2 * a.heads - 1) / (2 * a.heads)) * TL >= int64_t(sms) * 2048) a.heads *= 2;
    if (a.heads > heads) a.heads = heads;
    a.sets = (heads + a.heads - 1) / a.heads;
    const int64_t grid = (a.N * a.sets * TL + kRopeT - 1) / kRopeT;
    if (grid > INT32_MAX) return LR_ERR_UNSUPPORTED;
    return launch_early(rope_kernel<X, TL, U, NB>, dim3(unsigned(grid)), kRopeT, s, a);
}

template <typename IO, bool NB>
int rope_pairs(const RopeArgs &a, cudaStream_t s) {
    constexpr int V = 16 / sizeof(IO);
    // whole vectors where every head starts on one and no vector holds both partners' halves
    if (a.d % V == 0 && a.ldq % V == 0 && a.ldk % V == 0 && (NB || a.rot / 2 % V == 0)) {
        using X = Vec<IO, V>;
        const int units = (a.d / V + 1) / 2;
        if (units <= 2) return rope_go<X, 2, 1, NB>(a, s);
        if (units <= 4) return rope_go<X, 4, 1, NB>(a, s);
        if (units <= 8) return rope_go<X, 8, 1, NB>(a, s);
        if (units <= 16) return rope_go<X, 16, 1, NB>(a, s);
        if (units <= 32) return rope_go<X, 32, 1, NB>(a, s);
        if constexpr (V == 4) return rope_go<X, 32, 2, NB>(a, s);
    }
    using X = Vec<IO, 1>;
    const int units = (a.d + 1) / 2;
    if (units <= 32) return rope_go<X, 32, 1, NB>(a, s);
    if (units <= 64) return rope_go<X, 32, 2, NB>(a, s);
    if (units <= 128) return rope_go<X, 32, 4, NB>(a, s);
    return rope_go<X, 32, 8, NB>(a, s);
}

}  // namespace

int head_norm_rope_launch(const void *q, int64_t ldq, const void *k, int64_t ldk, const float *gq, const float *gk,
                          const float *freqs, const int32_t *pos, void *qo, void *ko, int64_t N, int64_t H, int64_t Hk,
                          int64_t d, int64_t rot, int norm, float eps, int pairs, int io_bf16, cudaStream_t stream) {
    if (N == 0 || H + Hk == 0) return LR_OK;
    const RopeArgs a{q, k, ldq, ldk, gq, gk, freqs, pos, qo, ko, N, int(H), int(Hk), int(d), int(rot), norm, eps, 0, 0};
    const bool nb = pairs == LR_PAIRS_NEIGHBOURS;
    if (io_bf16) return nb ? rope_pairs<__nv_bfloat16, true>(a, stream) : rope_pairs<__nv_bfloat16, false>(a, stream);
    return nb ? rope_pairs<float, true>(a, stream) : rope_pairs<float, false>(a, stream);
}

}  // namespace lr
