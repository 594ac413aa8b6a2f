// lr_rope.cu -- norm of every head of the queries and the keys, and the rotation of
// its pairs by the token's position, in one pass:
//   n = gamma x / sqrt(mean(x^2) + eps)   (rms; l2: the sum of the squares; none: gamma x)
//   (a, b) = pair i of n:  (a cos - b sin, b cos + a sin),  angle pos freqs[i]
//
// Every value is read once and written once, so memory bandwidth is the bound (the
// launch's latency for a few tokens).  The lanes that share a head each hold both
// partners of their pairs, so the norm is one sum over lanes and the rotation needs no
// exchange; gamma times cosine and sine stay in registers for all heads of a token that
// a set of lanes takes.  Measured on slices of a projection, in turn over 500 MB: bf16
// 16384 tokens, 16 + 4 heads of 128 32.5 us (76 % of the copy bandwidth), half rotated in
// neighbouring pairs 32.5; fp32 8192 tokens 27.7 (90 %); bf16 16384 tokens, 32 + 8 heads of
// 64 28.8; 8 tokens 2.0.  No unit is near its limit in bf16 (issue 59 %, LSU 38 %, fp32 pipe
// 24 %, 43 % of the warps): a set's loads wait for its last ones' sums and stores.  What its
// operations and loads cost on the way (27 million warp instructions at first):
//   angles for every set of lanes 37 us, once a token into shared memory 36
//   one head ahead in flight 38 us, four heads' loads at once 36
//   blocks of whole tokens, without 64-bit divisions, in sizes that fit them 32.6
//
// Angles.  freqs is turned into a 64-bit fraction of a turn, exact to 2^-64, whose product
// with the position wraps by itself: far positions and high frequencies lose nothing to the
// size of their angle (2^-33 of a turn at position 2^31).
#include "lr_decay.cuh"
#include "lr_vec.cuh"

namespace lr {
namespace {

constexpr int kRopeT = 256;   // threads of a block at most

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
    int sets, q_sets, heads;   // lane sets of a token, those of its queries, heads of each
    int tokens;                // of a block
};

// The part of a turn that a position adds, in units of 2^-64: the float's own 24 bits times
// 1 / 2 pi in 128.
__device__ __forceinline__ unsigned long long turn_of(float f) {
    constexpr unsigned long long kHi = 0x28be60db9391054aull, kLo = 0x7f09d5f47d4d3770ull;   // 1 / 2 pi, in units of 2^-64 and 2^-128
    const uint32_t u = __float_as_uint(f);
    const int ex = max(int(u >> 23 & 255), 1), s = 150 - ex;              // |f| = m 2^-s
    const unsigned long long m = (u & 0x7fffff) | ((u >> 23 & 255) != 0 ? 0x800000u : 0u);
    const unsigned long long c = __umul64hi(m, kLo), lo = m * kHi + c, hi = __umul64hi(m, kHi) + (lo < c);
    unsigned long long t = 0;
    if (s <= 0)
        t = s > -64 ? lo << -s : 0;
    else if (s < 64)
        t = lo >> s | hi << (64 - s);
    else if (s < 128)
        t = hi >> (s - 64);
    return u >> 31 ? 0 - t : t;
}

// Sine and cosine of a fraction of a turn.  EXACT: to fp32's last places; else by the
// special function unit, to 2^-21, which outputs of 8 bits do not see.
template <bool EXACT>
__device__ __forceinline__ void sin_cos(unsigned long long t, float &s, float &c) {
    if (EXACT) {
        sincospif(1.0842021724855044e-19f * __ll2float_rn(static_cast<long long>(t)), &s, &c);   // half turns
    } else {
        const float x = 1.4629180792671596e-9f * static_cast<float>(static_cast<int>(t >> 32));   // 2 pi 2^-32
        s = __sinf(x), c = __cosf(x);
    }
}
// Values at .. at + VN - 1 of the factors g (1 without any).
template <int VN>
__device__ __forceinline__ void factors_of(const float *g, int at, bool in, float *f) {
    if constexpr (VN % 4 == 0) {
#pragma unroll
        for (int e = 0; e < VN; e += 4) {
            float4 w = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
            if (g != nullptr && in) w = *reinterpret_cast<const float4 *>(g + at + e);
            f[e] = w.x, f[e + 1] = w.y, f[e + 2] = w.z, f[e + 3] = w.w;
        }
    } else {
        f[0] = g != nullptr && in ? g[at] : 1.0f;
    }
}

// TL lanes a head; U units a lane, each of two vectors of X::N values.
//   halves      (NB = 0, pair i: values i and i + rot / 2): unit u holds vectors u
//               and u + rot / 2 / N
//   neighbours  (pair i: values 2 i and 2 i + 1): vectors 2 u and 2 u + 1, whose pairs
//               lie inside them; of single values they are the pair
// Units past the rotated ones hold two vectors that are only normalised.  A set of lanes
// takes `heads` heads of one token, all queries or all keys, so that the factors of its
// pairs, gamma times cosine and sine, stay in registers: four products a pair.
// NH heads' loads are in flight at once, the first ones' while the angles are formed.
template <typename X, int TL, int U, int NH, bool NB>
__global__ void __launch_bounds__(kRopeT) rope_kernel(const RopeArgs a) {
    using Raw = typename X::Raw;
    constexpr int VN = X::N;
    constexpr bool INSIDE = NB && VN > 1;   // pairs inside a vector
    launch_dependents();
    grid_dependency_wait();
    const int l = threadIdx.x % TL;
    // a block takes whole tokens, or of one that has more sets than it a part
    int first = int(blockIdx.y * (blockDim.x / TL) + threadIdx.x / TL);
    const int token = first / a.sets;
    first -= token * a.sets;
    const int64_t n0 = int64_t(blockIdx.x) * a.tokens, n = n0 + token;
    const bool live = token < a.tokens && n < a.N;
    const bool key = first >= a.q_sets;
    if (key) first -= a.q_sets;
    first *= a.heads;
    const int H = key ? a.Hk : a.H, count = live ? min(a.heads, H - first) : 0;   // of the set's heads
    const int nv = a.d / VN, rv = a.rot / 2 / VN, nr = a.rot / 2;
    const Raw *src = static_cast<const Raw *>(key ? a.k : a.q) + n * ((key ? a.ldk : a.ldq) / VN) + int64_t(first) * nv;
    Raw *dst = static_cast<Raw *>(key ? a.ko : a.qo) + (n * H + first) * int64_t(nv);
    int va[U], vb[U];          // a unit's vectors
    bool ina[U], inb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int un = l + u * TL;
        const bool halves = !NB && un < rv;
        va[u] = halves ? un : 2 * un, vb[u] = halves ? un + rv : 2 * un + 1;
        ina[u] = va[u] < nv, inb[u] = vb[u] < nv;
    }
    Raw r[NH][U][2];
    auto load = [&](int i) {
#pragma unroll
        for (int k = 0; k < NH; ++k)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                r[k][u][0] = i + k < count && ina[u] ? src[k * nv + va[u]] : Raw{};
                r[k][u][1] = i + k < count && inb[u] ? src[k * nv + vb[u]] : Raw{};
            }
        src += NH * nv;
    };
    load(0);
    // cosines and sines of the block's tokens, once for all their sets
    extern __shared__ float2 turns[];
    if (nr > 0) {
        const int tokens = int(min(int64_t(a.tokens), a.N - n0));
        for (int i = threadIdx.x; i < tokens * nr; i += blockDim.x) {
            const int t = i / nr;
            const unsigned long long at =
                turn_of(a.freqs[i - t * nr]) * static_cast<unsigned long long>(static_cast<long long>(a.pos[n0 + t]));
            float s, c;
            sin_cos<sizeof(Raw) == VN * 4>(at, s, c);
            turns[i] = make_float2(c, s);
        }
        __syncthreads();
    }
    const float2 *mine = turns + token * nr;
    // pair e of a unit, (v, w):  v' = A v + B w,  w' = C w + D v
    float A[U][VN], Bc[U][VN], Cc[U][VN], Dc[U][VN];
    int turned[U];             // its pairs that are rotated
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int un = l + u * TL;
        turned[u] = NB ? max(0, min(VN, nr - un * VN)) : un < rv ? VN : 0;
        float ga[VN], gb[VN];
        const float *g = key ? a.gk : a.gq;
        factors_of<VN>(g, va[u] * VN, ina[u], ga);
        factors_of<VN>(g, vb[u] * VN, inb[u], gb);
#pragma unroll
        for (int e = 0; e < VN; ++e) {
            float s = 0.0f, c = 1.0f;
            if (live && e < turned[u]) c = mine[un * VN + e].x, s = mine[un * VN + e].y;
            const float gv = !INSIDE ? ga[e] : 2 * e < VN ? ga[(2 * e) % VN] : gb[(2 * e) % VN];
            const float gw = !INSIDE ? gb[e] : 2 * e < VN ? ga[(2 * e + 1) % VN] : gb[(2 * e + 1) % VN];
            A[u][e] = gv * c, Bc[u][e] = -gw * s, Cc[u][e] = gw * c, Dc[u][e] = gv * s;
        }
    }
    const float inv_d = a.norm == LR_NORM_RMS ? 1.0f / float(a.d) : 1.0f;
    // (every lane of the warp goes through all a.heads turns: the sum needs them)
    auto head = [&](Raw (&rk)[U][2], bool in) {
        float x[U][2 * VN];   // a unit's two vectors
        float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            X::widen(rk[u][0], x[u]);
            X::widen(rk[u][1], x[u] + VN);
#pragma unroll
            for (int e = 0; e < VN; ++e) s2 = __ffma2_rn(pair(x[u] + 2 * e), pair(x[u] + 2 * e), s2);
        }
        float rs = 1.0f;
        if (a.norm != LR_NORM_NONE) {
            float s = s2.x + s2.y;
#pragma unroll
            for (int m = TL / 2; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
            rs = rsqrtf(fmaf(s, inv_d, a.eps));
        }
        const float2 rs2 = make_float2(rs, rs);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float *p = x[u], *q = x[u] + VN;
            if constexpr (VN == 1 || INSIDE) {
#pragma unroll
                for (int e = 0; e < VN; ++e) {
                    float &v = x[u][INSIDE ? 2 * e : e], &w = x[u][INSIDE ? 2 * e + 1 : VN + e];
                    const float v0 = v * rs, w0 = w * rs;
                    v = A[u][e] * v0, w = Cc[u][e] * w0;
                    if (e < turned[u]) v = fmaf(Bc[u][e], w0, v), w = fmaf(Dc[u][e], v0, w);
                }
            } else {
#pragma unroll
                for (int e = 0; e < VN; e += 2) {
                    const float2 v0 = __fmul2_rn(pair(p + e), rs2), w0 = __fmul2_rn(pair(q + e), rs2);
                    float2 v = __fmul2_rn(pair(A[u] + e), v0), w = __fmul2_rn(pair(Cc[u] + e), w0);
                    if (turned[u] > 0) {
                        v = __ffma2_rn(pair(Bc[u] + e), w0, v);
                        w = __ffma2_rn(pair(Dc[u] + e), v0, w);
                    }
                    p[e] = v.x, p[e + 1] = v.y, q[e] = w.x, q[e + 1] = w.y;
                }
            }
            if (in && ina[u]) dst[va[u]] = X::narrow(p);
            if (in && inb[u]) dst[vb[u]] = X::narrow(q);
        }
        dst += nv;
    };
#pragma unroll 1
    for (int i = 0; i < a.heads; i += NH) {
        if (i > 0) load(i);
#pragma unroll
        for (int k = 0; k < NH; ++k) head(r[k], i + k < count);
    }
}

template <typename X, int TL, int U, int NH, bool NB>
int rope_go(RopeArgs a, cudaStream_t s) {
    int sms = 0;
    if (device_sm_count(&sms) != LR_OK) return LR_ERR_CUDA;
    // heads of a set: the fewest idle turns and repeated angles (which cost about two
    // heads), as long as every SM has its threads
    auto sets = [&](int64_t h) { return (a.H + h - 1) / h + (a.Hk + h - 1) / h; };
    a.heads = 1;
    for (int h = 2; h <= 8; ++h)
        if (sets(h) * (h + 2) < sets(a.heads) * (a.heads + 2) && a.N * sets(h) * TL >= int64_t(sms) * 1024) a.heads = h;
    a.sets = int(sets(a.heads));
    a.q_sets = (a.H + a.heads - 1) / a.heads;
    // tokens of a block: whole warps with the fewest idle lanes, of about 128 threads
    auto threads = [&](int64_t t) { return (t * a.sets * TL + 31) / 32 * 32; };
    a.tokens = 1;
    int block = int(threads(1) < kRopeT ? threads(1) : kRopeT);
    double best = 0.0;
    for (int t = 1; t == 1 || threads(t) <= kRopeT; ++t) {
        const double used = double(int64_t(t) * a.sets * TL) / double(threads(t)) + (threads(t) >= 128 ? 0.1 : 0.0);
        if (threads(t) <= kRopeT && used > best) best = used, a.tokens = t, block = int(threads(t));
        if (threads(t) >= 128 && best >= 1.1) break;
    }
    const int64_t parts = (int64_t(a.sets) * TL * a.tokens + block - 1) / block;   // (500000 heads: 62500)
    const dim3 grid(unsigned((a.N + a.tokens - 1) / a.tokens), unsigned(parts));
    // a head a set: without the registers of the others (decode: 2.6 us against 2.9)
    return launch_kernel(a.heads == 1 ? rope_kernel<X, TL, U, 1, NB> : rope_kernel<X, TL, U, NH, NB>, true,
                         grid, block, size_t(a.tokens) * (a.rot / 2) * sizeof(float2), s, a);
}

template <typename IO, bool NB>
int rope_pairs(const RopeArgs &a, cudaStream_t s) {
    constexpr int V = 4;
    // whole vectors where every head starts on one and no vector holds both partners' halves;
    // of four values in bf16 too: 16384 tokens 16 + 4 heads d128 32.6 us, with eight 38.4
    if (a.d % V == 0 && a.ldq % V == 0 && a.ldk % V == 0 && (NB || a.rot / 2 % V == 0)) {
        using X = Vec<IO, V>;
        const int units = (a.d / V + 1) / 2;
        if (units <= 2) return rope_go<X, 2, 1, 4, NB>(a, s);
        if (units <= 4) return rope_go<X, 4, 1, 4, NB>(a, s);
        if (units <= 8) return rope_go<X, 8, 1, 4, NB>(a, s);
        if (units <= 16) return rope_go<X, 16, 1, 4, NB>(a, s);
        if (units <= 32) return rope_go<X, 32, 1, 4, NB>(a, s);
        if constexpr (V == 4) return rope_go<X, 32, 2, 2, NB>(a, s);
    }
    using X = Vec<IO, 1>;
    const int units = (a.d + 1) / 2;
    if (units <= 32) return rope_go<X, 32, 1, 1, NB>(a, s);
    if (units <= 64) return rope_go<X, 32, 2, 1, NB>(a, s);
    if (units <= 128) return rope_go<X, 32, 4, 1, NB>(a, s);
    return rope_go<X, 32, 8, 1, NB>(a, s);
}

}  // namespace

int head_norm_rope_launch(const void *q, int64_t ldq, const void *k, int64_t ldk, const float *gq, const float *gk,
                          const float *freqs, const int32_t *pos, void *qo, void *ko, int64_t N, int64_t H, int64_t Hk,
                          int64_t d, int64_t rot, int norm, float eps, int pairs, int io_bf16, cudaStream_t stream) {
    if (N == 0 || H + Hk == 0) return LR_OK;
    const RopeArgs a{q, k, ldq, ldk, gq, gk, freqs, pos, qo, ko, N, int(H), int(Hk), int(d), int(rot), norm, eps, 0, 0, 0, 0};
    const bool nb = pairs == LR_PAIRS_NEIGHBOURS;
    if (io_bf16) return nb ? rope_pairs<__nv_bfloat16, true>(a, stream) : rope_pairs<__nv_bfloat16, false>(a, stream);
    return nb ? rope_pairs<float, true>(a, stream) : rope_pairs<float, false>(a, stream);
}

}  // namespace lr
