// lr_decay.cuh -- device helpers of the decayed linear attention.
//
// Log decays are summed in fixed point: a step's log2 decay becomes a 64-bit
// integer in units of 2^-32, so sums over any range are exact and do not
// depend on how the sequence is cut, and a reset (a decay of 0) does not eat
// the precision of the differences after it (2^-17 in a steep chunk's scores,
// whose exponents are kept in units of 2^-16).
#pragma once

#include "lr_decay.h"
#include "lr_device.cuh"

namespace lr {
namespace dec {

constexpr float kFixInv = 2.3283064365386963e-10f;   // 2^-32
// a step's floor: exp(-139) = 2^-200 is 0 in fp32, so this is a reset
constexpr float kFloor = -139.0f;
// The running state is kept divided by the decay since the last rescale, and
// rescaled once that decay falls below 2^-16.  Rescaling rarely matters for
// accuracy: a factor that is rounded once per chunk, and the same way every
// time, compounds over the slow heads' thousands of steps.
constexpr long long kRescale = -(16ll << 32);
// A chunk of the step-by-step kernel that alone decays further than this is
// run with the decay applied at every step.  With kRescale it bounds the
// factors 1 / A_t by 2^48, so v_t k_t products up to 2^80 stay finite.
constexpr long long kSteep = -(32ll << 32);

// log2 decay of a step in fixed point; `bad` is set for a value above 0 or
// not a number (read as 0).  The product with log2(e) is formed as a sum of two
// floats (its rounding error is exact by fma) and converted in two 16-bit
// steps: fp64 arithmetic, at 1/64 of the fp32 rate, made this the slowest
// link of the tensor-core kernel.
__device__ __forceinline__ long long to_fix(float l, bool &bad) {
    if (!(l <= 0.0f)) {
        bad = true;
        return 0;
    }
    constexpr float kHi = 1.44269504f, kLo = 1.92596299e-8f;   // log2(e) = kHi + kLo
    l = fmaxf(l, kFloor);
    const float p = l * kHi, r = fmaf(l, kLo, fmaf(l, kHi, -p));
    const int i1 = __float2int_rn(p * 65536.0f);                   // units of 2^-16, below 2^24
    const int i2 = __float2int_rn(fmaf(r, 4294967296.0f, (p * 65536.0f - float(i1)) * 65536.0f));
    return (static_cast<long long>(i1) << 16) + i2;
}

// A fixed-point exponent as a float.
__device__ __forceinline__ float fix_f(long long x) {
    return fmaf(static_cast<float>(static_cast<uint32_t>(x)), kFixInv, static_cast<float>(static_cast<int>(x >> 32)));
}

// An exponent of a chunk of 128 steps in units of 2^-16 (128 floors of -200.6 are above
// -2^15), so that a difference of two is exact however many resets lie before
// both; and one, or a difference, as a float.
__device__ __forceinline__ int units_of(long long x) { return static_cast<int>((x + (1 << 15)) >> 16); }
__device__ __forceinline__ float units_f(int u) { return 1.52587890625e-5f * static_cast<float>(u); }

// 2^x of a fixed-point exponent, for x below 127: 2^fraction times 2^integer,
// so the result is as exact for large exponents as for small ones (these
// factors multiply whole ranges of the state); 0 below 2^-126.
__device__ __forceinline__ float exp2_fix(long long x) {
    const int n = max(static_cast<int>(x >> 32), -127);
    return ex2_approx(static_cast<float>(static_cast<uint32_t>(x)) * kFixInv) * __int_as_float((n + 127) << 23);
}

// Step size of a selective scan with heads from dt + dt_bias.  softplus(x) = max(x, 0) +
// log1p(e), e = exp(-|x|) in (0, 1], with log1p(e) / e as a polynomial of degree 9 (its
// interpolation at Chebyshev nodes): 1.7e-7 relative with the roundings and an exact e, 2.7e-7
// with an e one place off, for x above -87; below, e itself is subnormal and has the error
// of its last place, 2^-149.
// The library's log1pf(expf(x)), four times in a row in one warp, took a chunk of the
// tensor-core kernel 10000 clocks against 4200 without.
__device__ __forceinline__ float step_size(float x, int softplus) {
    if (softplus == 0) return x;
    const float e = expf(-fabsf(x));
    float q = -0.00325637846f;
    q = fmaf(q, e, 0.0199071616f);
    q = fmaf(q, e, -0.0570642017f);
    q = fmaf(q, e, 0.106142648f);
    q = fmaf(q, e, -0.153118625f);
    q = fmaf(q, e, 0.196781173f);
    q = fmaf(q, e, -0.249545589f);
    q = fmaf(q, e, 0.333300054f);
    q = fmaf(q, e, -0.499999046f);
    q = fmaf(q, e, 1.0f);
    return fmaf(q, e, x > 0.0f ? x : 0.0f);
}

// A head's decays: of a step with gate value g the log decay, and in `w` the factor of
// its v k^T.
template <bool HEADS>
struct Gates {
    float l0, bias;
    int softplus;
    __device__ __forceinline__ Gates(const DecayArgs &a, int h) {
        l0 = a.a_log == nullptr ? 0.0f : a.a_log[h];
        if (HEADS) {
            l0 = -expf(l0);
            bias = a.hd.dt_bias == nullptr ? 0.0f : a.hd.dt_bias[h];
            softplus = a.hd.softplus;
        }
    }
    __device__ __forceinline__ float of(float g, float &w) const {
        w = HEADS ? step_size(g + bias, softplus) : 1.0f;
        if (HEADS) return w >= 0.0f ? l0 * w : 1.0f;   // (a negative or NaN step size is out of range)
        return l0 + g;
    }
    // elements between the gates of two steps
    __device__ __forceinline__ static int64_t pitch(const DecayArgs &a) { return HEADS ? a.hd.ldg : a.H; }
};

__device__ __forceinline__ int row_len(const int32_t *lens, int b, int64_t L) {
    if (lens == nullptr) return static_cast<int>(L);
    const int n = lens[b];
    return n < 0 ? 0 : (n > L ? static_cast<int>(L) : n);
}

// Whether one of segments 0 .. last of (batch row, head) bh left a tile that
// is not finite.  A whole warp calls it.
__device__ __forceinline__ bool any_bad(const DecayArgs &a, int64_t bh, int last, int tile) {
    int bad = 0;
    for (int s = threadIdx.x & 31; s <= last; s += 32) bad |= a.seg_bad[(bh * (a.n_seg - 1) + s) * a.seg_tiles + tile];
    return __any_sync(0xffffffffu, bad);
}

// The batch row of a grid's slot: rows by falling length, so that the longest
// start first and the last blocks to run are short.  The whole block calls it, with
// kOrderRows ints of shared memory.
__device__ __forceinline__ int row_at(const DecayArgs &a, int slot, int *scratch) {
    if (!a.by_length) return slot;
    const int n = int(a.B);
    for (int i = threadIdx.x; i < n; i += blockDim.x) scratch[i] = row_len(a.lens, i, a.L);
    __syncthreads();
    int at = -1;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        int before = 0;
        for (int j = 0; j < n; ++j) before += scratch[j] > scratch[i] || (scratch[j] == scratch[i] && j < i);
        if (before == slot) at = i;
    }
    __syncthreads();
    if (at >= 0) scratch[0] = at;
    __syncthreads();
    return scratch[0];
}

}  // namespace dec
}  // namespace lr
