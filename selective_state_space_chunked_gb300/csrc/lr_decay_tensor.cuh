// lr_decay_tensor.cuh -- what the tensor-core kernels of the decayed linear attention
// and of the selective scan with heads share.
#pragma once

#include <cudaTypedefs.h>

#include <mutex>

#include "lr_decay.cuh"
#include "lr_vec.cuh"

namespace lr {

namespace dt {
constexpr int C = kDecayChunk;
constexpr int RB = kDecayRows;
// the state is rescaled past this decay (log2)
constexpr long long kRescaleTensor = -(48ll << 32);
// decay of a chunk (log2) past which D is formed from differences
constexpr long long kSteepChunk = -(40ll << 32);

__device__ __forceinline__ void arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&p);
}
// One lane of a converged warp, the same at every call.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// w times a pair of bf16 values in three bf16 terms: what each leaves goes to
// the next, 24 bits in all.
__device__ __forceinline__ void three_terms(float w, uint32_t v, uint32_t &t1, uint32_t &t2, uint32_t &t3) {
    const float2 neg = make_float2(-1.0f, -1.0f);
    float2 y = __fmul2_rn(make_float2(w, w), make_float2(lo_f(v), hi_f(v)));
    t1 = pack(y.x, y.y);
    y = __ffma2_rn(neg, make_float2(lo_f(t1), hi_f(t1)), y);
    t2 = pack(y.x, y.y);
    y = __ffma2_rn(neg, make_float2(lo_f(t2), hi_f(t2)), y);
    t3 = pack(y.x, y.y);
}

// What a wait that does not succeed at once needs, in shared memory.
struct Ctl {
    unsigned long long *word;
    unsigned long long stamp;
    uint64_t timeout_ns;
    int abort_flag;
    int redo;   // a value that is not finite was written
    int row;    // the block's batch row
};
static_assert(sizeof(Ctl) <= 40, "");

// The slow path of every wait (one copy of the code): bounded; the first to
// run out makes every role leave its loop.  The limit is for this launch's own work: a
// role may be waiting for another that still waits for an earlier launch of the call, which
// may take longer (a segment's steps one at a time are 1 us each), so the first time that the
// limit runs out that launch's end is awaited and the limit starts over.
static __device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, Ctl *ctl) {
    uint64_t t0 = 0;
    bool alone = false;   // no earlier launch is still running
    for (uint32_t n = 1;; ++n) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((n & 15) != 0) continue;
        // reading the timer is slow: every 16th try
        if (*reinterpret_cast<volatile int *>(&ctl->abort_flag) != 0) return false;
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > ctl->timeout_ns && !alone) {
            grid_dependency_wait();
            alone = true;
            t0 = globaltimer_ns();
        } else if (now - t0 > ctl->timeout_ns) {
            *reinterpret_cast<volatile int *>(&ctl->abort_flag) = 1;
            status_report(StatusRef{ctl->word, ctl->stamp}, LR_ERR_TIMEOUT);
            return false;
        }
    }
}

// The limit of a call's waits.
inline uint64_t wait_limit_ns() {
    return g_withheld_split >= 1 ? uint64_t(g_withheld_timeout_ms) * 1000000ull : kDefaultTimeoutNs;
}

// 0 times the values that were written, added up: no 0 once one was not finite.
__device__ __forceinline__ bool not_finite(float2 z) { return !(z.x + z.y == 0.0f); }

// The block's value rows over its segment once more, a step at a time in fp32: the
// recurrence as it stands, for blocks whose products met an infinity, a NaN or
// an overflow.  The whole block calls it, with its operands' shared memory free.
// Four lanes share a value row.  The decay comes in two floats: one, rounded the
// same way at every step, would add up over the slow heads' thousands of steps.
// About 1 us a step, against 0.02 of the matrix form; only blocks that met such a
// value pay it.
template <bool STATE_ONLY, bool HEADS>
__device__ __forceinline__ void redo_block(const DecayArgs &a, int b, int n_vt, unsigned char *sm) {
    constexpr int T = 16, W = kPartKeys, RB = kDecayRows;
    using bf = __nv_bfloat16;
    float *sk = reinterpret_cast<float *>(sm), *sq = sk + T * W, *sv = sq + T * W;
    float2 *sa = reinterpret_cast<float2 *>(sv + T * RB);
    // [m][256]: key columns 4 p + 16 m .. + 3, each its thread's own (in registers, the
    // call's 64 made the kernel's other code slower: 87.9 us against 87.0)
    float *sd = reinterpret_cast<float *>(sa + T);   // [T] step sizes (heads)
    float4 *S = reinterpret_cast<float4 *>(sd + T) + threadIdx.x;
    // the block's place in the grid
    const int nseg = STATE_ONLY ? a.n_seg - 1 : a.n_seg;
    int x = blockIdx.x;
    const int vt = x % n_vt;
    x /= n_vt;
    const int part = x % a.parts;
    x /= a.parts;
    const int seg = x % nseg, h = x / nseg % a.H;
    const int tid = threadIdx.x, i = tid >> 2, p = tid & 3, ldk = a.dk, k0 = W * part;
    const int dk = min(W, ldk - k0), dv = a.dv, row = vt * RB + i, hk = h / (a.H / a.Hk);
    const bool mine = tid < 4 * RB, in = mine && row < dv;   // whole warps
    const int64_t bh = int64_t(b) * a.H + h, s0 = int64_t(seg) * a.seg_len;
    const int nrun = int(max(int64_t(0), min(int64_t(dec::row_len(a.lens, b, a.L)), min(a.L, s0 + a.seg_len)) - s0));
    const size_t HV = size_t(a.H) * dv, at0 = size_t(b) * a.L + s0, GP = dec::Gates<HEADS>::pitch(a);
    const size_t LK = HEADS ? size_t(a.hd.ldk) : size_t(a.Hk) * ldk, LQ = HEADS ? size_t(a.hd.ldq) : LK;
    const size_t LV = HEADS ? size_t(a.hd.ldv) : HV;
    const bf *q = static_cast<const bf *>(a.q) + at0 * LQ + size_t(hk) * ldk + k0;
    const bf *k = static_cast<const bf *>(a.k) + at0 * LK + size_t(hk) * ldk + k0;
    const bf *v = static_cast<const bf *>(a.v) + at0 * LV + size_t(h) * dv + vt * RB;
    const bf *g = a.g == nullptr ? nullptr : static_cast<const bf *>(a.g) + at0 * GP + h;
    const bf *z = nullptr;
    if (HEADS && !STATE_ONLY && a.hd.z != nullptr && a.parts == 1)
        z = static_cast<const bf *>(a.hd.z) + at0 * size_t(a.hd.ldz) + size_t(h) * dv + row;
    const bool has_skip = HEADS && !STATE_ONLY && a.hd.skip != nullptr && part == 0;
    const float skip = has_skip ? a.hd.skip[h] : 0.0f;
    bf *o = static_cast<bf *>(a.o) + at0 * HV + size_t(h) * dv + row;
    float *op = a.parts > 1 ? a.o_part + ((size_t(part) * a.B + b) * a.L + s0) * HV + size_t(h) * dv + row : nullptr;
    const dec::Gates<HEADS> gates(a, h);
    // this thread's columns: those that are there, of a row that is (dk is a multiple of 8)
    const int nm = in ? (dk / 4 - p + 3) / 4 : 0;
    const size_t at_S = size_t(row) * ldk + k0 + 4 * p;
    auto four = [&](const float *src, int m) { return *reinterpret_cast<const float4 *>(src + at_S + 16 * m); };
    const bool from_S0 = seg == 0 && a.S0 != nullptr;
#pragma unroll 1
    for (int m = 0; m < nm; ++m)
        S[256 * m] = from_S0 ? four(a.S0 + bh * dv * ldk, m) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (!STATE_ONLY && seg > 0) {
        grid_dependency_wait();
        long long acc = 0;
#pragma unroll 1
        for (int e = seg - 1; e >= 0; --e) {
            const size_t at = bh * (a.n_seg - 1) + e;
            const float f = dec::exp2_fix(acc);
#pragma unroll 1
            for (int m = 0; m < nm; ++m) {
                const float4 s = four(a.seg_state + at * dv * ldk, m), y = S[256 * m];
                S[256 * m] = make_float4(fmaf(f, s.x, y.x), fmaf(f, s.y, y.y), fmaf(f, s.z, y.z), fmaf(f, s.w, y.w));
            }
            acc = max(acc + a.seg_tot[at], -(1ll << 60));
        }
    }
#pragma unroll 1
    for (int t0 = 0; t0 < nrun; t0 += T) {
        const int n = min(T, nrun - t0);
        __syncthreads();   // the last steps have been read
#pragma unroll 1
        for (int e = tid; e < n * W; e += blockDim.x) {
            const int t = e / W, j = e % W;
            sk[e] = j < dk ? __bfloat162float(k[size_t(t0 + t) * LK + j]) : 0.0f;
            if (!STATE_ONLY) sq[e] = j < dk ? __bfloat162float(q[size_t(t0 + t) * LQ + j]) : 0.0f;
        }
#pragma unroll 1
        for (int e = tid; e < n * RB; e += blockDim.x)
            sv[e] = vt * RB + e % RB < dv ? __bfloat162float(v[size_t(t0 + e / RB) * LV + e % RB]) : 0.0f;
        if (tid < n) {
            float w, l = gates.of(g != nullptr ? __bfloat162float(g[size_t(t0 + tid) * GP]) : 0.0f, w);
            if (!(l <= 0.0f)) l = 0.0f;   // (has been reported)
            if (HEADS) sd[tid] = w;
            const float e = expm1f(l), hi = 1.0f + e;
            sa[tid] = l > -1.0f ? make_float2(hi, e - (hi - 1.0f)) : make_float2(expf(l), 0.0f);
        }
        __syncthreads();
        if (!mine) continue;
#pragma unroll 1
        for (int t = 0; t < n; ++t) {
            const float2 at = sa[t];
            const float vi = HEADS ? sd[t] * sv[t * RB + i] : sv[t * RB + i];
            float acc = 0.0f;
            auto step = [&](float x, float kj) {
                const float u = vi * kj;   // (the decay's rest may be 0 or negative: not times an infinity)
                return fmaf(at.x, x, fabsf(x) <= 3.4e38f ? fmaf(at.y, x, u) : u);
            };
#pragma unroll 1
            for (int m = 0; m < nm; ++m) {
                const float4 x = S[256 * m], k4 = reinterpret_cast<const float4 *>(sk + t * W)[p + 4 * m];
                const float4 y = make_float4(step(x.x, k4.x), step(x.y, k4.y), step(x.z, k4.z), step(x.w, k4.w));
                S[256 * m] = y;
                if (STATE_ONLY) continue;
                const float4 q4 = reinterpret_cast<const float4 *>(sq + t * W)[p + 4 * m];
                acc = fmaf(y.x, q4.x, fmaf(y.y, q4.y, fmaf(y.z, q4.z, fmaf(y.w, q4.w, acc))));
            }
            if (STATE_ONLY) continue;
            acc += __shfl_xor_sync(0xffffffffu, acc, 1);
            acc += __shfl_xor_sync(0xffffffffu, acc, 2);
            if (in && p == 0) {
                float y = a.scale * acc;
                if (has_skip) y = fmaf(skip, sv[t * RB + i], y);
                if (HEADS && z != nullptr) y *= silu_f(__bfloat162float(z[size_t(t0 + t) * a.hd.ldz]));
                if (op != nullptr)
                    op[size_t(t0 + t) * HV] = y;
                else
                    o[size_t(t0 + t) * HV] = __float2bfloat16_rn(y);
            }
        }
    }
    float *dst = STATE_ONLY ? a.seg_state + (bh * (a.n_seg - 1) + seg) * dv * ldk
                 : seg == a.n_seg - 1 && a.S_final != nullptr ? a.S_final + bh * dv * ldk : nullptr;
    if (dst == nullptr) return;
#pragma unroll 1
    for (int m = 0; m < nm; ++m) *reinterpret_cast<float4 *>(dst + at_S + 16 * m) = S[256 * m];
}
// The kernels' other code comes out best with this as a call without parts and
// inlined with them (B4 L4096 H16 d128 87.0 us against 87.1, B1 L32768 234 against
// 240; dk256 279 against 261).
template <bool STATE_ONLY, bool HEADS>
__device__ __noinline__ void redo_call(const DecayArgs &a, int b, int n_vt, unsigned char *sm) {
    redo_block<STATE_ONLY, HEADS>(a, b, n_vt, sm);
}
}  // namespace dt

// o = the parts' sum, rounded once; steps past a row's length are 0.  A block
// takes whole steps (all heads of one token).  Launched while the parts drain: B1
// L100 H8 dk256 13.0 us against 15.3, B2 L1500 H8 dk256 49.4 against 51.5 (11.9 and
// 48.0 now).  It lets
// nothing start before its own end (B4 L4096 H16 dk256 277 us against 270: the next
// call's blocks would take the SMs that it still needs).
template <bool HEADS>
__global__ void __launch_bounds__(256) decay_parts_kernel(const DecayArgs a) {
    using dt::pack;
    grid_dependency_wait();
    const int64_t rows = a.B * a.L, HV = int64_t(a.H) * a.dv;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const int b = int(row / a.L);
        const bool valid = row - b * a.L < dec::row_len(a.lens, b, a.L);
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.o) + row * HV);
        for (int i = threadIdx.x; i < HV / 8; i += 256) {
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f), y = x;
            if (valid) {
                for (int p = 0; p < a.parts; ++p) {
                    const float4 *src = reinterpret_cast<const float4 *>(a.o_part + (p * rows + row) * HV) + 2 * i;
                    const float4 u = __ldcs(src), v = __ldcs(src + 1);
                    x = make_float4(x.x + u.x, x.y + u.y, x.z + u.z, x.w + u.w);
                    y = make_float4(y.x + v.x, y.y + v.y, y.z + v.z, y.w + v.w);
                }
                if (HEADS && a.hd.z != nullptr) {
                    const uint4 z =
                        reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.hd.z) + row * a.hd.ldz)[i];
                    x = make_float4(x.x * silu_f(dt::lo_f(z.x)), x.y * silu_f(dt::hi_f(z.x)),
                                    x.z * silu_f(dt::lo_f(z.y)), x.w * silu_f(dt::hi_f(z.y)));
                    y = make_float4(y.x * silu_f(dt::lo_f(z.z)), y.y * silu_f(dt::hi_f(z.z)),
                                    y.z * silu_f(dt::lo_f(z.w)), y.w * silu_f(dt::hi_f(z.w)));
                }
            }
            dst[i] = make_uint4(pack(x.x, x.y), pack(x.z, x.w), pack(y.x, y.y), pack(y.z, y.w));
        }
    }
}

namespace {

PFN_cuTensorMapEncodeTiled_v12000 dt_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// bf16 map over (d, heads, L, B): 64 columns of one head by 128 steps, 128-byte
// swizzle; columns past d and steps past L arrive as zeros
// (ld: elements between steps, 0: dense)
bool dt_map(CUtensorMap *tm, const void *base, uint64_t d, uint64_t heads, uint64_t L, uint64_t B, uint64_t ld) {
    auto enc = dt_encoder();
    if (enc == nullptr) return false;
    const cuuint64_t dims[4] = {d, heads, L, B};
    if (ld == 0) ld = d * heads;
    const cuuint64_t strides[3] = {d * 2, ld * 2, ld * L * 2};
    const cuuint32_t box[4] = {64, 1, uint32_t(dt::C), 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

}  // namespace lr
