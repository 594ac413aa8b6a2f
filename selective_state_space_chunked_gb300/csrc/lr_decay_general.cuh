// lr_decay_general.cuh -- decayed linear attention on the CUDA cores: fp32
// I/O, head dims the tensor-core kernel does not take, and short sequences.
//
//   S_t = a_t S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t,   a_t = exp(l_t)
//
// Step by step in fp32.  A block owns RB value rows of one
// (batch row, head, time segment); a thread owns RT rows and CPT key columns
// of each, in registers, so P = DKP / CPT consecutive lanes share a row.  The
// columns come in groups of four dealt round-robin, so the lanes of a row
// read consecutive 16 bytes of k_t and q_t from shared memory.
//
// One decay for the whole state: instead of multiplying S by a_t at every
// step (a third operation beside the update's and the readout's), the thread
// keeps S^ = S / A_t, A_t the decay since the last rescale, and takes
//   S^ += (v_t / A_t) k_t^T,   o_t = scale A_t (S^ q_t),
// two packed fp32x2 operations per pair of state elements.  After a chunk
// with A < 2^-16 the state is rescaled.  A chunk that alone decays below
// 2^-32 (resets included) runs with the multiplication at every step.
//
// k, q, v arrive in chunks of TC steps, by TMA where every row start is
// 16-byte aligned, else element by element, kGB - 1 chunks ahead.
//
// The work is 2 dk dv fp32 fused multiply-adds per token and head and, in the
// n - 1 of n segments that the first launch runs, dk dv more.  Measured (fp32,
// H16 d128): B2 L2048 201 us, 9 segments, 3.1 G fused multiply-adds, 41 % of
// the fp32 pipes' rate; B4 L4096 668 us; B1 L32768 1267 us.  The packed fp32 pipe
// is busy 53-55 % of the time the SMs are; the rest goes to the latency of a step
// (its loads from shared memory, the chains of dependent sums, the sums over
// lanes), which four warps per scheduler do not cover, and to the last blocks.
//   chunks of 16 steps in two buffers against 8 in three: 222 us against 239
//   the steep chunk's multiplications in a loop of their own: 205 against 222
//   one barrier a chunk (outputs in two buffers): 204 against 205.5
//   two steps unrolled: 200 against 204; four: 213
//   two steps' sums over lanes taken together: 210 against 205 (spills)
//   blocks of 256 threads: 211 against 205; three blocks per SM: 266 against 204
// (each pair measured on the kernel of its time)
//
// Infinities and NaN go through the state as the recurrence takes them.  A segment
// says whether the state it leaves is finite (seg_bad), so that a later one does not
// pass over an infinity whose decay factor is 0.  S^ is up to 2^48 times S, so a
// state past 2^79 may overflow.
#pragma once

#include "lr_decay.cuh"

namespace lr {
namespace {

constexpr int kGB = 2;    // staging buffers

// A thread holds RT x CPT state elements.  4 x 16 leaves room for four warps
// per scheduler; 4 x 32 and 8 x 16 read less from shared memory per element but
// leave 1.5, and the packed fp32 pipe was then busy 37 % of the time (278 against
// 242 us at B2 L2048 H16 d128 fp32).  From 256 key columns three blocks per SM,
// without spills, take 115 us against 137 (fp32 B3 L1111 H6 dk192 dv96).  Up to
// 64 key columns chunks of 32 steps take 104 us against 118 (fp32 B1 L8192 H4
// d64), and 4 x 8 elements, which make twice the blocks, 73 against 91 there, 289
// against 310 at B4 L4096 H16 d64, 98 against 87 at B8 L1000 H8 d64; at 128 columns
// 4 x 8 take 410 us and 8 x 8 212 against 200 (B2 L2048 H16 d128).
template <int DKP_, bool NARROW>
struct DecCfg {
    static constexpr int DKP = DKP_;
    static constexpr int CPT = DKP <= 64 ? 8 : 16;
    static constexpr int RT = NARROW ? 1 : 4;
    static constexpr int NT = NARROW || DKP <= 64 ? 64 : 128;   // threads per block
    static constexpr int P = DKP / CPT;
    static constexpr int RB = RT * NT / P;
    static constexpr int KB = DKP < 256 ? DKP : 256;   // key columns per TMA box
    static constexpr int NH = DKP / KB;
    static constexpr int BPS = DKP >= 256 ? 3 : 512 / NT;   // blocks an SM is to hold
    // steps per staged chunk
    template <typename IO>
    __host__ __device__ static constexpr int steps() {
        constexpr int most = DKP <= 64 ? 32 : 16;
        return 16384 / int(DKP * sizeof(IO)) < most ? 16384 / int(DKP * sizeof(IO)) : most;
    }
    template <typename IO>
    __host__ __device__ static constexpr int pitch(int n) {
        return int((n * sizeof(IO) + 127) / 128 * 128 / sizeof(IO));
    }
    template <typename IO>
    static constexpr size_t smem_bytes() {
        constexpr int TC = steps<IO>();
        return sizeof(IO) * size_t(kGB) * (2 * pitch<IO>(TC * DKP) + pitch<IO>(TC * RB)) +
               sizeof(float) * (2 * TC * RB + 8 * TC) + kGB * sizeof(uint64_t) + 128;
    }
};

template <typename IO>
__device__ __forceinline__ float4 dec_ld4(const IO *p);
template <>
__device__ __forceinline__ float4 dec_ld4<float>(const float *p) {
    return *reinterpret_cast<const float4 *>(p);
}
template <>
__device__ __forceinline__ float4 dec_ld4<__nv_bfloat16>(const __nv_bfloat16 *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                       __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}

// Sums of RT values over the P lanes of a row group.  RT <= P: a reduce-scatter
// (RT - 1 shuffles), after which lane p holds the sum of value p % RT in a[0];
// RT = 1: every lane holds the sum.
template <int RT, int P>
__device__ __forceinline__ void row_sums(float (&a)[RT], int p) {
    static_assert(RT <= P, "a lane per value");
#pragma unroll
    for (int m = 1, n = RT; m < RT; m <<= 1, n >>= 1) {   // n values left, lanes m apart
        const bool up = p & m;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float keep = up ? a[2 * i + 1] : a[2 * i], send = up ? a[2 * i] : a[2 * i + 1];
            a[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
        }
    }
#pragma unroll
    for (int m = RT; m < P; m <<= 1) a[0] += __shfl_xor_sync(0xffffffffu, a[0], m);
}

// Columns j .. j + 3 of a state row of dk columns; v4: 16-byte rows.
__device__ __forceinline__ float4 state_ld4(const float *r, int j, int dk, bool v4) {
    if (v4) return j < dk ? *reinterpret_cast<const float4 *>(r + j) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    return make_float4(j < dk ? r[j] : 0.0f, j + 1 < dk ? r[j + 1] : 0.0f, j + 2 < dk ? r[j + 2] : 0.0f,
                       j + 3 < dk ? r[j + 3] : 0.0f);
}
__device__ __forceinline__ void state_st4(float *r, int j, int dk, bool v4, float4 s) {
    if (v4) {
        if (j < dk) *reinterpret_cast<float4 *>(r + j) = s;
        return;
    }
    if (j < dk) r[j] = s.x;
    if (j + 1 < dk) r[j + 1] = s.y;
    if (j + 2 < dk) r[j + 2] = s.z;
    if (j + 3 < dk) r[j + 3] = s.w;
}

// STATE_ONLY: the first launch of a segmented call (no q, no output; segments
// 0 .. n_seg - 2).
template <typename IO, typename C, bool STATE_ONLY>
__global__ void __launch_bounds__(C::NT, C::BPS)
    decay_general_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const DecayArgs a, int nrb, bool tma,
                         uint64_t timeout_ns, StatusRef sref) {
    constexpr int CPT = C::CPT, RT = C::RT, P = C::P, RB = C::RB, KB = C::KB, NT = C::NT;
    constexpr int TC = C::template steps<IO>(), VT = TC * RB;
    constexpr int KT = C::template pitch<IO>(TC * C::DKP), VTP = C::template pitch<IO>(VT);
    extern __shared__ __align__(128) unsigned char smem[];
    IO *ks = reinterpret_cast<IO *>(smem);   // [GB][NH][TC][KB] (pitch KT)
    IO *qs = ks + kGB * KT;
    IO *vs = qs + kGB * KT;                  // [GB][TC][RB] (pitch VTP)
    float *os = reinterpret_cast<float *>(vs + kGB * VTP);   // [2][TC][RB]: one barrier a chunk
    float *mu = os + 2 * VT;                     // [2][TC] readout factors scale A_t
    float *mw = mu + 2 * TC;                 // [2][TC] 1 / A_t (1 in a steep chunk)
    float *ma = mw + 2 * TC;                 // [2][TC] a_t of a steep chunk
    float *mm = ma + 2 * TC;                 // [2][2] factors before and after the chunk
    uint64_t *full = reinterpret_cast<uint64_t *>(mm + 2 * TC);

    const int tid = threadIdx.x, lane = tid & 31;
    // a call of one launch starts while the kernel before it drains
    if (!STATE_ONLY && a.n_seg == 1) grid_dependency_wait();
    if (!STATE_ONLY) launch_dependents();
    const int nseg = STATE_ONLY ? a.n_seg - 1 : a.n_seg;
    int x = blockIdx.x;
    const int rb = x % nrb;
    x /= nrb;
    const int seg = x % nseg;
    x /= nseg;
    const int h = x % a.H, hk = h / (a.H / a.Hk);
    static_assert(2 * VT >= kOrderRows, "os holds the rows' order before it holds outputs");
    const int b = dec::row_at(a, x / a.H, reinterpret_cast<int *>(os)), bh = b * a.H + h;
    if (tid == 0 && blockIdx.x == 0) status_begin(sref);
    const int p = tid % P, rg = tid / P;
    const int row0 = rb * RB, dk = a.dk, dv = a.dv;
    const int rbv = min(RB, dv - row0);
    const int64_t L = a.L;
    const int len = dec::row_len(a.lens, b, L);
    const int64_t s0 = int64_t(seg) * a.seg_len;
    const int64_t send = min(L, s0 + a.seg_len);             // the segment's end
    const int nrun = int(max(int64_t(0), min(int64_t(len), send) - s0));   // its steps inside the row
    const size_t HK = size_t(a.Hk) * dk, HV = size_t(a.H) * dv;
    const size_t t_base = size_t(b) * L + s0;
    const IO *kb = static_cast<const IO *>(a.k) + t_base * HK + size_t(hk) * dk;
    const IO *qb = static_cast<const IO *>(a.q) + t_base * HK + size_t(hk) * dk;
    const IO *vb = static_cast<const IO *>(a.v) + t_base * HV + size_t(h) * dv + row0;
    const IO *gb = a.g == nullptr ? nullptr : static_cast<const IO *>(a.g) + t_base * a.H + h;
    IO *ob = static_cast<IO *>(a.o) + t_base * HV + size_t(h) * dv + row0;

    if (tma) {
        if (tid == 0) {
            for (int i = 0; i < kGB; ++i) mbar_init(&full[i], 1);
            fence_mbar_init();
        }
    } else {   // what the element copies never write: columns past dk, rows past dv
        for (int e = tid; e < kGB * KT; e += NT) ks[e] = qs[e] = Io<IO>::from_f(0.0f);
        for (int e = tid; e < kGB * VTP; e += NT) vs[e] = Io<IO>::from_f(0.0f);
    }

    const int nchunks = (nrun + TC - 1) / TC;
    auto stage = [&](int c, int buf) {
        const int t0 = c * TC;
        IO *kd = ks + buf * KT, *qd = qs + buf * KT, *vd = vs + buf * VTP;
        if (tma) {
            if (tid == 0) {
                mbar_arrive_expect_tx(&full[buf], uint32_t(sizeof(IO)) * ((STATE_ONLY ? 1 : 2) * TC * C::DKP + VT));
                const int row = int(t_base) + t0;
#pragma unroll
                for (int hh = 0; hh < C::NH; ++hh) {
                    tma_load_3d(kd + hh * TC * KB, &tm_k, &full[buf], hh * KB, hk, row);
                    if (!STATE_ONLY) tma_load_3d(qd + hh * TC * KB, &tm_q, &full[buf], hh * KB, hk, row);
                }
                tma_load_3d(vd, &tm_v, &full[buf], row0, h, row);
            }
        } else {
            const int nt = min(TC, nrun - t0);
            for (int t = 0; t < nt; ++t) {
                const size_t sk = size_t(t0 + t) * HK, sv = size_t(t0 + t) * HV;
                for (int j = tid; j < dk; j += NT) {
                    const int at = (j / KB) * TC * KB + t * KB + j % KB;
                    kd[at] = kb[sk + j];
                    if (!STATE_ONLY) qd[at] = qb[sk + j];
                }
                for (int r = tid; r < rbv; r += NT) vd[t * RB + r] = vb[sv + r];
            }
        }
    };

    // decay factors of a chunk by warp 0, lane t its step t.  base: log2 decay
    // since the last rescale; tot: since the segment's start.
    const float lh = a.a_log == nullptr ? 0.0f : a.a_log[h];
    long long base = 0, tot = 0;
    bool bad = false;
    auto load_g = [&](int c) -> float {
        const int t = c * TC + lane;
        return gb != nullptr && lane < TC && t < nrun ? Io<IO>::to_f(gb[size_t(t) * a.H]) : 0.0f;
    };
    auto factors = [&](int c, float gv) {   // warp 0
        const int t = c * TC + lane;
        const long long own = lane < TC && t < nrun ? dec::to_fix(lh + gv, bad) : 0;
        long long cum = own;
#pragma unroll
        for (int m = 1; m < TC; m <<= 1) {
            const long long up = __shfl_up_sync(0xffffffffu, cum, m);
            if (lane >= m) cum += up;
        }
        const long long all = __shfl_sync(0xffffffffu, cum, TC - 1);
        const bool steep = all < dec::kSteep;
        float *u = mu + (c & 1) * TC, *w = mw + (c & 1) * TC, *m = mm + (c & 1) * 2;
        if (lane < TC) {
            u[lane] = a.scale * (steep ? 1.0f : dec::exp2_fix(base + cum));
            w[lane] = steep ? 1.0f : dec::exp2_fix(-(base + cum));
            ma[(c & 1) * TC + lane] = steep ? dec::exp2_fix(own) : 1.0f;
        }
        if (steep) {
            if (lane == 0) {
                m[0] = dec::exp2_fix(base);
                m[1] = -1.0f;   // marks a steep chunk
            }
            base = 0;
        } else {
            base += all;
            const bool re = base < dec::kRescale;
            if (lane == 0) {
                m[0] = 1.0f;
                m[1] = re ? dec::exp2_fix(base) : 1.0f;
            }
            if (re) base = 0;
        }
        tot = max(tot + all, -(1ll << 60));
    };

    // S[rr][2m + e] holds columns 4 (m P + p) + 2e + {0, 1} of row row0 + rg RT + rr
    float2 S[RT][CPT / 2];
    if (!STATE_ONLY && seg > 0) grid_dependency_wait();   // the first launch's states
    auto rows16 = [&](const float *x) { return (dk & 3) == 0 && (reinterpret_cast<uintptr_t>(x) & 15) == 0; };
    auto add_state = [&](const float *src, float f) {   // S += f src, a dv x dk state
        const bool v4 = rows16(src);
#pragma unroll
        for (int rr = 0; rr < RT; ++rr) {
            const int i = row0 + rg * RT + rr;
            if (i >= dv) continue;
#pragma unroll
            for (int m = 0; m < CPT / 4; ++m) {
                const float4 s = state_ld4(src + size_t(i) * dk, 4 * (m * P + p), dk, v4);
                S[rr][2 * m] = __ffma2_rn(make_float2(f, f), make_float2(s.x, s.y), S[rr][2 * m]);
                S[rr][2 * m + 1] = __ffma2_rn(make_float2(f, f), make_float2(s.z, s.w), S[rr][2 * m + 1]);
            }
        }
    };
#pragma unroll
    for (int rr = 0; rr < RT; ++rr)
#pragma unroll
        for (int m = 0; m < CPT / 2; ++m) S[rr][m] = make_float2(0.0f, 0.0f);
    if (seg == 0 && a.S0 != nullptr) add_state(a.S0 + size_t(bh) * dv * dk, 1.0f);
    if (!STATE_ONLY && seg > 0) {   // the decayed sum of the ranges before this one
        long long acc = 0;
        int s = seg - 1;
        for (; s >= 0; --s) {
            const float f = dec::exp2_fix(acc);
            if (f == 0.0f) break;
            const size_t at = size_t(bh) * (a.n_seg - 1) + s;
            add_state(a.seg_state + at * dv * dk, f);
            acc = max(acc + a.seg_tot[at], -(1ll << 60));
        }
        // nothing is left of the ranges before, unless it is not finite
        if (s >= 0 && dec::any_bad(a, bh, s, rb))
            for (; s >= 0; --s) add_state(a.seg_state + (size_t(bh) * (a.n_seg - 1) + s) * dv * dk, 0.0f);
    }
    if (STATE_ONLY) launch_dependents();

    if (tid < 32 && nchunks > 0) factors(0, load_g(0));
    __syncthreads();   // barriers initialised or buffers cleared, factors of chunk 0
    for (int c = 0; c < kGB - 1 && c < nchunks; ++c) stage(c, c);
    if (!tma) __syncthreads();
    for (int c = 0; c < nchunks; ++c) {
        const int buf = c % kGB;
        const bool more = c + 1 < nchunks;
        float gn = 0.0f;
        if (tid < 32 && more) gn = load_g(c + 1);
        if (c + kGB - 1 < nchunks) stage(c + kGB - 1, (c + kGB - 1) % kGB);
        const bool ok = !tma || mbar_wait_bounded(&full[buf], (c / kGB) & 1, timeout_ns);
        float *oc = os + (c & 1) * VT;
        const int nt = min(TC, nrun - c * TC);
        const float *u = mu + (c & 1) * TC, *w = mw + (c & 1) * TC, *wa = ma + (c & 1) * TC, *mf = mm + (c & 1) * 2;
        const float after = mf[1];
        const bool steep = after < 0.0f;
        const IO *vr = vs + buf * VTP + rg * RT;
        auto mul = [&](float f) {
            const float2 f2 = make_float2(f, f);
#pragma unroll
            for (int rr = 0; rr < RT; ++rr)
#pragma unroll
                for (int m = 0; m < CPT / 2; ++m) S[rr][m] = __fmul2_rn(S[rr][m], f2);
        };
        auto step = [&](int t) {
            const IO *kr = ks + buf * KT + t * KB + 4 * p, *qr = qs + buf * KT + t * KB + 4 * p;
            const float wt = w[t];
            float2 v2[RT], acc[RT][2];
#pragma unroll
            for (int rr = 0; rr < RT; ++rr) {
                const float vv = wt * Io<IO>::to_f(vr[t * RB + rr]);
                v2[rr] = make_float2(vv, vv);
                acc[rr][0] = acc[rr][1] = make_float2(0.0f, 0.0f);
            }
#pragma unroll
            for (int m = 0; m < CPT / 4; ++m) {
                const int off = ((4 * P * m) / KB) * TC * KB + (4 * P * m) % KB;
                const float4 k4 = dec_ld4<IO>(kr + off);
                const float2 k01 = make_float2(k4.x, k4.y), k23 = make_float2(k4.z, k4.w);
                float4 q4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (!STATE_ONLY) q4 = dec_ld4<IO>(qr + off);
                const float2 q01 = make_float2(q4.x, q4.y), q23 = make_float2(q4.z, q4.w);
#pragma unroll
                for (int rr = 0; rr < RT; ++rr) {
                    S[rr][2 * m] = __ffma2_rn(v2[rr], k01, S[rr][2 * m]);
                    S[rr][2 * m + 1] = __ffma2_rn(v2[rr], k23, S[rr][2 * m + 1]);
                    if (!STATE_ONLY) {
                        acc[rr][0] = __ffma2_rn(S[rr][2 * m], q01, acc[rr][0]);
                        acc[rr][1] = __ffma2_rn(S[rr][2 * m + 1], q23, acc[rr][1]);
                    }
                }
            }
            if (!STATE_ONLY) {
                float r[RT];
#pragma unroll
                for (int rr = 0; rr < RT; ++rr)
                    r[rr] = (acc[rr][0].x + acc[rr][0].y) + (acc[rr][1].x + acc[rr][1].y);
                row_sums<RT, P>(r, p);
                const float ut = u[t];
                if (p < RT) oc[t * RB + rg * RT + p] = ut * r[0];
            }
        };
        if (steep) {   // a loop of its own: the common one carries no trace of it
            mul(mf[0]);
#pragma unroll 1
            for (int t = 0; t < nt; ++t) {
                mul(wa[t]);
                step(t);
            }
        } else {
#pragma unroll 2
            for (int t = 0; t < nt; ++t) step(t);
            if (after != 1.0f) mul(after);
        }
        if (tid < 32 && more) factors(c + 1, gn);   // its buffer was last read in chunk c - 1
        // chunk c's buffer, its outputs, the next factors.  After a wait that ran
        // out every thread leaves here, once the copies in flight have landed.
        if (__syncthreads_or(!ok)) {
            if (tid == 0) {
                status_report(sref, LR_ERR_TIMEOUT);
                for (int c2 = c + 1; c2 < c + kGB && c2 < nchunks; ++c2)
                    mbar_wait_bounded(&full[c2 % kGB], (c2 / kGB) & 1, timeout_ns);
            }
            break;
        }
        if (!STATE_ONLY) {
            for (int e = tid; e < TC * RB; e += NT) {
                const int t = e / RB, r = e % RB;
                if (t < nt && r < rbv) ob[size_t(c * TC + t) * HV + r] = Io<IO>::from_f(oc[e]);
            }
        }
    }

    if (tid < 32 && bad) status_report(sref, LR_ERR_RANGE);
    // steps of the segment past the row's length
    if (!STATE_ONLY) {
        const int64_t nseg_steps = send - s0;
        for (int64_t e = int64_t(nrun) * RB + tid; e < nseg_steps * RB; e += NT) {
            const int64_t t = e / RB;
            const int r = int(e % RB);
            if (r < rbv) ob[size_t(t) * HV + r] = Io<IO>::from_f(0.0f);
        }
    }
    // the state as it stands is S / 2^base
    float *dst0 = nullptr;
    if (STATE_ONLY)
        dst0 = a.seg_state + (size_t(bh) * (a.n_seg - 1) + seg) * dv * dk;
    else if (seg == a.n_seg - 1 && a.S_final != nullptr)
        dst0 = a.S_final + size_t(bh) * dv * dk;
    if (STATE_ONLY && rb == 0 && tid == 0) a.seg_tot[size_t(bh) * (a.n_seg - 1) + seg] = tot;
    if (dst0 != nullptr) {
        if (tid == 0) mm[0] = dec::exp2_fix(base);   // warp 0 holds base
        __syncthreads();
        const float f = mm[0];
        const bool v4 = rows16(dst0);
        if (STATE_ONLY) {
            float2 zero = make_float2(0.0f, 0.0f);   // 0 times what is written
#pragma unroll
            for (int rr = 0; rr < RT; ++rr)
#pragma unroll
                for (int m = 0; m < CPT / 2; ++m)
                    zero = __ffma2_rn(__fmul2_rn(S[rr][m], make_float2(f, f)), make_float2(0.0f, 0.0f), zero);
            const int bad = __syncthreads_or(!(zero.x + zero.y == 0.0f));
            if (tid == 0) a.seg_bad[(size_t(bh) * (a.n_seg - 1) + seg) * a.seg_tiles + rb] = bad;
        }
#pragma unroll
        for (int rr = 0; rr < RT; ++rr) {
            const int i = row0 + rg * RT + rr;
            if (i >= dv) continue;
#pragma unroll
            for (int m = 0; m < CPT / 4; ++m) {
                const float2 s0 = S[rr][2 * m], s1 = S[rr][2 * m + 1];
                state_st4(dst0 + size_t(i) * dk, 4 * (m * P + p), dk, v4,
                          make_float4(f * s0.x, f * s0.y, f * s1.x, f * s1.y));
            }
        }
    }
}

template <typename IO, typename C>
int launch_general_cfg(const DecayArgs &a, StatusRef st, cudaStream_t stream) {
    constexpr int TC = C::template steps<IO>();
    const int nrb = (a.dv + C::RB - 1) / C::RB;
    const size_t es = sizeof(IO);
    auto al = [](const void *x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; };
    // tensor copies need 16-byte row starts and strides and 32-bit row coordinates
    bool tma = (a.dk * es) % 16 == 0 && (a.dv * es) % 16 == 0 && (C::RB * es) % 16 == 0 && al(a.q) && al(a.k) &&
               al(a.v) && a.B * a.L <= INT32_MAX;
    CUtensorMap mq{}, mk{}, mv{};
    if (tma) {
        const auto tt = Io<IO>::kTmType;
        const uint64_t rows = uint64_t(a.B) * a.L;
        tma = encode_map_3d(&mq, a.q, tt, es, a.dk, a.Hk, rows, C::KB, 1, TC) &&
              encode_map_3d(&mk, a.k, tt, es, a.dk, a.Hk, rows, C::KB, 1, TC) &&
              encode_map_3d(&mv, a.v, tt, es, a.dv, a.H, rows, C::RB, 1, TC);
    }
    const size_t smem = C::template smem_bytes<IO>();
    auto first = decay_general_kernel<IO, C, true>;
    auto main = decay_general_kernel<IO, C, false>;
    if (smem > 48 * 1024 &&
        (cudaFuncSetAttribute(first, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) != cudaSuccess ||
         cudaFuncSetAttribute(main, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) != cudaSuccess))
        return LR_ERR_CUDA;
    const int64_t per_seg = a.B * a.H * nrb;
    if (per_seg * a.n_seg > INT32_MAX) return LR_ERR_UNSUPPORTED;
    if (a.n_seg > 1) {
        const int rc = launch_kernel(first, false, dim3(unsigned(per_seg * (a.n_seg - 1))), C::NT, smem, stream, mq,
                                     mk, mv, a, nrb, tma, kDefaultTimeoutNs, st);
        if (rc != LR_OK) return rc;
    }
    // dependent launch: of the kernel before the call, or of the first launch, of
    // which segment 0 needs nothing
    return launch_kernel(main, true, dim3(unsigned(per_seg * a.n_seg)), C::NT, smem, stream, mq, mk, mv, a, nrb, tma,
                         kDefaultTimeoutNs, st);
}

template <typename IO, int DKP>
int launch_general_dk(const DecayArgs &a, bool narrow, StatusRef st, cudaStream_t stream) {
    return narrow ? launch_general_cfg<IO, DecCfg<DKP, true>>(a, st, stream)
                  : launch_general_cfg<IO, DecCfg<DKP, false>>(a, st, stream);
}

}  // namespace

template <typename IO>
int decay_general_launch(const DecayArgs &a, const DecayPlan &p, StatusRef st, cudaStream_t stream) {
    if (a.dk <= 32) return launch_general_dk<IO, 32>(a, p.narrow, st, stream);
    if (a.dk <= 64) return launch_general_dk<IO, 64>(a, p.narrow, st, stream);
    if (a.dk <= 128) return launch_general_dk<IO, 128>(a, p.narrow, st, stream);
    if (a.dk <= 256) {
        if constexpr (sizeof(IO) == 4) return launch_general_dk<IO, 256>(a, p.narrow, st, stream);
        return launch_general_cfg<IO, DecCfg<256, false>>(a, st, stream);
    }
    return launch_general_cfg<IO, DecCfg<512, false>>(a, st, stream);
}

}  // namespace lr
