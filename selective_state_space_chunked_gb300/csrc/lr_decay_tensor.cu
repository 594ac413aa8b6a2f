// lr_decay_tensor.cu -- decayed linear attention, bf16 I/O, on the sm_103a
// tensor cores (tcgen05, accumulators in TMEM, operands by TMA).
//
//   S_t = a_t S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t,   a_t = exp(l_t)
//
// One decay per head and step, so a chunk of C = 128 steps is three matrix
// products around a 128 x 128 table of scalars.  With L_t the log2 decay from
// the chunk's start through step t and S the state before the chunk:
//
//   O  = scale ( [(Q K^T) . D] V + diag(2^L) Q S^T ),   D_ts = 2^(L_t - L_s), s <= t
//   S' = 2^L_C S + sum_s 2^(L_C - L_s) v_s k_s^T
//
// Every D_ts <= 1 and is formed from the difference itself: no reference
// point, no range limit, resets included.
//
// Precision.  D . (Q K^T) and the copy of S that Q S^T reads are rounded to
// bf16 once (matrix operands; o is rounded to bf16 anyway).  The carried state
// is not: w_s v_s (w_s the decay weight, fp32) is split into three bf16 terms
// (24 bits), which sit side by side as one N = 192 operand, so that K is read
// once for the three; their sum is added to the fp32 state.  The state is kept
// as S^ = S / (decay since the last rescale): w_s = 2^(-L_s) and no
// multiplication of S while that decay is above 2^-16; the chunk that takes
// it below uses w_s = 2^(L_C - L_s) and multiplies S once.
//
// A thread block owns 64 value rows of one (batch row, head, time segment),
// 128 key columns.  Roles, connected by mbarriers:
//   TMA warp   Q, K, V two chunks deep, released separately (K first: it is
//              not needed once dS is done)
//   scan warp  log decays of the next chunk -> L (fp32), w, the chunk's factors
//   weight (4) w_s v_s in three terms; rows past the end of the row zeroed
//   MMA warp   dS = K^T [W1 W2 W3]  M=128 N=192   (independent of the state)
//              P  = Q K^T           M=128 N=128   one chunk ahead
//              OI = PD V            M=128 N=64    PD from TMEM
//   front (4)  PD = bf16(D . P), in place in P's first 64 columns
//   OX warp    OX = Q S^T           M=128 N=64    into P's other 64 columns
//   back (4)   S = m S + dS (fp32, thread j holds key column j of the 64
//              rows), its bf16 copy, then the outputs
// TMEM: P 2 x 128 columns (PD and OX inside), OI 64, dS 192: all 512.
#include <cudaTypedefs.h>

#include <mutex>

#include "lr_decay.cuh"

namespace lr {

namespace dt {
constexpr int C = kDecayChunk;
constexpr int RB = kDecayRows;
constexpr int FRONT = 4, WEIGHT = 8, TMA_WARP = 12, MMA_WARP = 13, OX_WARP = 14, SCAN_WARP = 15;
constexpr int THREADS = 16 * 32;

constexpr uint32_t HALF = C * 128;              // 64 columns of Q or K: 128 rows of 128 bytes
constexpr uint32_t Q_BYTES = 2 * HALF, V_BYTES = C * RB * 2;
constexpr uint32_t OFF_Q = 0, OFF_K = 2 * Q_BYTES, OFF_V = 4 * Q_BYTES;
constexpr uint32_t OFF_W = OFF_V + 2 * V_BYTES;     // three terms [128 s][64 i]
constexpr uint32_t OFF_SB = OFF_W + 3 * V_BYTES;    // bf16 state [128 j][64 i]
constexpr uint32_t OFF_L = OFF_SB + 128 * RB * 2;   // 2 x L [128] fp32
constexpr uint32_t OFF_WT = OFF_L + 2 * C * 4;      // 2 x w [128] fp32
constexpr uint32_t OFF_F = OFF_WT + 2 * C * 4;      // 2 x (m, base as log2)
constexpr uint32_t OFF_BAR = OFF_F + 2 * 8;
// barriers
enum {
    FULL_Q = 0, EMPTY_Q = 2, FULL_K = 4, EMPTY_K = 6, FULL_V = 8, EMPTY_V = 10, P_READY = 12, F_DONE = 14,
    K_DONE = 16, M_READY = 18, OI_DONE = 20, OX_DONE, SB_READY, DS_DONE, DS_FREE, W_READY, MMA_END, NBAR
};
constexpr uint32_t OFF_TMEM = OFF_BAR + NBAR * 8;
constexpr uint32_t OFF_END = OFF_TMEM + 4;
constexpr uint32_t OFF_FLAG = OFF_TMEM + 8;
constexpr uint32_t SMEM = OFF_FLAG + 8;
static_assert(SMEM <= 227 * 1024, "one block per SM");

constexpr uint32_t T_P = 0, T_OI = 256, T_DS = 320;
constexpr uint32_t IDESC_P = umma_idesc_bf16(128, 128, 0, 0);
constexpr uint32_t IDESC_O = umma_idesc_bf16(128, 64, 0, 1);
constexpr uint32_t IDESC_DS = umma_idesc_bf16(128, 192, 1, 1);

__device__ __forceinline__ void arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&p);
}
__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// Bounded wait; the first to run out makes every role leave its loop.
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, volatile int *abort_flag,
                                              uint64_t timeout_ns, StatusRef sref) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (*abort_flag != 0) return false;
        if (globaltimer_ns() - t0 > timeout_ns) {
            *abort_flag = 1;
            status_report(sref, LR_ERR_TIMEOUT);
            return false;
        }
    }
    return true;
}
}  // namespace dt

template <bool STATE_ONLY>
__global__ void __launch_bounds__(dt::THREADS, 1)
    decay_tensor_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const DecayArgs a, int n_vt, uint64_t timeout_ns,
                        StatusRef sref) {
    using namespace dt;
    using bf = __nv_bfloat16;
    extern __shared__ __align__(1024) unsigned char sm[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (STATE_ONLY) launch_dependents();
    if (tid == 0 && blockIdx.x == 0) status_begin(sref);
    if ((smem_u32(sm) & 1023u) != 0) {   // swizzled tiles need a 1024-byte aligned base
        if (tid == 0) status_report(sref, LR_ERR_CUDA);
        return;
    }
    const int nseg = STATE_ONLY ? a.n_seg - 1 : a.n_seg;
    int x = blockIdx.x;
    const int vt = x % n_vt;
    x /= n_vt;
    const int seg = x % nseg, bh = x / nseg;
    const int b = bh / a.H, h = bh - b * a.H, hk = h / (a.H / a.Hk);
    const int len = dec::row_len(a.lens, b, a.L);
    const int s0 = int(int64_t(seg) * a.seg_len);
    const int send = int(min(a.L, int64_t(s0) + a.seg_len));
    const int nrun = max(0, min(len, send) - s0);
    const int n_chunks = (nrun + C - 1) / C;
    const int dk = a.dk, dv = a.dv;
    const int nkk = (dk + 15) / 16;          // 16-wide steps over the key columns
    const bool two = dk > 64;                // two 64-column halves of Q and K

    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + OFF_BAR);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + OFF_TMEM);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + OFF_FLAG);
    float *sL = reinterpret_cast<float *>(sm + OFF_L), *sW = reinterpret_cast<float *>(sm + OFF_WT),
          *sF = reinterpret_cast<float *>(sm + OFF_F);
    if (tid == 0) {
        for (int i = 0; i < NBAR; ++i) {
            const bool four = (i >= F_DONE && i < M_READY) || i == SB_READY || i == DS_FREE || i == W_READY;
            mbar_init(&bar[i], four ? 4 : i == MMA_END ? 2 : 1);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto hw = [&](int i, int phase) -> bool {
        return wait_or_abort(&bar[i], uint32_t(phase) & 1u, abort_flag, timeout_ns, sref);
    };

    if (warp == TMA_WARP) {   // ------------------------------------------- TMA
        if (lane == 0) {
            int nk = 0, nq = 0, nv = 0;
            for (int c = 0; c < n_chunks; ++c) {
                const int st = c & 1, t = s0 + c * C;
                if (c >= 2 && !hw(EMPTY_K + st, (c - 2) >> 1)) break;
                mbar_arrive_expect_tx(&bar[FULL_K + st], two ? Q_BYTES : HALF);
                tma_load_4d(sm + OFF_K + st * Q_BYTES, &tm_k, &bar[FULL_K + st], 0, hk, t, b);
                if (two) tma_load_4d(sm + OFF_K + st * Q_BYTES + HALF, &tm_k, &bar[FULL_K + st], 64, hk, t, b);
                ++nk;
                if (!STATE_ONLY) {
                    if (c >= 2 && !hw(EMPTY_Q + st, (c - 2) >> 1)) break;
                    mbar_arrive_expect_tx(&bar[FULL_Q + st], two ? Q_BYTES : HALF);
                    tma_load_4d(sm + OFF_Q + st * Q_BYTES, &tm_q, &bar[FULL_Q + st], 0, hk, t, b);
                    if (two) tma_load_4d(sm + OFF_Q + st * Q_BYTES + HALF, &tm_q, &bar[FULL_Q + st], 64, hk, t, b);
                    ++nq;
                }
                if (c >= 2 && !hw(EMPTY_V + st, (c - 2) >> 1)) break;
                mbar_arrive_expect_tx(&bar[FULL_V + st], V_BYTES);
                tma_load_4d(sm + OFF_V + st * V_BYTES, &tm_v, &bar[FULL_V + st], vt * RB, h, t, b);
                ++nv;
            }
            // copies still in flight land before the block exits
            for (int c = max(nk - 2, 0); c < nk; ++c)
                mbar_wait_bounded(&bar[FULL_K + (c & 1)], (c >> 1) & 1, timeout_ns);
            for (int c = max(nq - 2, 0); c < nq; ++c)
                mbar_wait_bounded(&bar[FULL_Q + (c & 1)], (c >> 1) & 1, timeout_ns);
            for (int c = max(nv - 2, 0); c < nv; ++c)
                mbar_wait_bounded(&bar[FULL_V + (c & 1)], (c >> 1) & 1, timeout_ns);
        }
    } else if (warp == MMA_WARP) {   // ------------------------------------ MMA
        if (lane == 0) {
            auto issue_p = [&](int c) {
                const uint32_t sQ = smem_u32(sm + OFF_Q + (c & 1) * Q_BYTES),
                               sK = smem_u32(sm + OFF_K + (c & 1) * Q_BYTES);
                for (int kk = 0; kk < nkk; ++kk) {
                    const uint32_t off = (kk >> 2) * HALF + (kk & 3) * 32;
                    umma_bf16(tmem + T_P + (c & 1) * 128, umma_smem_desc(sQ + off, 16, 1024),
                              umma_smem_desc(sK + off, 16, 1024), IDESC_P, kk > 0);
                }
                umma_commit(&bar[P_READY + (c & 1)]);
            };
            bool ok = n_chunks > 0;
            if (ok) ok = hw(FULL_K, 0);
            if (ok && !STATE_ONLY) {
                ok = hw(FULL_Q, 0);
                if (ok) {
                    tc_fence_after();
                    issue_p(0);
                }
            }
            for (int c = 0; ok && c < n_chunks; ++c) {
                const int st = c & 1;
                const uint32_t sK = smem_u32(sm + OFF_K + st * Q_BYTES), sV = smem_u32(sm + OFF_V + st * V_BYTES),
                               sWt = smem_u32(sm + OFF_W);
                // dS once the weighted values are there and the back has read the last one
                if (STATE_ONLY && !hw(FULL_K + st, c >> 1)) break;
                if (!hw(W_READY, c) || (c >= 1 && !hw(DS_FREE, c - 1))) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < C / 16; ++kk)
                    umma_bf16(tmem + T_DS, umma_smem_desc(sK + kk * 2048, HALF, 1024),
                              umma_smem_desc(sWt + kk * 2048, V_BYTES, 1024), IDESC_DS, kk > 0);
                umma_commit(&bar[DS_DONE]);
                umma_commit(&bar[EMPTY_K + st]);   // P_c, issued before, is covered too
                if (STATE_ONLY) {
                    umma_commit(&bar[EMPTY_V + st]);
                    continue;
                }
                // P of the next chunk; its buffer (and OI's) held chunk c - 1's
                if (c >= 1 && !hw(K_DONE + ((c - 1) & 1), (c - 1) >> 1)) break;
                if (c + 1 < n_chunks) {
                    const int sn = (c + 1) & 1;
                    if (!hw(FULL_K + sn, (c + 1) >> 1) || !hw(FULL_Q + sn, (c + 1) >> 1)) break;
                    tc_fence_after();
                    issue_p(c + 1);
                }
                if (!hw(F_DONE + st, c >> 1)) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < C / 16; ++kk)
                    umma_bf16_ts(tmem + T_OI, tmem + T_P + st * 128 + kk * 8,
                                 umma_smem_desc(sV + kk * 2048, HALF, 1024), IDESC_O, kk > 0);
                umma_commit(&bar[OI_DONE]);
                umma_commit(&bar[EMPTY_V + st]);
            }
            // nothing of this block's may still run on the tensor cores when its TMEM is released
            umma_commit(&bar[MMA_END]);
            mbar_wait_bounded(&bar[MMA_END], 0, timeout_ns);
        }
    } else if (warp == OX_WARP) {   // -------------------------------------- OX
        if (lane == 0) {
            for (int c = 0; !STATE_ONLY && c < n_chunks; ++c) {
                const int st = c & 1;
                // the state before chunk c; P_c read (its columns 64.. are free)
                if (!hw(SB_READY, c) || !hw(F_DONE + st, c >> 1)) break;
                tc_fence_after();
                const uint32_t sQ = smem_u32(sm + OFF_Q + st * Q_BYTES), sS = smem_u32(sm + OFF_SB);
                for (int kk = 0; kk < nkk; ++kk)
                    umma_bf16(tmem + T_P + st * 128 + 64,
                              umma_smem_desc(sQ + (kk >> 2) * HALF + (kk & 3) * 32, 16, 1024),
                              umma_smem_desc(sS + kk * 2048, HALF, 1024), IDESC_O, kk > 0);
                umma_commit(&bar[OX_DONE]);
                umma_commit(&bar[EMPTY_Q + st]);
            }
            umma_commit(&bar[MMA_END]);
            mbar_wait_bounded(&bar[MMA_END], 0, timeout_ns);
        }
    } else if (warp == SCAN_WARP) {   // ---------------------------------- scan
        // lane i: steps 4 i .. 4 i + 3 of the chunk
        const float lh = a.a_log == nullptr ? 0.0f : a.a_log[h];
        const bf *g = a.g == nullptr ? nullptr : static_cast<const bf *>(a.g) + (size_t(b) * a.L + s0) * a.H + h;
        long long base = 0, tot = 0;
        bool bad = false;
        float gn[4];
        auto load = [&](int c) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = c * C + 4 * lane + i;
                gn[i] = g != nullptr && t < nrun ? __bfloat162float(g[size_t(t) * a.H]) : 0.0f;
            }
        };
        load(0);
        for (int c = 0; c < n_chunks; ++c) {
            long long cum[4], run = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (c * C + 4 * lane + i < nrun) run += dec::to_fix(lh + gn[i], bad);
                cum[i] = run;
            }
            if (c + 1 < n_chunks) load(c + 1);
            long long incl = run;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const long long up = __shfl_up_sync(0xffffffffu, incl, m);
                if (lane >= m) incl += up;
            }
            const long long all = __shfl_sync(0xffffffffu, incl, 31), before = incl - run;
            const long long end = base + all;            // since the last rescale
            const bool re = end < dec::kRescale;
            bool ok = c < 2 || hw(K_DONE + (c & 1), (c - 2) >> 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            float lv[4], wv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const long long l = before + cum[i];
                lv[i] = float(l) * dec::kFixInv;
                wv[i] = dec::exp2_fix(re ? all - l : -(base + l));
            }
            float *pl = sL + (c & 1) * C + 4 * lane, *pw = sW + (c & 1) * C + 4 * lane;
            *reinterpret_cast<float4 *>(pl) = make_float4(lv[0], lv[1], lv[2], lv[3]);
            *reinterpret_cast<float4 *>(pw) = make_float4(wv[0], wv[1], wv[2], wv[3]);
            if (lane == 0) {
                sF[2 * (c & 1)] = re ? dec::exp2_fix(end) : 1.0f;
                sF[2 * (c & 1) + 1] = float(base) * dec::kFixInv;
            }
            __syncwarp();
            if (lane == 0) arrive(&bar[M_READY + (c & 1)]);
            base = re ? 0 : end;
            tot = max(tot + all, -(1ll << 60));
        }
        if (bad) status_report(sref, LR_ERR_RANGE);
        if (STATE_ONLY && vt == 0 && lane == 0) a.seg_tot[size_t(bh) * (a.n_seg - 1) + seg] = tot;
        // the decay that S^ still lacks, for the state that the block leaves
        if (lane == 0) *reinterpret_cast<float *>(sm + OFF_END) = dec::exp2_fix(base);
    } else if (warp >= WEIGHT) {   // ----------------------------------- weight
        const int s = tid - 32 * WEIGHT;   // this thread's step of the chunk
        for (int c = 0; c < n_chunks; ++c) {
            const int st = c & 1;
            unsigned char *V = sm + OFF_V + st * V_BYTES;
            const bool in = c * C + s < nrun;
            bool ok = hw(M_READY + st, c >> 1) && hw(FULL_V + st, c >> 1);
            if (ok && c * C + C > nrun) ok = hw(FULL_K + st, c >> 1);
            if (ok && c >= 1) ok = hw(DS_DONE, c - 1);   // the three terms' buffer is free
            if (!__all_sync(0xffffffffu, ok)) break;
            const float w = sW[st * C + s];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t at = sw128_offset(s, 8 * k);
                const uint4 u = *reinterpret_cast<const uint4 *>(V + at);
                const uint32_t uv[4] = {u.x, u.y, u.z, u.w};
                uint32_t w1[4], w2[4], w3[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float y0 = in ? w * lo_f(uv[e]) : 0.0f, y1 = in ? w * hi_f(uv[e]) : 0.0f;
                    w1[e] = pack(y0, y1);
                    y0 -= lo_f(w1[e]), y1 -= hi_f(w1[e]);
                    w2[e] = pack(y0, y1);
                    y0 -= lo_f(w2[e]), y1 -= hi_f(w2[e]);
                    w3[e] = pack(y0, y1);
                }
                *reinterpret_cast<uint4 *>(sm + OFF_W + at) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
                *reinterpret_cast<uint4 *>(sm + OFF_W + V_BYTES + at) = make_uint4(w2[0], w2[1], w2[2], w2[3]);
                *reinterpret_cast<uint4 *>(sm + OFF_W + 2 * V_BYTES + at) = make_uint4(w3[0], w3[1], w3[2], w3[3]);
            }
            if (!in) {   // past the row's end: whatever stands there must not reach a product
                const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    *reinterpret_cast<uint4 *>(V + s * 128 + 16 * k) = z;
                    *reinterpret_cast<uint4 *>(sm + OFF_K + st * Q_BYTES + s * 128 + 16 * k) = z;
                    if (two) *reinterpret_cast<uint4 *>(sm + OFF_K + st * Q_BYTES + HALF + s * 128 + 16 * k) = z;
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) arrive(&bar[W_READY]);
        }
    } else if (warp >= FRONT) {   // ------------------------------------- front
        const int fw = warp - FRONT, t = 32 * fw + lane;   // this thread's row
        const uint32_t lanes = uint32_t(fw * 32) << 16;
        for (int c = 0; !STATE_ONLY && c < n_chunks; ++c) {
            const int st = c & 1;
            const uint32_t P = tmem + T_P + st * 128 + lanes;
            const bool ok = hw(M_READY + st, c >> 1) && hw(P_READY + st, c >> 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const float *l = sL + st * C;
            const float lt = l[t];
            const int nv = nrun - c * C;   // valid steps of the chunk
#pragma unroll 1
            for (int kb = 0; kb < 4; ++kb) {
                uint32_t r[16];
                if (kb <= fw) {
                    float p[32];
                    tmem_ld32_nowait(P + 32 * kb, p);
                    tmem_ld_wait_tied(p);
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const int sx = 32 * kb + e;
                        const float4 ls = *reinterpret_cast<const float4 *>(l + sx);
                        const float y0 = sx <= t && sx < nv ? p[e] * ex2_approx(lt - ls.x) : 0.0f;
                        const float y1 = sx + 1 <= t && sx + 1 < nv ? p[e + 1] * ex2_approx(lt - ls.y) : 0.0f;
                        const float y2 = sx + 2 <= t && sx + 2 < nv ? p[e + 2] * ex2_approx(lt - ls.z) : 0.0f;
                        const float y3 = sx + 3 <= t && sx + 3 < nv ? p[e + 3] * ex2_approx(lt - ls.w) : 0.0f;
                        r[e / 2] = pack(y0, y1);
                        r[e / 2 + 1] = pack(y2, y3);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) r[e] = 0;
                }
                // columns 16 kb .. hold P columns that this thread has read
                tmem_st16_nowait(P + 16 * kb, r);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive(&bar[F_DONE + st]);
        }
    } else {   // ---------------------------------------------------------- back
        const int j = tid;   // key column
        const uint32_t lanes = uint32_t(warp * 32) << 16;
        const int i0 = vt * RB;
        float S[RB];
        const float *s_in = seg > 0 ? nullptr : a.S0;
#pragma unroll
        for (int r = 0; r < RB; ++r)
            S[r] = s_in != nullptr && j < dk && i0 + r < dv ? s_in[(size_t(bh) * dv + i0 + r) * dk + j] : 0.0f;
        if (!STATE_ONLY && seg > 0) {   // the decayed sum of the ranges before this one
            grid_dependency_wait();
            long long acc = 0;
            for (int s = seg - 1; s >= 0; --s) {
                const float f = dec::exp2_fix(acc);
                if (f == 0.0f) break;
                const size_t at = size_t(bh) * (a.n_seg - 1) + s;
                const float *src = a.seg_state + (at * dv + i0) * dk + j;
#pragma unroll
                for (int r = 0; r < RB; ++r)
                    if (j < dk && i0 + r < dv) S[r] = fmaf(f, src[size_t(r) * dk], S[r]);
                acc = max(acc + a.seg_tot[at], -(1ll << 60));
            }
        }
        auto publish = [&]() {   // bf16 copy: row j, 64 value rows in 8 swizzled groups
#pragma unroll
            for (int k = 0; k < 8; ++k)
                *reinterpret_cast<uint4 *>(sm + OFF_SB + sw128_offset(j, 8 * k)) =
                    make_uint4(pack(S[8 * k], S[8 * k + 1]), pack(S[8 * k + 2], S[8 * k + 3]),
                               pack(S[8 * k + 4], S[8 * k + 5]), pack(S[8 * k + 6], S[8 * k + 7]));
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) arrive(&bar[SB_READY]);
        };
        if (!STATE_ONLY) publish();
        const size_t HV = size_t(a.H) * dv;
        bf *ob = static_cast<bf *>(a.o) + (size_t(b) * a.L + s0) * HV + size_t(h) * dv + i0;
        for (int c = 0; c < n_chunks; ++c) {
            const int st = c & 1;
            bool ok = hw(M_READY + st, c >> 1) && hw(DS_DONE, c);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const float m = sF[2 * st], base = sF[2 * st + 1];
#pragma unroll
            for (int q = 0; q < RB; q += 16) {   // small terms first
                float d1[16], d2[16];
                tmem_ld16_nowait(tmem + T_DS + lanes + 128 + q, d1);
                tmem_ld16_nowait(tmem + T_DS + lanes + 64 + q, d2);
                tmem_ld_wait_tied(d1, d2);
#pragma unroll
                for (int r = 0; r < 16; ++r) d2[r] += d1[r];
                tmem_ld16_nowait(tmem + T_DS + lanes + q, d1);
                tmem_ld_wait_tied(d1);
#pragma unroll
                for (int r = 0; r < 16; ++r) S[q + r] = fmaf(m, S[q + r], d1[r] + d2[r]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive(&bar[DS_FREE]);
            if (!STATE_ONLY) {
                ok = hw(OX_DONE, c);   // the bf16 copy has been read
                if (!__all_sync(0xffffffffu, ok)) break;
                if (c + 1 < n_chunks) publish();
                ok = hw(OI_DONE, c);
                if (!__all_sync(0xffffffffu, ok)) break;
                tc_fence_after();
                const int t = c * C + tid;   // this thread's row of the outputs
                const float u = exp2f(base + sL[st * C + tid]) * a.scale;
                const bool valid = t < nrun, store = s0 + t < send;
                bf *dst = ob + size_t(t) * HV;
#pragma unroll
                for (int q = 0; q < RB; q += 16) {
                    float oi[16], ox[16];
                    tmem_ld16_nowait(tmem + T_OI + lanes + q, oi);
                    tmem_ld16_nowait(tmem + T_P + st * 128 + 64 + lanes + q, ox);
                    tmem_ld_wait_tied(oi, ox);
                    uint32_t w[8];
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        w[r] = valid ? pack(fmaf(u, ox[2 * r], a.scale * oi[2 * r]),
                                            fmaf(u, ox[2 * r + 1], a.scale * oi[2 * r + 1]))
                                     : 0u;
                    if (store && i0 + q < dv)
                        *reinterpret_cast<uint4 *>(dst + q) = make_uint4(w[0], w[1], w[2], w[3]);
                    if (store && i0 + q + 8 < dv)
                        *reinterpret_cast<uint4 *>(dst + q + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                }
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) arrive(&bar[K_DONE + st]);
        }
        // the state after the segment, in the launch's last lines below
        asm volatile("bar.sync 1, 160;" ::: "memory");   // the scan warp's last factor
        float *out = STATE_ONLY ? a.seg_state + (size_t(bh) * (a.n_seg - 1) + seg) * dv * dk
                     : seg == a.n_seg - 1 && a.S_final != nullptr ? a.S_final + size_t(bh) * dv * dk
                                                                  : nullptr;
        if (out != nullptr && j < dk) {
            const float f = *reinterpret_cast<const float *>(sm + OFF_END);
#pragma unroll
            for (int r = 0; r < RB; ++r)
                if (i0 + r < dv) out[size_t(i0 + r) * dk + j] = f * S[r];
        }
    }
    if (warp == SCAN_WARP) asm volatile("bar.sync 1, 160;" ::: "memory");

    if (!STATE_ONLY) {   // whole chunks past the row's end
        const int g8 = min(RB, dv - vt * RB) / 8;
        const int64_t first = s0 + int64_t(n_chunks) * C;
        bf *ob = static_cast<bf *>(a.o) + size_t(h) * dv + vt * RB;
        for (int64_t e = tid; e < (send - first) * g8; e += THREADS)
            *reinterpret_cast<uint4 *>(ob + (size_t(b) * a.L + first + e / g8) * size_t(a.H) * dv + (e % g8) * 8) =
                make_uint4(0, 0, 0, 0);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
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
bool dt_map(CUtensorMap *tm, const void *base, uint64_t d, uint64_t heads, uint64_t L, uint64_t B) {
    auto enc = dt_encoder();
    if (enc == nullptr) return false;
    const cuuint64_t dims[4] = {d, heads, L, B};
    const cuuint64_t strides[3] = {d * 2, d * heads * 2, d * heads * L * 2};
    const cuuint32_t box[4] = {64, 1, uint32_t(dt::C), 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool dt_setup_once() {
    static std::once_flag once;
    static bool ok = false;
    std::call_once(once, [] {
        ok = cudaFuncSetAttribute(decay_tensor_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  int(dt::SMEM)) == cudaSuccess &&
             cudaFuncSetAttribute(decay_tensor_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  int(dt::SMEM)) == cudaSuccess;
    });
    return ok;
}

}  // namespace

int decay_tensor_launch(const DecayArgs &a, StatusRef st, cudaStream_t stream) {
    CUtensorMap mq, mk, mv;
    if (!dt_map(&mq, a.q, a.dk, a.Hk, a.L, a.B) || !dt_map(&mk, a.k, a.dk, a.Hk, a.L, a.B) ||
        !dt_map(&mv, a.v, a.dv, a.H, a.L, a.B) || !dt_setup_once())
        return LR_ERR_CUDA;
    const int n_vt = (a.dv + dt::RB - 1) / dt::RB;
    const int64_t per_seg = a.B * a.H * n_vt;
    if (per_seg * a.n_seg > INT32_MAX) return LR_ERR_UNSUPPORTED;
    if (a.n_seg > 1) {
        decay_tensor_kernel<true><<<unsigned(per_seg * (a.n_seg - 1)), dt::THREADS, dt::SMEM, stream>>>(
            mq, mk, mv, a, n_vt, kDefaultTimeoutNs, st);
        if (cudaGetLastError() != cudaSuccess) return LR_ERR_CUDA;
    }
    // dependent launch: segment 0 needs nothing of the first launch
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(per_seg * a.n_seg));
    cfg.blockDim = dim3(dt::THREADS);
    cfg.dynamicSmemBytes = dt::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.n_seg > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, decay_tensor_kernel<false>, mq, mk, mv, a, n_vt,
                                             uint64_t(kDefaultTimeoutNs), st);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? LR_OK : LR_ERR_CUDA;
}

}  // namespace lr
