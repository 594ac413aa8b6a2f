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
// A chunk that decays by less than 2^-40 in all takes D as a product: the
// columns of Q K^T are multiplied by the same w_s that weigh the state's
// update and the rows of the result by 2^L_t / (their common factor), one
// multiplication an element.  A steeper chunk (resets included) forms each
// D_ts <= 1 from its difference, so there is no range limit.
//
// Precision.  D . (Q K^T) and the copy of S that Q S^T reads are rounded to
// bf16 once (matrix operands; o is rounded to bf16 anyway).  The carried state
// is not: w_s v_s (w_s the decay weight, fp32) is split into three bf16 terms
// (24 bits), which sit side by side as one N = 192 operand, so that K is read
// once for the three, and accumulate in fp32.  The state is kept as S^ = S /
// (decay since the last rescale): w_s = 2^(-L_s) and no multiplication of S
// while that decay is above 2^-48; the chunk that takes it below uses
// w_s = 2^(L_C - L_s) and multiplies S once.  Scores and state carry the same
// factor, so Q S^T and PD V meet in one accumulator and o_t takes 1 / w_t.
//
// A thread block owns 64 value rows of one (batch row, head, time segment),
// 128 key columns.  Roles, connected by mbarriers:
//   TMA warps    Q, K, V two chunks deep, one warp each: they are released at
//                different points of a chunk
//   scan warp    log decays -> w (and L where the chunk is steep) and the
//                chunk's factors, up to four chunks ahead
//   weight (4)   w_s v_s in three terms, 32 steps a warp, each quarter handed
//                over by itself; rows past the end of the row zeroed
//   dS warp      dS = K^T [W1 W2 W3]   M=128 N=192
//   O warp       O  = Q S^T            M=128 N=64
//                O += PD V             M=128 N=64, PD from TMEM
//   P warp       P  = Q K^T            M=128 N=128, one chunk ahead
//                (a whole warp runs each issue loop, one elected lane issues:
//                in code that only one lane reaches, the operands' moves to
//                uniform registers made the issue the bottleneck)
//   front (8)    PD = bf16(D . P) in place, 64 columns a warp
//   state (8)    S = m S + dS (fp32, in registers: a thread holds 32 value rows of
//                one key column), its bf16 copy for the next Q S^T.  dS is
//                released as soon as it is read, so the next chunk's dS waits
//                for nothing else of the state's
//   output (4)   o = scale / w O (a steep chunk's Q S^T is scaled by rows before
//                PD V is added)
// More than 128 keys (PARTS): the state's key columns are independent of one
// another and o_t = sum over j of S_t[:, j] q_t[j], so each 128 of them run as a
// recurrence of their own, in blocks of their own, and a last launch adds their
// fp32 outputs and rounds the sum.  The scores' products with V are repeated by
// every part; at B2 L1500 H8 dk256 dv128 48 us against 169 on the CUDA cores, B4
// L4096 H16 dk256 dv128 262 against 1528, B4 L1024 H8 dk512 dv128 76 against 387,
// B1 L64 H4 dk192 dv64 12 against 56 (the last three of the CUDA cores as measured
// when the parts came in).
// TMEM: P 2 x 128 columns (PD inside), O 64, dS 3 x 64: all 512.
// Infinities and NaN.  The products take a masked score as 0, and 0 v_s is no 0
// where v_s is not finite; the terms of an infinity, and finite values past about
// 2^80 under a weight of 2^48, leave nothing finite either.  Whatever goes wrong so
// is not finite in an output of the block or in the state that it leaves, so the
// output and state warps look for that (one packed operation for four outputs), and
// a block that finds it goes through its steps again as the recurrence itself
// (redo_block): every row's earlier steps, and its infinities, are then what the
// definition says.
// Loops over columns stay rolled and waits share one slow path: with every
// role's code unrolled the warps waited for instruction fetches more than for
// anything else (95 us against 90 at B4 L4096 H16 d128 for the last part of it).
//
// Measured (d128, H16): B4 L4096 86.5 us, 273 MB and 17 GFLOP, 47 % of the copy
// bandwidth and 10 % of the tensor peak, 110.5 us with steep chunks alone; B1 L32768
// 235-243 us in four segments; B1 L77 9.8.  d64: B8 L1017 H32, ragged, 38-47.  No pipe
// is near its limit (over all SMs tensor 28 % busy, issue 36 %, DRAM 36 %): a chunk
// takes about 2.7 us, the chain of its hand-overs, with one block per SM, which its
// operands (227 KB) and TMEM fill.  At 64 registers a thread 100 bytes spill (120 with
// parts); a variant that spilled 40 took 88 us.
// 128-step chunks rather than 64 halve the hand-overs; 64 value rows rather than
// 128 make twice the blocks.  Measured against 91 us and not taken: P and dS issued
// by one warp 98, weights by eight warps or by half chunks 98-100, one warp polling
// for all products 192, two state terms instead of three 89 (with the state's error
// a hundred times larger), sleeping waits 91.
#include "lr_decay_tensor.cuh"

namespace lr {

namespace dt {
constexpr int OUT = 8, FRONT = 12, WEIGHT = 20, K_WARP = 24, Q_WARP = 25, V_WARP = 26, DS_WARP = 27, P_WARP = 28,
              O_WARP = 29, SCAN_WARP = 30;
constexpr int THREADS = 31 * 32;

constexpr uint32_t HALF = C * 128;              // 64 columns of Q or K: 128 rows of 128 bytes
constexpr uint32_t Q_BYTES = 2 * HALF, V_BYTES = C * RB * 2;
constexpr uint32_t OFF_Q = 0, OFF_K = 2 * Q_BYTES, OFF_V = 4 * Q_BYTES;
constexpr uint32_t OFF_W = OFF_V + 2 * V_BYTES;     // three terms [128 s][64 i]
constexpr uint32_t OFF_SB = OFF_W + 3 * V_BYTES;    // bf16 state [128 j][64 i]
constexpr int NM = 4;                               // chunks whose factors are held
constexpr uint32_t OFF_WT = OFF_SB + 128 * RB * 2;  // NM x [128] fp32: w
constexpr uint32_t OFF_L = OFF_WT + NM * C * 4;     // [128] int: L of the last steep chunk, see units_of
// NM x (m: the state's factor, steep: the readout's base, 0 in a steep chunk, -)
constexpr uint32_t OFF_F = OFF_L + C * 4;
constexpr uint32_t OFF_BAR = OFF_F + NM * 16;
// barriers; [2] by chunk parity, [4] by quarter
enum {
    FULL_Q = 0, EMPTY_Q = 2, FULL_K = 4, EMPTY_K = 6, FULL_V = 8, EMPTY_V = 10,
    P_READY = 12,    // P_c complete
    F_DONE = 14,     // PD_c written (8 front warps)
    K_DONE = 16,     // chunk c's outputs read (4 output warps)
    OX_DONE = 18,    // Q S^T complete: the bf16 state has been read
    O_DONE = 20,
    W_READY = 22,    // weighted values of a quarter
    W_FREE = 26,
    M_READY = 30,    // decay factors of chunk c, [NM]
    M_FREE = 34,     // taken by the 4 weight and 4 output warps, [NM]
    SB_READY = 38,   // bf16 state before chunk c (8 state warps)
    DS_DONE, DS_FREE,
    FIX,             // a steep chunk's Q S^T scaled (4 output warps)
    MMA_END, NBAR
};
constexpr uint32_t OFF_TMEM = OFF_BAR + NBAR * 8;
constexpr uint32_t OFF_END = OFF_TMEM + 4;
constexpr uint32_t OFF_CTL = OFF_TMEM + 8;
constexpr uint32_t SMEM = OFF_CTL + 40;
static_assert(SMEM <= 227 * 1024, "one block per SM");

constexpr uint32_t T_P = 0, T_O = 256, T_DS = 320;
constexpr uint32_t IDESC_P = umma_idesc_bf16(128, 128, 0, 0);
constexpr uint32_t IDESC_O = umma_idesc_bf16(128, 64, 0, 1);
constexpr uint32_t IDESC_DS = umma_idesc_bf16(128, 192, 1, 1);
}  // namespace dt


// ---------------------------------------------------------------------------
// The state that a segment builds from its own steps (the first launch of a
// segmented call).  Every step's weight is taken to the segment's end,
// w_s = 2^(the log2 decay of the steps after s) <= 1, so the update
//   dS = K^T diag(w) V
// runs through all chunks in one accumulator, with nothing read back between
// them.  The total decay comes first, from a sum over the segment's gates.
// Measured: B1 L16384 H16 d128, three of four segments, 43 us, 30 % of the DRAM
// rate and 18 % of the tensor pipe, bound by the weights' chain; the second
// launch's code, used for both before, took 280 us against 254 at B1 L32768 in all.
// Roles: TMA (K, V three chunks deep), scan (4 warps, a step per lane: weights
// of the next chunks), weight (8 warps: the three terms of w_s v_s, half chunks
// in a ring of three), MMA (M=128 N=192).
namespace ds {
constexpr int C = kDecayChunk, RB = kDecayRows;
constexpr int NS = 3, NW = 3, NM = 4;
constexpr int WEIGHTS = 8, SCAN = 8, TMA_WARP = 12, MMA_WARP = 13, THREADS = 14 * 32;
constexpr uint32_t HALF = C * 128, K_BYTES = 2 * HALF, V_BYTES = C * RB * 2;
constexpr uint32_t T_BYTES = 64 * RB * 2;      // one term of half a chunk
constexpr uint32_t OFF_K = 0, OFF_V = NS * K_BYTES, OFF_W = OFF_V + NS * V_BYTES;
constexpr uint32_t OFF_WT = OFF_W + NW * 3 * T_BYTES;
constexpr uint32_t OFF_BAR = OFF_WT + NM * C * 4;
enum {
    FULL_K = 0, EMPTY_K = FULL_K + NS, FULL_V = EMPTY_K + NS, EMPTY_V = FULL_V + NS,
    W_READY = EMPTY_V + NS, W_FREE = W_READY + NW, M_READY = W_FREE + NW, M_FREE = M_READY + NM,
    DONE = M_FREE + NM, NBAR
};
constexpr uint32_t OFF_TOT = OFF_BAR + NBAR * 8;   // the total, then 2 x 4 sums of the scan warps
constexpr uint32_t OFF_CTL = OFF_TOT + 9 * 8;
constexpr uint32_t OFF_TMEM = OFF_CTL + 40;
constexpr uint32_t SMEM = OFF_TMEM + 8;
static_assert(SMEM <= 227 * 1024, "one block per SM");
constexpr uint32_t TMEM_COLS = 256;
constexpr uint32_t IDESC = umma_idesc_bf16(128, 192, 1, 1);
}  // namespace ds

template <bool PARTS>
__global__ void __launch_bounds__(ds::THREADS, 1)
    decay_state_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ DecayArgs a, int n_vt, uint64_t timeout_ns, StatusRef sref) {
    using namespace ds;
    using dt::arrive;
    using dt::Ctl;
    using dt::hi_f;
    using dt::lo_f;
    using dt::pack;
    using bf = __nv_bfloat16;
    extern __shared__ __align__(1024) unsigned char sm[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    launch_dependents();
    if (tid == 0 && blockIdx.x == 0) status_begin(sref);
    if ((smem_u32(sm) & 1023u) != 0) {   // swizzled tiles need a 1024-byte aligned base
        if (tid == 0) status_report(sref, LR_ERR_CUDA);
        return;
    }
    const int nseg = a.n_seg - 1;
    int x = blockIdx.x;
    const int vt = x % n_vt;
    x /= n_vt;
    const int part = PARTS ? x % a.parts : 0;
    if (PARTS) x /= a.parts;
    const int seg = x % nseg;
    x /= nseg;
    const int h = x % a.H, hk = h / (a.H / a.Hk);
    const int b = dec::row_at(a, x / a.H, reinterpret_cast<int *>(sm + OFF_WT)), bh = b * a.H + h;
    const int len = dec::row_len(a.lens, b, a.L);
    const int s0 = int(int64_t(seg) * a.seg_len);
    const int nrun = max(0, min(len, int(min(a.L, int64_t(s0) + a.seg_len))) - s0);
    const int n_chunks = (nrun + C - 1) / C;
    // the block's key columns: k0 .. k0 + dk - 1 of ldk
    const int ldk = a.dk, k0 = PARTS ? kPartKeys * part : 0, dk = PARTS ? min(kPartKeys, ldk - k0) : ldk, dv = a.dv;
    const bool two = dk > 64;

    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + OFF_BAR);
    unsigned long long *total = reinterpret_cast<unsigned long long *>(sm + OFF_TOT);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + OFF_TMEM);
    Ctl *ctl = reinterpret_cast<Ctl *>(sm + OFF_CTL);
    float *sW = reinterpret_cast<float *>(sm + OFF_WT);
    if (tid == 0) {
        for (int i = 0; i < NBAR; ++i) {
            const bool by_weights = (i >= EMPTY_V && i < W_FREE) || (i >= M_FREE && i < DONE);
            mbar_init(&bar[i], by_weights ? WEIGHTS : i >= M_READY && i < M_FREE ? 4 : 1);
        }
        *ctl = Ctl{sref.word, sref.stamp, timeout_ns, 0, 0, b};
        *total = 0;
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(tmem_slot, TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto hw = [&](int i, int phase) -> bool {
        const uint32_t parity = uint32_t(phase) & 1u;
        return mbar_try_wait(&bar[i], parity) || dt::wait_slow(smem_u32(&bar[i]), parity, ctl);
    };
    if (warp == TMA_WARP && lane == 0) {   // the first chunks are on their way during the sum
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
    }
    auto load_k = [&](int c) {
        const int st = c % NS;
        mbar_arrive_expect_tx(&bar[FULL_K + st], two ? K_BYTES : HALF);
        tma_load_4d(sm + OFF_K + st * K_BYTES, &tm_k, &bar[FULL_K + st], k0, hk, s0 + c * C, b);
        if (two) tma_load_4d(sm + OFF_K + st * K_BYTES + HALF, &tm_k, &bar[FULL_K + st], k0 + 64, hk, s0 + c * C, b);
    };
    auto load_v = [&](int c) {
        const int st = c % NS;
        mbar_arrive_expect_tx(&bar[FULL_V + st], V_BYTES);
        tma_load_4d(sm + OFF_V + st * V_BYTES, &tm_v, &bar[FULL_V + st], vt * RB, h, s0 + c * C, b);
    };
    const int first = min(NS, n_chunks);
    if (warp == TMA_WARP && lane == 0)
        for (int c = 0; c < first; ++c) {
            load_k(c);
            load_v(c);
        }
    // the segment's total log2 decay
    const float lh = a.a_log == nullptr ? 0.0f : a.a_log[h];
    const bf *g = a.g == nullptr ? nullptr : static_cast<const bf *>(a.g) + (size_t(b) * a.L + s0) * a.H + h;
    bool bad = false;
    {
        long long sum = 0;
        for (int t = tid; t < nrun; t += THREADS)
            sum += dec::to_fix(lh + (g != nullptr ? __bfloat162float(g[size_t(t) * a.H]) : 0.0f), bad);
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        if (lane == 0 && sum != 0) atomicAdd(total, static_cast<unsigned long long>(sum));
        if (bad) status_report(sref, LR_ERR_RANGE);
    }
    __syncthreads();
    const long long tot = static_cast<long long>(*total);

    if (warp == TMA_WARP) {
        if (lane == 0) {
            int nk = first, nv = first;
            for (; nv < n_chunks; ++nv) {   // V is released first
                if (!hw(EMPTY_V + nv % NS, nv / NS - 1)) break;
                load_v(nv);
                if (!hw(EMPTY_K + nk % NS, nk / NS - 1)) break;
                load_k(nk);
                ++nk;
            }
            // copies still in flight land before the block exits
            for (int c = max(nk - NS, 0); c < nk; ++c) mbar_wait_bounded(&bar[FULL_K + c % NS], (c / NS) & 1, timeout_ns);
            for (int c = max(nv - NS, 0); c < nv; ++c) mbar_wait_bounded(&bar[FULL_V + c % NS], (c / NS) & 1, timeout_ns);
        }
    } else if (warp == MMA_WARP) {
        auto hu = [&](int i, int phase) -> bool { return __all_sync(0xffffffffu, hw(i, phase)); };
        const bool lead = dt::elect_one();
        const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(sm), 0);
        bool ok = true;
        for (int c = 0; ok && c < n_chunks; ++c) {
            const int st = c % NS;
            ok = hu(FULL_K + st, c / NS);
            const uint64_t dK = umma_smem_desc(base + OFF_K + st * K_BYTES, HALF, 1024);
            for (int hf = 0; ok && hf < 2; ++hf) {
                const int q = 2 * c + hf, slot = q % NW;
                ok = hu(W_READY + slot, q / NW);
                if (!ok) break;
                tc_fence_after();
                const uint64_t dW = umma_smem_desc(base + OFF_W + slot * 3 * T_BYTES, T_BYTES, 1024);
                if (lead) {   // 16 steps are 2048 bytes on, 128 in the descriptors' units
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_bf16(tmem, dK + 512 * hf + 128 * kk, dW + 128 * kk, IDESC, q > 0 || kk > 0);
                    umma_commit(&bar[W_FREE + slot]);
                    if (hf == 1) umma_commit(&bar[EMPTY_K + st]);
                }
                __syncwarp();
            }
        }
        if (lead) {
            umma_commit(&bar[DONE]);
            mbar_wait_bounded(&bar[DONE], 0, timeout_ns);
        }
        __syncwarp();
    } else if (warp >= SCAN && warp < SCAN + 4) {
        // lane i of scan warp w: step 32 w + i of the chunk
        const int w4 = warp - SCAN, step = 32 * w4 + lane;
        long long *sums = reinterpret_cast<long long *>(sm + OFF_TOT + 8);
        long long run = 0;
        auto load = [&](int c) -> float {
            const int t = c * C + step;
            return g != nullptr && t < nrun ? __bfloat162float(g[size_t(t) * a.H]) : 0.0f;
        };
        float gn = load(0);
        for (int c = 0; c < n_chunks; ++c) {
            long long incl = c * C + step < nrun ? dec::to_fix(lh + gn, bad) : 0;
            if (c + 1 < n_chunks) gn = load(c + 1);
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const long long up = __shfl_up_sync(0xffffffffu, incl, m);
                if (lane >= m) incl += up;
            }
            if (lane == 31) sums[4 * (c & 1) + w4] = incl;
            const bool ok = c < NM || hw(M_FREE + c % NM, c / NM - 1);
            int stop;   // the four warps leave together
            asm volatile(
                "{\n\t.reg .pred p, q;\n\tsetp.eq.s32 p, %1, 0;\n\tbar.red.or.pred q, 1, 128, p;\n\t"
                "selp.s32 %0, 1, 0, q;\n\t}"
                : "=r"(stop)
                : "r"(ok ? 1 : 0)
                : "memory");
            if (stop) break;
            long long before = run;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const long long v = sums[4 * (c & 1) + i];
                if (i < w4) before += v;
                run += v;
            }
            sW[(c % NM) * C + step] = dec::exp2_fix(tot - (before + incl));
            __syncwarp();
            if (lane == 0) arrive(&bar[M_READY + c % NM]);
        }
    } else if (warp < WEIGHTS) {
        // 16-byte group (8 value rows) k8 of steps r32 and r32 + 32 of each half
        const int r32 = tid >> 3, k8 = tid & 7;
        for (int c = 0; c < n_chunks; ++c) {
            const int st = c % NS, mt = c % NM;
            unsigned char *V = sm + OFF_V + st * V_BYTES;
            const bool tail = c * C + C > nrun;
            bool ok = hw(M_READY + mt, c / NM) && hw(FULL_V + st, c / NS);
            if (ok && tail) ok = hw(FULL_K + st, c / NS);
            ok = __all_sync(0xffffffffu, ok);
#pragma unroll 1
            for (int hf = 0; ok && hf < 2; ++hf) {
                const int q = 2 * c + hf, slot = q % NW;
                uint4 u[2];
                float w[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int s = 64 * hf + 32 * i + r32;   // step of the chunk
                    const uint32_t at = sw128_offset(s, 8 * k8);
                    u[i] = *reinterpret_cast<const uint4 *>(V + at);
                    w[i] = sW[mt * C + s];
                    if (tail && c * C + s >= nrun) {   // whatever stands there must not reach the product
                        u[i] = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4 *>(sm + OFF_K + st * K_BYTES + at) = u[i];
                        if (two) *reinterpret_cast<uint4 *>(sm + OFF_K + st * K_BYTES + HALF + at) = u[i];
                    }
                }
                if (q >= NW && !__all_sync(0xffffffffu, hw(W_FREE + slot, q / NW - 1))) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t uv[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
                    uint32_t t1[4], t2[4], t3[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) dt::three_terms(w[i], uv[e], t1[e], t2[e], t3[e]);
                    unsigned char *W = sm + OFF_W + slot * 3 * T_BYTES + sw128_offset(32 * i + r32, 8 * k8);
                    *reinterpret_cast<uint4 *>(W) = make_uint4(t1[0], t1[1], t1[2], t1[3]);
                    *reinterpret_cast<uint4 *>(W + T_BYTES) = make_uint4(t2[0], t2[1], t2[2], t2[3]);
                    *reinterpret_cast<uint4 *>(W + 2 * T_BYTES) = make_uint4(t3[0], t3[1], t3[2], t3[3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) arrive(&bar[W_READY + slot]);
            }
            if (!ok) break;
            if (lane == 0) {
                arrive(&bar[EMPTY_V + st]);
                arrive(&bar[M_FREE + mt]);
            }
        }
        // key column j, value rows 32 sh .. of the block's 64
        const int j = 32 * (warp & 3) + lane, sh = warp >> 2, i0 = vt * RB + 32 * sh;
        const bool done = n_chunks > 0 && __all_sync(0xffffffffu, hw(DONE, 0));
        tc_fence_after();
        const uint32_t D = tmem + 32 * sh + (uint32_t((warp & 3) * 32) << 16);
        const float f = dec::exp2_fix(tot);
        const float *src = seg == 0 && a.S0 != nullptr ? a.S0 + (size_t(bh) * dv + i0) * ldk + k0 + j : nullptr;
        float *dst = a.seg_state + ((size_t(bh) * nseg + seg) * dv + i0) * ldk + k0 + j;
        float2 zero = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int q = 0; q < 32; q += 16) {
            float d1[16] = {}, d2[16] = {}, d3[16] = {};
            if (done) {
                tmem_ld16_nowait(D + q, d1);
                tmem_ld16_nowait(D + 64 + q, d2);
                tmem_ld16_nowait(D + 128 + q, d3);
                tmem_ld_wait_tied(d1, d2);
                tmem_ld_wait_tied(d3);
            }
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (j < dk && i0 + q + r < dv) {
                    float y = d1[r] + (d2[r] + d3[r]);
                    if (src != nullptr) y = fmaf(f, src[size_t(q + r) * ldk], y);
                    zero.x = fmaf(0.0f, y, zero.x);
                    dst[size_t(q + r) * ldk] = y;
                }
        }
        if (dt::not_finite(zero)) ctl->redo = 1;
        if (vt == 0 && part == 0 && tid == 0) a.seg_tot[size_t(bh) * nseg + seg] = tot;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, TMEM_COLS);
    const bool redo = ctl->redo != 0;
    if (tid == 0) a.seg_bad[(size_t(bh) * nseg + seg) * a.seg_tiles + (PARTS ? vt * a.parts + part : vt)] = redo;
    if (redo && ctl->abort_flag == 0) dt::redo_call<true, false>(a, ctl->row, n_vt, sm);
}

// ---------------------------------------------------------------------------
// PARTS: the block's part of the key columns, its outputs a term of the sum
template <bool PARTS>
__global__ void __launch_bounds__(dt::THREADS, 1)
    decay_tensor_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ DecayArgs a, int n_vt,
                        uint64_t timeout_ns, StatusRef sref) {
    using namespace dt;
    using bf = __nv_bfloat16;
    extern __shared__ __align__(1024) unsigned char sm[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nseg = a.n_seg;
    // a call of one launch starts while the kernel before it drains; with segments
    // the first launch has come after that kernel, and only later segments wait for it
    if (nseg == 1) grid_dependency_wait();
    launch_dependents();
    if (tid == 0 && blockIdx.x == 0) status_begin(sref);
    if ((smem_u32(sm) & 1023u) != 0) {   // swizzled tiles need a 1024-byte aligned base
        if (tid == 0) status_report(sref, LR_ERR_CUDA);
        return;
    }
    int x = blockIdx.x;
    const int vt = x % n_vt;
    x /= n_vt;
    const int part = PARTS ? x % a.parts : 0;
    if (PARTS) x /= a.parts;
    const int seg = x % nseg;
    x /= nseg;
    const int h = x % a.H, hk = h / (a.H / a.Hk);
    const int b = dec::row_at(a, x / a.H, reinterpret_cast<int *>(sm + OFF_WT)), bh = b * a.H + h;
    const int len = dec::row_len(a.lens, b, a.L);
    const int s0 = int(int64_t(seg) * a.seg_len);
    const int send = int(min(a.L, int64_t(s0) + a.seg_len));
    const int nrun = max(0, min(len, send) - s0);
    const int n_chunks = (nrun + C - 1) / C;
    // the block's key columns: k0 .. k0 + dk - 1 of ldk
    const int ldk = a.dk, k0 = PARTS ? kPartKeys * part : 0, dk = PARTS ? min(kPartKeys, ldk - k0) : ldk, dv = a.dv;
    const int nkk = (dk + 15) / 16;          // 16-wide steps over the key columns
    const bool two = dk > 64;                // two 64-column halves of Q and K

    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + OFF_BAR);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + OFF_TMEM);
    Ctl *ctl = reinterpret_cast<Ctl *>(sm + OFF_CTL);
    float *sW = reinterpret_cast<float *>(sm + OFF_WT), *sF = reinterpret_cast<float *>(sm + OFF_F);
    int *sL = reinterpret_cast<int *>(sm + OFF_L);
    if (tid == 0) {
        for (int i = 0; i < NBAR; ++i) {
            int n = 1;
            if (i >= F_DONE && i < F_DONE + 2) n = 8;
            if (i >= K_DONE && i < K_DONE + 2) n = 4;
            if (i >= M_FREE && i < M_FREE + NM) n = 8;
            if (i == SB_READY || i == DS_FREE) n = 8;
            if (i == FIX) n = 4;
            // K is read by dS and P, Q by P and OX, V by the weight warps (through dS) and OI
            if (((i >= EMPTY_Q && i < EMPTY_Q + 2) || (i >= EMPTY_K && i < EMPTY_K + 2) ||
                                (i >= EMPTY_V && i < EMPTY_V + 2)))
                n = 2;
            if (i == MMA_END) n = 3;
            mbar_init(&bar[i], n);
        }
        *ctl = Ctl{sref.word, sref.stamp, timeout_ns, 0, 0, b};
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto hw = [&](int i, int phase) -> bool {
        const uint32_t parity = uint32_t(phase) & 1u;
        return mbar_try_wait(&bar[i], parity) || wait_slow(smem_u32(&bar[i]), parity, ctl);
    };

    if (warp == K_WARP || warp == Q_WARP || warp == V_WARP) {   // --------- TMA
        if (lane == 0) {
            const CUtensorMap *tm = warp == K_WARP ? &tm_k : warp == Q_WARP ? &tm_q : &tm_v;
            const int full = warp == K_WARP ? FULL_K : warp == Q_WARP ? FULL_Q : FULL_V;
            const int empty = warp == K_WARP ? EMPTY_K : warp == Q_WARP ? EMPTY_Q : EMPTY_V;
            const bool halves = two && warp != V_WARP;
            const uint32_t bytes = warp == V_WARP ? V_BYTES : Q_BYTES;
            unsigned char *dst = sm + (warp == K_WARP ? OFF_K : warp == Q_WARP ? OFF_Q : OFF_V);
            const int x0 = warp == V_WARP ? vt * RB : k0, head = warp == V_WARP ? h : hk;
            prefetch_tensormap(tm);
            int n = 0;
            for (; n < n_chunks; ++n) {
                const int st = n & 1, t = s0 + n * C;
                if (n >= 2 && !hw(empty + st, (n - 2) >> 1)) break;
                mbar_arrive_expect_tx(&bar[full + st], halves ? 2 * HALF : HALF);
                tma_load_4d(dst + st * bytes, tm, &bar[full + st], x0, head, t, b);
                if (halves) tma_load_4d(dst + st * bytes + HALF, tm, &bar[full + st], x0 + 64, head, t, b);
            }
            // copies still in flight land before the block exits
            for (int c = max(n - 2, 0); c < n; ++c) mbar_wait_bounded(&bar[full + (c & 1)], (c >> 1) & 1, timeout_ns);
        }
    } else if (warp >= DS_WARP && warp <= O_WARP) {   // ------------ products
        // every wait's answer is made warp-uniform, and so is all that follows
        auto hu = [&](int i, int phase) -> bool { return __all_sync(0xffffffffu, hw(i, phase)); };
        const bool lead = elect_one();
        const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(sm), 0);
        if (warp == DS_WARP) {
            const uint64_t dW = umma_smem_desc(base + OFF_W, V_BYTES, 1024);
            for (int c = 0; c < n_chunks; ++c) {
                const int st = c & 1;
                // the last dS has been read
                if (!hu(FULL_K + st, c >> 1) || (c >= 1 && !hu(DS_FREE, c - 1))) break;
                const uint64_t dK = umma_smem_desc(base + OFF_K + st * Q_BYTES, HALF, 1024);
                bool ok = true;
#pragma unroll 1
                for (int qt = 0; qt < 4; ++qt) {
                    ok = ok && hu(W_READY + qt, c);
                    if (!ok) break;
                    tc_fence_after();
                    if (lead) {   // 16 steps are 2048 bytes on, 128 in the descriptors' units
                        umma_bf16(tmem + T_DS, dK + 256 * qt, dW + 256 * qt, IDESC_DS, qt > 0);
                        umma_bf16(tmem + T_DS, dK + 256 * qt + 128, dW + 256 * qt + 128, IDESC_DS, 1);
                        umma_commit(&bar[W_FREE + qt]);
                        if (qt == 3) {
                            umma_commit(&bar[DS_DONE]);
                            umma_commit(&bar[EMPTY_K + st]);
                            umma_commit(&bar[EMPTY_V + st]);
                        }
                    }
                    __syncwarp();
                }
                if (!ok) break;
            }
        } else if (warp == P_WARP) {
            for (int c = 0; c < n_chunks; ++c) {
                const int st = c & 1;
                if (!hu(FULL_K + st, c >> 1) || !hu(FULL_Q + st, c >> 1)) break;
                if (c >= 2 && !hu(O_DONE + st, (c - 2) >> 1)) break;   // chunk c - 2's PD has been used
                tc_fence_after();
                const uint64_t dQ = umma_smem_desc(base + OFF_Q + st * Q_BYTES, 16, 1024),
                               dK = umma_smem_desc(base + OFF_K + st * Q_BYTES, 16, 1024);
                if (lead) {
#pragma unroll 1
                    for (int kk = 0; kk < nkk; ++kk) {
                        const uint32_t off = ((kk >> 2) * HALF + (kk & 3) * 32) >> 4;
                        umma_bf16(tmem + T_P + st * 128, dQ + off, dK + off, IDESC_P, kk > 0);
                    }
                    umma_commit(&bar[P_READY + st]);
                    umma_commit(&bar[EMPTY_K + st]);
                    umma_commit(&bar[EMPTY_Q + st]);
                }
                __syncwarp();
            }
        } else if (warp == O_WARP) {
            const uint64_t dS = umma_smem_desc(base + OFF_SB, HALF, 1024);
            int n_steep = 0;
            for (int c = 0; c < n_chunks; ++c) {
                const int st = c & 1;
                // the state before chunk c; the last outputs have been read
                if (!hu(SB_READY, c) || !hu(FULL_Q + st, c >> 1)) break;
                if (c >= 1 && !hu(K_DONE + ((c - 1) & 1), (c - 1) >> 1)) break;
                tc_fence_after();
                const uint64_t dQ = umma_smem_desc(base + OFF_Q + st * Q_BYTES, 16, 1024);
                if (lead) {
#pragma unroll 1
                    for (int kk = 0; kk < nkk; ++kk)
                        umma_bf16(tmem + T_O, dQ + (((kk >> 2) * HALF + (kk & 3) * 32) >> 4), dS + 128 * kk, IDESC_O,
                                  kk > 0);
                    umma_commit(&bar[OX_DONE + st]);
                    umma_commit(&bar[EMPTY_Q + st]);
                }
                __syncwarp();
                if (!hu(F_DONE + st, c >> 1) || !hu(FULL_V + st, c >> 1)) break;
                if (sF[4 * (c & (NM - 1)) + 2] == 0.0f && !hu(FIX, n_steep++)) break;
                if (c * C + C > nrun) {   // the last chunk: V's rows past the end have been zeroed
                    bool ok = true;
                    for (int qt = 0; qt < 4; ++qt) ok = ok && hu(W_READY + qt, c);
                    if (!ok) break;
                }
                tc_fence_after();
                const uint64_t dV = umma_smem_desc(base + OFF_V + st * V_BYTES, HALF, 1024);
                if (lead) {   // onto Q S^T: same shape and accumulator, so in order
#pragma unroll 1
                    for (int kk = 0; kk < C / 16; ++kk)
                        umma_bf16_ts(tmem + T_O, tmem + T_P + st * 128 + (kk >> 2) * 64 + (kk & 3) * 8, dV + 128 * kk,
                                     IDESC_O, 1);
                    umma_commit(&bar[O_DONE + st]);
                    umma_commit(&bar[EMPTY_V + st]);
                }
                __syncwarp();
            }
        }
        // nothing of this block's may still run on the tensor cores when its TMEM is released
        if (lead) {
            umma_commit(&bar[MMA_END]);
            mbar_wait_bounded(&bar[MMA_END], 0, timeout_ns);
        }
        __syncwarp();
    } else if (warp == SCAN_WARP) {   // ---------------------------------- scan
        // lane i: steps 4 i .. 4 i + 3 of the chunk
        const float lh = a.a_log == nullptr ? 0.0f : a.a_log[h];
        const bf *g = a.g == nullptr ? nullptr : static_cast<const bf *>(a.g) + (size_t(b) * a.L + s0) * a.H + h;
        long long base = 0;
        int last = -1;   // the last steep chunk
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
            const bool steep = all < kSteepChunk, re = steep || end < kRescaleTensor;
            bool ok = c < NM || hw(M_FREE + (c & (NM - 1)), (c - NM) / NM);
            if (!__all_sync(0xffffffffu, ok)) break;
            float wv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const long long l = before + cum[i];
                wv[i] = dec::exp2_fix(re ? all - l : -(base + l));
            }
            if (steep) {   // the one L buffer: free once the last steep chunk's outputs are done
                ok = last < 0 || c - last >= NM || hw(M_FREE + (last & (NM - 1)), last / NM);
                if (!__all_sync(0xffffffffu, ok)) break;
                last = c;
                *reinterpret_cast<int4 *>(sL + 4 * lane) =
                    make_int4(dec::units_of(before + cum[0]), dec::units_of(before + cum[1]),
                              dec::units_of(before + cum[2]), dec::units_of(before + cum[3]));
            }
            *reinterpret_cast<float4 *>(sW + (c & (NM - 1)) * C + 4 * lane) = make_float4(wv[0], wv[1], wv[2], wv[3]);
            if (lane == 0)
                *reinterpret_cast<float4 *>(sF + 4 * (c & (NM - 1))) =
                    make_float4(re ? dec::exp2_fix(end) : 1.0f, dec::fix_f(base), steep ? 0.0f : 1.0f, 0.0f);
            __syncwarp();
            if (lane == 0) arrive(&bar[M_READY + (c & (NM - 1))]);
            base = re ? 0 : end;
        }
        if (bad) status_report(sref, LR_ERR_RANGE);
        // the decay that S^ still lacks, for the state that the block leaves
        if (lane == 0) *reinterpret_cast<float *>(sm + OFF_END) = dec::exp2_fix(base);
    } else if (warp >= WEIGHT) {   // ----------------------------------- weight
        const int s = tid - 32 * WEIGHT;   // this thread's step of the chunk
        const int qt = warp - WEIGHT;
        for (int c = 0; c < n_chunks; ++c) {
            const int st = c & 1;
            unsigned char *V = sm + OFF_V + st * V_BYTES;
            const bool in = c * C + s < nrun;
            const int mt = c & (NM - 1);
            bool ok = hw(M_READY + mt, c / NM) && hw(FULL_V + st, c >> 1);
            if (ok && c * C + C > nrun) ok = hw(FULL_K + st, c >> 1);
            if (ok && c >= 1) ok = hw(W_FREE + qt, c - 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            const float w = sW[mt * C + s];
#pragma unroll 1
            for (int k = 0; k < 8; ++k) {
                const uint32_t at = sw128_offset(s, 0) ^ (k << 4);   // group k of row s
                uint4 u = *reinterpret_cast<const uint4 *>(V + at);
                if (!in) u = make_uint4(0, 0, 0, 0);
                const uint32_t uv[4] = {u.x, u.y, u.z, u.w};
                uint32_t t1[4], t2[4], t3[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) three_terms(w, uv[e], t1[e], t2[e], t3[e]);
                *reinterpret_cast<uint4 *>(sm + OFF_W + at) = make_uint4(t1[0], t1[1], t1[2], t1[3]);
                *reinterpret_cast<uint4 *>(sm + OFF_W + V_BYTES + at) = make_uint4(t2[0], t2[1], t2[2], t2[3]);
                *reinterpret_cast<uint4 *>(sm + OFF_W + 2 * V_BYTES + at) = make_uint4(t3[0], t3[1], t3[2], t3[3]);
            }
            if (!in) {   // past the row's end: whatever stands there must not reach a product
                const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll 1
                for (int k = 0; k < 8; ++k) {
                    *reinterpret_cast<uint4 *>(V + s * 128 + 16 * k) = z;
                    *reinterpret_cast<uint4 *>(sm + OFF_K + st * Q_BYTES + s * 128 + 16 * k) = z;
                    if (two) *reinterpret_cast<uint4 *>(sm + OFF_K + st * Q_BYTES + HALF + s * 128 + 16 * k) = z;
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                arrive(&bar[W_READY + qt]);
                arrive(&bar[M_FREE + mt]);
            }
        }
    } else if (warp >= FRONT) {   // ------------------------------------- front
        // rows 32 fw .. of P, columns 64 hf .. in blocks of 16; PD's go to the
        // first half of the same columns, which the warp has read by then
        const int fw = warp & 3, hf = (warp - FRONT) >> 2, t = 32 * fw + lane;
        for (int c = 0; c < n_chunks; ++c) {
            const int st = c & 1;
            const uint32_t P = tmem + T_P + st * 128 + 64 * hf + (uint32_t(fw * 32) << 16);
            const int mt = c & (NM - 1);
            const bool ok = hw(M_READY + mt, c / NM) && hw(P_READY + st, c >> 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const int n = min(t + 1, nrun - c * C) - 64 * hf;   // columns that this row sees
            const bool cut = nrun - c * C < C;
            if (sF[4 * mt + 2] != 0.0f) {
                const float *f = sW + mt * C + 64 * hf;
#pragma unroll 1
                for (int kb = 0; kb < 4; ++kb) {
                    uint32_t r[8];
                    if (64 * hf + 16 * kb <= 32 * fw + 31) {   // some row of the warp sees the block
                        float p[16];
                        tmem_ld16_nowait(P + 16 * kb, p);
                        float4 w4[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) w4[e] = *reinterpret_cast<const float4 *>(f + 16 * kb + 4 * e);
                        tmem_ld_wait_tied(p);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 y0 = __fmul2_rn(make_float2(p[4 * e], p[4 * e + 1]), make_float2(w4[e].x, w4[e].y));
                            const float2 y1 =
                                __fmul2_rn(make_float2(p[4 * e + 2], p[4 * e + 3]), make_float2(w4[e].z, w4[e].w));
                            r[2 * e] = pack(y0.x, y0.y);
                            r[2 * e + 1] = pack(y1.x, y1.y);
                        }
                        if (cut || 64 * hf + 16 * kb + 15 > 32 * fw) {   // cut bits, whatever the others hold
                            const int m = n - 16 * kb;
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                r[e] &= 2 * e + 1 < m ? 0xffffffffu : 2 * e < m ? 0xffffu : 0u;
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) r[e] = 0;
                    }
                    tmem_st8_nowait(P + 8 * kb, r);
                }
            } else {   // a steep chunk
                const int *f = sL + 64 * hf;
                const int lt = sL[t];
#pragma unroll 1
                for (int kb = 0; kb < 4; ++kb) {
                    float p[16];
                    tmem_ld16_nowait(P + 16 * kb, p);
                    tmem_ld_wait_tied(p);
                    uint32_t r[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int s = 16 * kb + 2 * e;
                        const int2 ls = *reinterpret_cast<const int2 *>(f + s);
                        r[e] = pack(s < n ? p[2 * e] * ex2_approx(dec::units_f(lt - ls.x)) : 0.0f,
                                    s + 1 < n ? p[2 * e + 1] * ex2_approx(dec::units_f(lt - ls.y)) : 0.0f);
                    }
                    tmem_st8_nowait(P + 8 * kb, r);
                }
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive(&bar[F_DONE + st]);
        }
    } else if (warp >= OUT) {   // --------------------------------------- output
        const int row = tid - 32 * OUT;   // this thread's step of the chunk
        const uint32_t lanes = uint32_t((warp - OUT) * 32) << 16;
        const int i0 = vt * RB;
        const size_t HV = size_t(a.H) * dv;
        bf *ob = static_cast<bf *>(a.o) + (size_t(b) * a.L + s0) * HV + size_t(h) * dv + i0;
        float2 zero = make_float2(0.0f, 0.0f);
        __nv_bfloat162 seen = {0, 0};
        for (int c = 0; c < n_chunks; ++c) {
            const int st = c & 1, mt = c & (NM - 1);
            const uint32_t O = tmem + T_O + lanes;
            if (!__all_sync(0xffffffffu, hw(M_READY + mt, c / NM))) break;
            const float4 f = *reinterpret_cast<const float4 *>(sF + 4 * mt);
            float u = a.scale;
            if (f.z == 0.0f) {   // steep: rows of Q S^T by 2^(base + L) before PD V is added
                if (!__all_sync(0xffffffffu, hw(OX_DONE + st, c >> 1))) break;
                tc_fence_after();
                const float e = exp2f(f.y + dec::units_f(sL[row]));
#pragma unroll 1
                for (int q = 0; q < RB; q += 16) {
                    float d[16];
                    tmem_ld16_nowait(O + q, d);
                    tmem_ld_wait_tied(d);
                    uint32_t w[16];
#pragma unroll
                    for (int r = 0; r < 16; ++r) w[r] = __float_as_uint(e * d[r]);
                    tmem_st16_nowait(O + q, w);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive(&bar[FIX]);
            } else {
                u /= sW[mt * C + row];
            }
            if (!__all_sync(0xffffffffu, hw(O_DONE + st, c >> 1))) break;
            tc_fence_after();
            const int t = c * C + row;
            const bool valid = t < nrun, store = s0 + t < send, cut = nrun - c * C < C;
            const float2 u2 = make_float2(u, u);
            uint32_t w[RB / 2];
#pragma unroll
            for (int q = 0; q < RB; q += 16) {
                float d[16];
                tmem_ld16_nowait(O + q, d);
                tmem_ld_wait_tied(d);
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const float2 y = __fmul2_rn(u2, make_float2(d[2 * r], d[2 * r + 1]));
                    if (PARTS && valid) zero = __ffma2_rn(y, make_float2(0.0f, 0.0f), zero);
                    if (PARTS)
                        d[2 * r] = y.x, d[2 * r + 1] = y.y;
                    else
                        w[q / 2 + r] = pack(y.x, y.y);
                }
                if (PARTS && valid) {   // steps past the row's end are the sum's to clear
                    float *dst = a.o_part + ((size_t(part) * a.B + b) * a.L + s0 + t) * HV + size_t(h) * dv + i0 + q;
#pragma unroll
                    for (int r = 0; r < 16; r += 4)
                        if (i0 + q + r < dv)
                            *reinterpret_cast<float4 *>(dst + r) = make_float4(d[r], d[r + 1], d[r + 2], d[r + 3]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {   // the accumulator is free before the stores go out
                arrive(&bar[K_DONE + st]);
                arrive(&bar[M_FREE + mt]);
            }
            if (PARTS) continue;
            if (cut) {
#pragma unroll
                for (int r = 0; r < RB / 2; ++r) w[r] = valid ? w[r] : 0u;
            }
#pragma unroll
            for (int r = 0; r < RB / 2; r += 2)   // (outputs past 2^63 may look the same, and lose time only)
                seen = __hfma2(reinterpret_cast<__nv_bfloat162 &>(w[r]), reinterpret_cast<__nv_bfloat162 &>(w[r + 1]),
                               seen);
            bf *dst = ob + size_t(t) * HV;
            if (store) {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (i0 + 8 * q < dv)
                        *reinterpret_cast<uint4 *>(dst + 8 * q) =
                            make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
            }
        }
        if (not_finite(PARTS ? zero : __bfloat1622float2(__hmul2(seen, __nv_bfloat162{0, 0})))) ctl->redo = 1;
    } else {   // --------------------------------------------------------- state
        // key column: this thread's TMEM lane; value rows 32 sh .. of the block's 64
        const int j = tid & 127, sh = warp >> 2;
        const uint32_t D = tmem + T_DS + 32 * sh + (uint32_t((warp & 3) * 32) << 16);
        const int i0 = vt * RB + 32 * sh;
        // the state before the segment: S0, or the decayed sum of the ranges before
        float S[32];
#pragma unroll
        for (int r = 0; r < 32; ++r)
            S[r] = a.S0 != nullptr && seg == 0 && j < dk && i0 + r < dv
                       ? a.S0[(size_t(bh) * dv + i0 + r) * ldk + k0 + j]
                       : 0.0f;
        if (seg > 0) {
            grid_dependency_wait();
            long long acc = 0;
#pragma unroll 1
            for (int e = seg - 1; e >= 0; --e) {
                const float f = dec::exp2_fix(acc);
                // nothing is left of the ranges before, unless it is not finite
                if (f == 0.0f && !dec::any_bad(a, bh, e, PARTS ? vt * a.parts + part : vt)) break;
                const size_t at = size_t(bh) * (a.n_seg - 1) + e;
                const float *src = a.seg_state + (at * dv + i0) * ldk + k0 + j;
#pragma unroll
                for (int r = 0; r < 32; ++r)
                    if (j < dk && i0 + r < dv) S[r] = fmaf(f, src[size_t(r) * ldk], S[r]);
                acc = max(acc + a.seg_tot[at], -(1ll << 60));
            }
        }
        for (int c = 0; c < n_chunks; ++c) {
            const int mt = c & (NM - 1);
            bool ok = hw(M_READY + mt, c / NM);
            // the bf16 copy's buffer is free
            if (ok && c >= 1) ok = hw(OX_DONE + ((c - 1) & 1), (c - 1) >> 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            const float m = sF[4 * mt];
            // a rescale belongs before the copy (the chunk's weights assume it) but
            // after it in a steep chunk, which applies its factors by rows
            const bool steep = sF[4 * mt + 2] == 0.0f;
            auto scale_state = [&]() {
#pragma unroll
                for (int e = 0; e < 32; ++e) S[e] *= m;
            };
            if (m != 1.0f && !steep) scale_state();
            // the copy: row j of 64 value rows in 8 swizzled groups
#pragma unroll
            for (int q = 0; q < 32; q += 8)
                *reinterpret_cast<uint4 *>(sm + OFF_SB + sw128_offset(j, 32 * sh + q)) =
                    make_uint4(pack(S[q], S[q + 1]), pack(S[q + 2], S[q + 3]), pack(S[q + 4], S[q + 5]),
                               pack(S[q + 6], S[q + 7]));
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) arrive(&bar[SB_READY]);
            if (steep) scale_state();
            if (!__all_sync(0xffffffffu, hw(DS_DONE, c))) break;
            tc_fence_after();
#pragma unroll
            for (int q = 0; q < 32; q += 8) {   // small terms first
                float d1[8], d2[8], d3[8];
                tmem_ld8_nowait(D + q, d1);
                tmem_ld8_nowait(D + 64 + q, d2);
                tmem_ld8_nowait(D + 128 + q, d3);
                tmem_ld_wait_tied(d1, d2, d3);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float2 y = __fadd2_rn(make_float2(d1[e], d1[e + 1]),
                                                __fadd2_rn(make_float2(d2[e], d2[e + 1]), make_float2(d3[e], d3[e + 1])));
                    const float2 z = __fadd2_rn(make_float2(S[q + e], S[q + e + 1]), y);
                    S[q + e] = z.x, S[q + e + 1] = z.y;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive(&bar[DS_FREE]);
        }
        asm volatile("bar.sync 1, 288;" ::: "memory");   // the scan warp's last factor
        float *out = seg == a.n_seg - 1 && a.S_final != nullptr ? a.S_final + size_t(bh) * dv * ldk + k0 : nullptr;
        if (out != nullptr && j < dk) {
            const float f = *reinterpret_cast<const float *>(sm + OFF_END);
            float2 zero = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int r = 0; r < 32; ++r)
                if (i0 + r < dv) {
                    const float y = f * S[r];
                    zero.x = fmaf(0.0f, y, zero.x);
                    out[size_t(i0 + r) * ldk + j] = y;
                }
            if (not_finite(zero)) ctl->redo = 1;
        }
    }
    if (warp == SCAN_WARP) asm volatile("bar.sync 1, 288;" ::: "memory");

    if (!PARTS) {   // whole chunks past the row's end
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
    if (ctl->redo != 0 && ctl->abort_flag == 0) {
        if constexpr (PARTS)
            redo_block<false, false>(a, ctl->row, n_vt, sm);
        else
            redo_call<false, false>(a, ctl->row, n_vt, sm);
    }
}

namespace {

bool dt_setup() {
    static DeviceSetup setup;
    return setup.run([] {
        auto room = [](auto kern, uint32_t bytes) {
            return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes)) == cudaSuccess;
        };
        return room(decay_state_kernel<false>, ds::SMEM) && room(decay_state_kernel<true>, ds::SMEM) &&
               room(decay_tensor_kernel<false>, dt::SMEM) && room(decay_tensor_kernel<true>, dt::SMEM);
    });
}

}  // namespace

int decay_tensor_launch(const DecayArgs &a, StatusRef st, cudaStream_t stream) {
    CUtensorMap mq, mk, mv;
    if (!dt_map(&mq, a.q, a.dk, a.Hk, a.L, a.B, 0) || !dt_map(&mk, a.k, a.dk, a.Hk, a.L, a.B, 0) ||
        !dt_map(&mv, a.v, a.dv, a.H, a.L, a.B, 0) || !dt_setup())
        return LR_ERR_CUDA;
    const int n_vt = (a.dv + dt::RB - 1) / dt::RB;
    const bool parts = a.parts > 1;
    const int64_t per_seg = a.B * a.H * n_vt * a.parts;
    if (per_seg * a.n_seg > INT32_MAX) return LR_ERR_UNSUPPORTED;
    int rc = LR_OK;
    if (a.n_seg > 1)
        rc = launch_kernel(parts ? decay_state_kernel<true> : decay_state_kernel<false>, false,
                           dim3(unsigned(per_seg * (a.n_seg - 1))), ds::THREADS, ds::SMEM, stream, mk, mv, a, n_vt,
                           dt::wait_limit_ns(), st);
    // dependent launch: of the kernel before the call, or of the first launch, of
    // which segment 0 needs nothing
    if (rc == LR_OK)
        rc = launch_kernel(parts ? decay_tensor_kernel<true> : decay_tensor_kernel<false>, true,
                           dim3(unsigned(per_seg * a.n_seg)), dt::THREADS, dt::SMEM, stream, mq, mk, mv, a, n_vt,
                           dt::wait_limit_ns(), st);
    if (rc != LR_OK || !parts) return rc;
    const int64_t rows = a.B * a.L;
    return launch_early(decay_parts_kernel<false>, dim3(unsigned(rows < (1 << 20) ? rows : 1 << 20)), 256, stream, a);
}

}  // namespace lr
